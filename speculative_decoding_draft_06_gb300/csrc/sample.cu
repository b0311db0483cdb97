// Tokens drawn from rows of logits (dartree_sample).
//
// A row is the work of one thread-block cluster (one CTA where there are
// many rows).  Every cut (top-k, min-p, top-p) keeps a prefix of the order
// (logit desc, index asc), so the kept tokens are those whose 50-bit key
// (ordered logit, inverted index) is at least one threshold.
//
// The weights w = 2^((l - max) log2(e) / T) are integers in units of 2^-44
// (weight44): sums of them are exact whatever their order, so the shared
// histograms may be filled by atomics, and "mass >= top_p Z" and "running
// sum > u Z" are decided on whole numbers.  32-bit sums would not do: a row
// of 150 000 tokens has as many borders, and a running sum that is off by
// 2^-20 of the total moves the draw over one of them every few rows.
//
// Most rows are decided by about a thousand candidates (from_list):
// 1. a sample of the row gives a bound that about that many tokens reach;
// 2. one pass over the row notes the 16-byte units that hold such tokens and
//    sums the weights of all others in fp32, with a bound of the sum's error;
// 3. the candidates go to a list in shared memory; the cuts and the draw are
//    made on it in integers.  The rest of the row only enters top-p's total:
//    the row is decided if the crossing is the same at both ends of the
//    total's interval.
// A row that this does not decide (no cuts, a kept set beyond the list, a
// border inside the interval, infinities, NaN) takes further passes over the
// row itself, all in integers (whole_row).
//
// Bound, in rows that the candidates decide, by latency: a block's steps (sample,
// pass, list, cut, draw) wait for one another, and four blocks to an SM (by
// registers and shared memory) do not cover it: greedy issues 0.34 a cycle with
// DRAM at half its rate, 6 instructions a token.  Of the rows that they do not
// decide each stays with the one block that found out, 35 to 100 instructions a
// token, and the last of them set the end of the launch.
// 2064 rows of 151936 bf16 logits: greedy 149 us (4.2 TB/s, 63% of a copy),
// top-k 20 218, top-p 0.9 at T = 0.7 357 to 375, top-p 0.95 at T = 1 (85% of
// these rows by whole rows) 1065, no cut 660; 129 rows in fp32: 23, 36, 42, 188,
// 112; 17 rows of 32000 17 to 21 us, latency.
//
// A cut: a histogram of counts and masses over 1024 classes of -log2 w
// (monotone in the logit) gives the class in which it falls; the class is
// gathered (refined by digits of the key while it is large), sorted, and the
// cut's token found in it.
#include <cuda_bf16.h>

#include "block.cuh"
#include "cache.cuh"
#include "ptx.cuh"

namespace dt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1024;
constexpr float kBinsPer2 = 20.f;    // classes per power of two
constexpr float kMassUnit = 16000.f; // 2^18 2^(1/40) units fit 32 bits
constexpr int kTable = 768;          // bf16 logits of a sign whose weights are tabled
constexpr int kList = 2944;          // candidates
constexpr float kWant = 1800.f;      // candidates aimed at
constexpr int kClass = 1024;         // members of a class that are sorted
constexpr int kRanked = 128;         // members of a class that are ranked by comparisons
constexpr int kUnits = 4096;         // 16-byte units of a CTA that may hold candidates
constexpr int kMaxCl = 8;
constexpr int kIdxBits = 18;
constexpr float kZeroBelow = -46.f;  // 2^-46 rounds to 0 in units of 2^-44
constexpr int kExpBits = 10;

// 2^(j / 1024) as the sum of two floats.
struct alignas(16) ExpTable {
  float v[2 << kExpBits];  // hi, lo
};
constexpr double exp2_fraction(double x) {  // x in [0, 1): the exponential series of x ln 2
  const double t = x * 0.69314718055994530941723212145818;
  double sum = 1.0, term = 1.0;
  for (int k = 1; k < 24; ++k) {
    term *= t / k;
    sum += term;
  }
  return sum;
}
constexpr ExpTable make_exp_table() {
  ExpTable t{};
  for (int j = 0; j < (1 << kExpBits); ++j) {
    const double x = exp2_fraction(static_cast<double>(j) / (1 << kExpBits));
    t.v[2 * j] = static_cast<float>(x);
    t.v[2 * j + 1] = static_cast<float>(x - static_cast<double>(t.v[2 * j]));
  }
  return t;
}
__device__ constexpr ExpTable g_exp = make_exp_table();

struct SampleParams {
  const void* logits;
  long long row_stride;
  int V, rows, rows_per_req;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *u;
  int32_t* token;
  float* prob;
};

struct Ctl {             // the leader's decisions, read by the whole cluster
  unsigned long long prefix, mask;  // class within the bin
  unsigned long long keep;          // threshold key
  unsigned long long left, total;   // draw: mass before the token in the warp's share, whole mass
  float top;                        // the row's largest logit
  int bin, last;
  int refine;            // 1: another digit, 0: gather
  int warp;              // draw: the warp (of the cluster)
  int done;              // the list decided the row
};

struct Part {            // a CTA's share of the pass, for the leader
  float top, sum, off;
  int lost;              // more units than kUnits
};

struct Smem {
  __align__(16) float2 exp[1 << kExpBits];
  union {
    struct {
      unsigned mass_lo[kBins], mass_hi[kBins];
      unsigned count[kBins];
    };
    unsigned long long weight[2 * kTable];
    unsigned codes[2 * kTable];
  };
  unsigned long long list[kList];
  union {
    unsigned long long cls[kClass];
    uint16_t unit[kUnits];
  };
  unsigned long long wsum[kMaxCl * kWarps], wtot[kMaxCl * kWarps];
  unsigned long long scan_m[kWarps];
  unsigned scan_c[kWarps];
  float wmax[kWarps], wval[kWarps];
  __align__(16) unsigned sample[kThreads];
  float sbound, sbound2, smax;
  Part part[kMaxCl];
  unsigned list_n, units_n, cls_n;
  int picked;
  unsigned picked_n, picked_c;
  unsigned long long picked_m;
  Ctl ctl;
};

// One row's weights.
struct Weights {
  float top;      // the largest logit
  float ch, cl;   // log2(e) / T as a sum of two floats
  const float2* exp;

  // log2 of the weight, rounded to fp32 (monotone in x; x finite or -inf)
  __device__ __forceinline__ float log2w(float x) const { return x == top ? 0.f : (x - top) * ch; }

  // The weight in units of 2^-44, to about 2^-45.  l - top and its product
  // with log2(e) / T are carried as sums of two floats, the fraction is split
  // into a table entry 2^(j/1024) and |t| <= 2^-11, and 2^t - 1 =
  // t ln2 + t^2 (ln2^2/2 + t ln2^3/6) needs the low parts of its first term
  // only.
  __device__ __forceinline__ unsigned long long weight44(float x) const {
    if (x == top) return 1ull << 44;
    const float s = x - top;
    const float p = s * ch;
    if (!(p >= kZeroBelow)) return 0ull;  // (also -inf)
    const float bb = s - x;               // x - top = s + err exactly
    const float err = (x - (s - bb)) - (top + bb);
    float e = fmaf(s, ch, -p);
    e = fmaf(s, cl, e);
    e = fmaf(err, ch, e);
    // n = the nearest multiple of 1/1024 to p, by adding 1.5 2^13 (ulp 2^-10)
    const float big = p + 12288.f;
    const float t0 = p - (big - 12288.f);  // exact, |t0| <= 2^-11
    const float t = t0 + e;
    e -= t - t0;                          // t + e unchanged, |e| < 2^-35
    const int n = __float_as_int(big) - __float_as_int(12288.f);  // 1024 n
    const float2 T = exp[n & 1023];
    constexpr float kL1 = 0.693147182464599609375f;  // ln 2 = kL1 + kL1lo
    constexpr float kL1lo = -1.904654299957768e-9f;
    const float a = t * kL1;
    float b = fmaf(t, kL1, -a);
    b = fmaf(t, kL1lo, b);
    b = fmaf(e, kL1, b);
    b = fmaf(t * t, fmaf(t, 0.05550410866f, 0.24022650696f), b);  // 2^(t+e) - 1 = a + b
    const float m = T.x * a;              // |m| < 2^-10
    float lo = fmaf(T.x, a, -m);
    lo = fmaf(T.x, b, lo);
    lo = fmaf(T.y, a, lo);
    lo += T.y;                            // T (1 + a + b) = T.x + m + lo, |lo| < 2^-22
    // in units of 2^-45: T.x's mantissa, m in multiples of 2^-32 (the low bits
    // of m + 1.5 2^-9, whose ulp that is), what m has left and lo (ulp 2^-44
    // at 1.5 2^-21)
    constexpr float kC1 = 1.5f / 512.f, kC2 = 1.5f / 2097152.f;
    const float m1 = m + kC1;
    const float rest = (m - (m1 - kC1)) + lo;
    const float m2 = rest + kC2;
    const int i1 = __float_as_int(m1) - __float_as_int(kC1), i2 = __float_as_int(m2) - __float_as_int(kC2);
    const long long w45 = (static_cast<long long>((__float_as_int(T.x) & 0x7FFFFF) | 0x800000) << 22) +
                          (static_cast<long long>(i1) << 13) + 2 * i2;
    const int down = 1 - (n >> 10);       // 1 .. 47
    return static_cast<unsigned long long>((w45 + (1ll << (down - 1))) >> down);
  }
};

// (-0 + 0 = 0: the two zeros are one logit)
__device__ __forceinline__ unsigned long long key50(float x, int idx) {
  return (static_cast<unsigned long long>(float_order(x + 0.f)) << kIdxBits) |
         static_cast<unsigned>((1 << kIdxBits) - 1 - idx);
}
__device__ __forceinline__ float key50_value(unsigned long long k) {
  return order_float(static_cast<uint32_t>(k >> kIdxBits));
}

// Inclusive scan of (count, mass) over the block's threads.
__device__ __forceinline__ void block_scan(Smem& sm, unsigned& c, unsigned long long& m) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned cy = __shfl_up_sync(kFullMask, c, o);
    const unsigned long long my = __shfl_up_sync(kFullMask, m, o);
    if (lane >= o) {
      c += cy;
      m += my;
    }
  }
  if (lane == 31) {
    sm.scan_c[warp] = c;
    sm.scan_m[warp] = m;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    c += sm.scan_c[w];
    m += sm.scan_m[w];
  }
  __syncthreads();
}

template <typename E>
__device__ __forceinline__ float logit(const E* row, int i);
template <>
__device__ __forceinline__ float logit<float>(const float* row, int i) {
  const float x = __ldg(row + i);
  return x == x ? x : -INFINITY;
}
template <>
__device__ __forceinline__ float logit<uint16_t>(const uint16_t* row, int i) {
  const float x = bf16_bits_to_float(__ldg(row + i));
  return x == x ? x : -INFINITY;
}

// floor(x 2^64) for x in (0, 1).
__device__ __forceinline__ unsigned long long fraction64(float x) {
  const unsigned b = __float_as_uint(x);
  const int e = static_cast<int>(b >> 23);  // x = m 2^(e - 150), subnormals as if e were 1
  const unsigned long long m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int up = max(e, 1) - 86;
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0ull;
}

// w / z to fp32, for w <= z: both as sums of two floats (49 bits or more), the
// quotient of the upper ones corrected once.  (An fp64 division: 0.7 us.)
__device__ __forceinline__ float share_of(unsigned long long w, unsigned long long z) {
  const float wh = __ull2float_rn(w), zh = __ull2float_rn(z);
  const float wl = __ll2float_rn(static_cast<long long>(w - __float2ull_rn(wh)));
  const float zl = __ll2float_rn(static_cast<long long>(z - __float2ull_rn(zh)));
  const float q = __fdiv_rn(wh, zh);
  return q + __fdiv_rn(fmaf(-q, zh, wh) + fmaf(-q, zl, wl), zh);
}

// ceil(p z) for p in (0, 1) (fp32) and z < 2^63, at least 1.
__device__ __forceinline__ unsigned long long ceil_share(float p, unsigned long long z) {
  const unsigned long long f = fraction64(p) >> 1;
  const unsigned long long hi = __umul64hi(f, z), lo = f * z;
  const unsigned long long q = (hi << 1) | (lo >> 63);
  const unsigned long long c = q + ((lo << 1) != 0ull ? 1ull : 0ull);
  return c > 0ull ? c : 1ull;
}

// A row in 16-byte units: `head` logits before the first aligned address,
// `units` units, the rest behind them.  Warp w of the cluster's n has the
// units [w share, (w + 1) share), warp 0 the head too and warp n - 1 the
// rest: the shares follow the index order.
template <typename E>
struct Row {
  static constexpr int kPer = 16 / static_cast<int>(sizeof(E));
  const E* src;
  int V, head, units;
  __device__ __forceinline__ Row(const E* p, int v) : src(p), V(v) {
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    head = off == 0 ? 0 : (16 - off) / static_cast<int>(sizeof(E));
    head = head < v ? head : v;
    units = (v - head) / kPer;
  }
  __device__ __forceinline__ uint4 load(int u) const {
    return __ldg(reinterpret_cast<const uint4*>(src + head) + u);
  }
  __device__ __forceinline__ int index(int u) const { return head + u * kPer; }
};

template <typename E>
__device__ __forceinline__ void unpack(uint4 v, float (&x)[16 / sizeof(E)]);
template <>
__device__ __forceinline__ void unpack<float>(uint4 v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack<uint16_t>(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// The largest of a unit's logits (fmaxf drops NaN; all NaN: NaN, which no
// comparison takes).
template <int N>
__device__ __forceinline__ float max_of(const float (&x)[N]) {
  float m = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) m = fmaxf(m, x[k]);
  return m;
}

// f(unit, its number) for the lane's units of a warp's [ub, ue), with a load
// in flight ahead (three: 4% to 7% slower by their moves).
template <typename E, typename F>
__device__ __forceinline__ void each_unit(const Row<E>& row, int ub, int ue, F f) {
  int u = ub + (threadIdx.x & 31);
  auto at = [&](int q) { return q < ue ? row.load(q) : make_uint4(0, 0, 0, 0); };
  uint4 next = at(u);
#pragma unroll 1
  for (; u < ue; u += 32) {
    const uint4 v = next;
    next = at(u + 32);
    f(v, u);
  }
}

// What the cuts work on.  LIST: the leader's list of candidates, by the
// leader's block alone; otherwise the whole row, by the cluster.
template <bool LIST, typename E>
struct Source {
  Smem& sm;
  Smem& ls;
  Row<E> row;
  int ub, ue;      // the warp's units (row)
  int first, last; // 1: the warp has the head, the rest
  int n;           // list entries
  int cl;
  bool lead;
  int gw, share;   // the warp in the cluster, units per warp (row)
  using Elem = E;
  __device__ __forceinline__ void sync() const {
    if constexpr (LIST) __syncthreads();
    else cluster_sync();
  }
  // f(logit, index) for the row's logits above -inf, in no particular order
  template <typename F>
  __device__ __forceinline__ void each_value(F f) const {
    const int lane = threadIdx.x & 31;
    auto one = [&](float x, int i) {
      if (x > -INFINITY) f(x, i);  // (not NaN either)
    };
    if (first && lane < row.head) one(logit<E>(row.src, lane), lane);
    const int rest = row.index(row.units);
    if (last && lane < row.V - rest) one(logit<E>(row.src, rest + lane), rest + lane);
    each_unit(row, ub, ue, [&](uint4 v, int u) {
      float x[Row<E>::kPer];
      unpack<E>(v, x);
#pragma unroll
      for (int k = 0; k < Row<E>::kPer; ++k) one(x[k], row.index(u) + k);
    });
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {  // f(logit, key)
    if constexpr (LIST) {
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long k = sm.list[i];
        f(key50_value(k), k);
      }
    } else {
      each_value([&](float x, int i) { f(x, key50(x, i)); });
    }
  }
  // class b's sums over the cluster (leader)
  __device__ __forceinline__ void sums(int b, unsigned* c, unsigned long long* m) const {
    *c = 0;
    *m = 0;
    for (int q = 0; q < (LIST ? 1 : cl); ++q) {
      const Smem* o = LIST ? &sm : at_rank(&sm, q);
      *c += o->count[b];
      *m += (static_cast<unsigned long long>(o->mass_hi[b]) << 32) + o->mass_lo[b];
    }
  }
};

// A 64-bit sum in shared memory from two 32-bit atomics (shared memory has
// no 64-bit add): the low word's add that wraps carries.
__device__ __forceinline__ void add_mass(Smem& sm, int b, unsigned long long w) {
  const unsigned lo = static_cast<unsigned>(w);
  const unsigned old = atomicAdd(&sm.mass_lo[b], lo);
  const unsigned hi = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(&sm.mass_hi[b], hi);
}

__device__ __forceinline__ void clear_classes(Smem& sm) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    sm.mass_lo[i] = 0;
    sm.mass_hi[i] = 0;
    sm.count[i] = 0;
  }
}

// Among the classes (ascending class = descending order) finds the one in
// which the running count or mass reaches `target`; the leader's block.
// c_before, m_before: what lies before the first class, then before the one
// found.  Returns the class; *members: its count.
template <typename S>
__device__ __forceinline__ int pick_class(const S& s, bool by_count, unsigned long long target, unsigned& c_before,
                                          unsigned long long& m_before, unsigned* members) {
  constexpr int kPer = kBins / kThreads;
  Smem& sm = s.sm;
  unsigned cs[kPer], c = 0;
  unsigned long long ms[kPer], m = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    s.sums(threadIdx.x * kPer + j, &cs[j], &ms[j]);
    c += cs[j];
    m += ms[j];
  }
  unsigned bc = c_before - c;
  unsigned long long bm = m_before - m;
  block_scan(sm, c, m);
  bc += c;
  bm += m;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (by_count ? (bc < target && target <= bc + cs[j]) : (bm < target && target <= bm + ms[j])) {
      sm.picked = threadIdx.x * kPer + j;
      sm.picked_n = cs[j];
      sm.picked_c = bc;
      sm.picked_m = bm;
    }
    bc += cs[j];
    bm += ms[j];
  }
  __syncthreads();
  c_before = sm.picked_c;
  m_before = sm.picked_m;
  *members = sm.picked_n;
  const int k = sm.picked;
  __syncthreads();
  return k;
}

constexpr float kBinBig = 12582912.f;

// The classes of the cuts: -log2 w in steps of 1 / kBinsPer2, to the nearest
// (by adding 1.5 2^23, whose ulp is 1).
__device__ __forceinline__ int bin_of_log2(float y) {
  return min(kBins - 1, __float_as_int(fmaf(y, -kBinsPer2, kBinBig)) - __float_as_int(kBinBig));
}
__device__ __forceinline__ int bin_of(const Weights& wt, float x) { return bin_of_log2(wt.log2w(x)); }

// The element at which the running count (by_count) or mass in the order
// reaches `target`: its key becomes `keep`; the mass up to and with it is
// left in the leader's *upto.  The bins' sums are in place.  All threads of
// the source call it.  Returns whether the bins' sums were used for digits
// (else those before the cut's bin still hold).
template <typename S>
__device__ bool cut(const S& s, const Weights& wt, bool by_count, unsigned long long target,
                    unsigned long long& keep, unsigned long long* upto) {
  Smem& sm = s.sm;
  Ctl& ctl = s.ls.ctl;
  unsigned c_before = 0, members = 0;
  unsigned long long m_before = 0;
  if (s.lead) {
    const int b = pick_class(s, by_count, target, c_before, m_before, &members);
    if (threadIdx.x == 0) {
      ctl.bin = b;
      ctl.prefix = ctl.mask = 0;
      ctl.refine = members > kClass;
    }
  }
  s.sync();
  // a class too large to be gathered: by digits of its keys, 10 bits each
  bool refined = false;
  for (int shift = 40; ctl.refine; shift -= 10) {
    refined = true;
    const int bin = ctl.bin;
    const unsigned long long pre = ctl.prefix, msk = ctl.mask;
    clear_classes(sm);
    __syncthreads();
    s.each([&](float x, unsigned long long key) {
      if (key < keep || (key & msk) != pre || bin_of(wt, x) != bin) return;
      const unsigned long long w = wt.weight44(x);
      if (w == 0) return;
      const int d = 1023 - static_cast<int>((key >> shift) & 1023);
      atomicAdd(&sm.count[d], 1u);
      add_mass(sm, d, w);
    });
    s.sync();
    if (s.lead) {
      const int d = pick_class(s, by_count, target, c_before, m_before, &members);
      if (threadIdx.x == 0) {
        ctl.prefix |= static_cast<unsigned long long>(1023 - d) << shift;
        ctl.mask |= 1023ull << shift;
        ctl.refine = members > kClass;
      }
    }
    s.sync();
  }
  {
    const int bin = ctl.bin;
    const unsigned long long pre = ctl.prefix, msk = ctl.mask;
    s.each([&](float x, unsigned long long key) {
      if (key < keep || (key & msk) != pre || bin_of(wt, x) != bin || wt.weight44(x) == 0) return;
      const unsigned at = atomicAdd(&s.ls.cls_n, 1u);
      if (at < kClass) s.ls.cls[at] = key;
    });
  }
  s.sync();
  if (s.lead) {
    const int n = min(static_cast<int>(sm.cls_n), kClass);
    if (n <= kRanked) {
      // few: each thread adds up what precedes its member
      const int i = threadIdx.x;
      unsigned long long key = 0, w = 0;
      if (i < n) {
        key = sm.cls[i];
        w = wt.weight44(key50_value(key));
        sm.cls[kRanked + i] = w;
      }
      __syncthreads();
      if (i < n) {
        unsigned bc = c_before;
        unsigned long long bm = m_before;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const bool before = sm.cls[j] > key;
          bc += before;
          bm += before ? sm.cls[kRanked + j] : 0ull;
        }
        if (by_count ? bc + 1 == target : (bm < target && target <= bm + w)) {
          ctl.keep = key;
          sm.picked_m = bm + w;
        }
      }
    } else {
      const int n2 = pow2_at_least(n);
      for (int i = n + threadIdx.x; i < n2; i += kThreads) sm.cls[i] = 0;
      __syncthreads();
      block_sort_desc(reinterpret_cast<uint64_t*>(sm.cls), n2);
      constexpr int kQ = kClass / kThreads;
      unsigned long long ms[kQ], m = 0;
      unsigned c = 0;
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const int i = threadIdx.x * kQ + j;
        ms[j] = i < n ? wt.weight44(key50_value(sm.cls[i])) : 0ull;
        c += i < n ? 1u : 0u;
        m += ms[j];
      }
      unsigned bc = c_before - c;
      unsigned long long bm = m_before - m;
      block_scan(sm, c, m);
      bc += c;
      bm += m;
#pragma unroll
      for (int j = 0; j < kQ; ++j) {
        const int i = threadIdx.x * kQ + j;
        if (i < n && (by_count ? bc + 1 == target : (bm < target && target <= bm + ms[j]))) {
          ctl.keep = sm.cls[i];
          sm.picked_m = bm + ms[j];
        }
        bc += i < n ? 1u : 0u;
        bm += ms[j];
      }
    }
    if (threadIdx.x == 0) sm.cls_n = 0;
    __syncthreads();
    *upto = sm.picked_m;
  }
  s.sync();
  keep = ctl.keep;
  return refined;
}

// A request's settings for a row.
struct Rule {
  float tp, mp;
  int k;
  bool use_k, use_p;
};

// Smallest key whose weight is at least min_p: 32 probes a round over the
// ordered logits (every warp finds the same).
__device__ unsigned long long min_p_key(const Weights& wt, float mp) {
  const int lane = threadIdx.x & 31;
  const unsigned long long need = static_cast<unsigned long long>(ceil(ldexp(static_cast<double>(mp), 44)));
  unsigned lo = 0, hi = float_order(wt.top);  // the answer lies in (lo, hi]
  while (hi - lo > 1) {
    const unsigned step = (hi - lo + 31) / 32;
    const unsigned long long at = static_cast<unsigned long long>(lo) + static_cast<unsigned long long>(lane + 1) * step;
    const bool in = at >= hi || wt.weight44(order_float(static_cast<unsigned>(at))) >= need;
    const int f = __ffs(__ballot_sync(kFullMask, in)) - 1;  // (the last probe is at or behind hi)
    const unsigned long long nhi = static_cast<unsigned long long>(lo) + static_cast<unsigned long long>(f + 1) * step;
    lo += static_cast<unsigned>(f) * step;
    hi = nhi < hi ? static_cast<unsigned>(nhi) : hi;
  }
  return static_cast<unsigned long long>(hi) << kIdxBits;
}

// floor(u total) for the draw, below total.
__device__ __forceinline__ unsigned long long draw_mark(float u, unsigned long long total) {
  unsigned long long t = 0;
  if (u > 0.f)
    t = u >= 1.f ? total : __umul64hi(fraction64(u), total);
  return t < total ? t : total - 1;
}

// The row's classes: counts and masses of what is above `keep`.
template <typename S>
__device__ void fill_bins(const S& s, const Weights& wt, unsigned long long keep) {
  clear_classes(s.sm);
  __syncthreads();
  s.each([&](float x, unsigned long long key) {
    if (key < keep) return;
    const unsigned long long w = wt.weight44(x);
    if (w == 0) return;
    const int b = bin_of(wt, x);
    atomicAdd(&s.sm.count[b], 1u);
    add_mass(s.sm, b, w);
  });
  s.sync();
}

// Count and mass over all classes (leader's block).
template <typename S>
__device__ void all_classes(const S& s, unsigned* count, unsigned long long* mass) {
  constexpr int kPer = kBins / kThreads;
  unsigned c = 0, cj;
  unsigned long long m = 0, mj;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    s.sums(threadIdx.x * kPer + j, &cj, &mj);
    c += cj;
    m += mj;
  }
  block_scan(s.sm, c, m);
  if (threadIdx.x == kThreads - 1) {
    s.sm.picked_c = c;
    s.sm.picked_m = m;
  }
  __syncthreads();
  *count = s.sm.picked_c;
  *mass = s.sm.picked_m;
  __syncthreads();
}

// bf16 logits near the largest are few different values: kTable codes downward
// from it and kTable negative ones from -1/4 (or from it, if that is lower)
// have places, in descending order.  What lies between the two and what lies
// below them has none.
// (Behind the last place of an extreme largest logit lies -inf: weight 0.)
struct Codes {
  int top, neg0;
  __device__ __forceinline__ explicit Codes(float t) {
    top = __float_as_int(t) >> 16;
    neg0 = max(0x3E80, top < 0 ? top & 0x7FFF : 0);
  }
  // the place or -1
  __device__ __forceinline__ int place(float x) const {
    const int b = __float_as_int(x) >> 16;
    const int j = b < 0 ? (b & 0x7FFF) - neg0 : top - b;
    return static_cast<unsigned>(j) < kTable ? j + (b < 0 ? kTable : 0) : -1;
  }
  // x without a place: whether it lies below them all
  __device__ __forceinline__ bool below(float x) const {
    const int b = __float_as_int(x) >> 16;
    return b < 0 && (b & 0x7FFF) >= neg0;
  }
  // whether zero has no place (its two codes would be two logits)
  __device__ __forceinline__ bool sound() const { return top >= kTable || top < 0; }
  __device__ __forceinline__ float value(int j) const {  // (-inf behind the last)
    const int code = j < kTable ? max(top - j, 0) : 0x8000 | min(neg0 + j - kTable, 0x7F80);
    return bf16_bits_to_float(static_cast<uint16_t>(code));
  }
  __device__ __forceinline__ unsigned long long weight(const Weights& wt, int j) const {
    const float x = value(j);
    return x > -INFINITY && x <= wt.top ? wt.weight44(x) : 0ull;
  }
};

// coded(x, index, place) and other(x, index) for the row's bf16 logits, in no
// particular order, but for -inf and NaN without a place.
template <typename S, typename F, typename G>
__device__ __forceinline__ void each_code(const S& s, const Codes& c, F coded, G other) {
  using E = typename S::Elem;
  constexpr int kPer = Row<E>::kPer;
  const int lane = threadIdx.x & 31;
  auto one = [&](float x, int i) {
    const int j = c.place(x);
    if (j >= 0) coded(x, i, j);
    else if (x > -INFINITY) other(x, i);
  };
  if (s.first && lane < s.row.head) one(logit<E>(s.row.src, lane), lane);
  const int rest = s.row.index(s.row.units);
  if (s.last && lane < s.row.V - rest) one(logit<E>(s.row.src, rest + lane), rest + lane);
  each_unit(s.row, s.ub, s.ue, [&](uint4 v, int u) {
    float x[kPer];
    unpack<E>(v, x);
    unsigned others = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int j = c.place(x[k]);
      if (j >= 0) coded(x[k], s.row.index(u) + k, j);
      else others |= 1u << k;
    }
    for (; others; others &= others - 1) {
      const int k = __ffs(others) - 1;
      const uint32_t pair = k < 4 ? (k < 2 ? v.x : v.y) : (k < 6 ? v.z : v.w);
      const float y = __uint_as_float(k & 1 ? pair & 0xFFFF0000u : pair << 16);
      if (y > -INFINITY) other(y, s.row.index(u) + k);
    }
  });
}

// f(logit, index, weight) for the row's logits that have a weight (and some
// without), in no particular order; the classes' memory is used.  The weights of the codes that have
// places come from a table (weight44 is some 70 instructions: 2064 rows of
// 151936 without cuts take 670 us, 1050 without the table).
template <typename S, typename F>
__device__ __forceinline__ void each_weight(const S& s, const Weights& wt, F f) {
  if constexpr (sizeof(typename S::Elem) == 4) {
    s.each_value([&](float x, int i) { f(x, i, wt.weight44(x)); });
  } else {
    const Codes c(wt.top);
    for (int j = threadIdx.x; j < 2 * kTable; j += kThreads) s.sm.weight[j] = c.weight(wt, j);
    __syncthreads();
    each_code(s, c, [&](float x, int i, int j) { f(x, i, s.sm.weight[j]); },
              [&](float x, int i) { f(x, i, wt.weight44(x)); });
  }
}

// top-k and top-p of a bf16 row by counts of its codes: they and the codes'
// weights give the running counts and masses exactly, so a cut falls on a code
// and a number of its ties, the first in index order.  Left are that value
// (*value), the kept tokens' mass per warp in wsum and the number of ties a
// warp keeps in wtot.  False where a cut falls on a logit without a place.
// (2064 rows of 151936, top-p 0.95: at T = 1 1090 us, with the approximate
// classes below 1300; at T = 1.3 1110 and 2120, where many rows had more tied
// tokens about the cut than the list holds.)
template <typename S>
__device__ bool code_cuts(const S& s, const Weights& wt, const Rule& rule, float* value) {
  Smem& sm = s.sm;
  Ctl& ctl = s.ls.ctl;
  const int tid = threadIdx.x, lane = tid & 31, warps = s.cl * kWarps;
  constexpr int kN = 2 * kTable + 2, kPer = (kN + kThreads - 1) / kThreads;
  const Codes code(wt.top);
  if (!code.sound()) return false;
  float v = -INFINITY;
  {
    for (int j = tid; j < 2 * kTable; j += kThreads) sm.codes[j] = 0;
    __syncthreads();
    unsigned between = 0, below = 0;
    unsigned long long between_m = 0, below_m = 0;
    each_code(s, code, [&](float, int, int j) { atomicAdd(&sm.codes[j], 1u); },
              [&](float x, int) {
                const unsigned long long w = wt.weight44(x);
                const bool low = code.below(x);
                between += !low;
                below += low;
                between_m += low ? 0ull : w;
                below_m += low ? w : 0ull;
              });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      between += __shfl_xor_sync(kFullMask, between, o);
      below += __shfl_xor_sync(kFullMask, below, o);
      between_m += __shfl_xor_sync(kFullMask, between_m, o);
      below_m += __shfl_xor_sync(kFullMask, below_m, o);
    }
    if (lane == 0) {  // (the list is not in use)
      unsigned long long* to = &s.ls.list[4 * s.gw];
      to[0] = between;
      to[1] = between_m;
      to[2] = below;
      to[3] = below_m;
    }
    s.sync();
    if (s.lead) {
      // entries in order: the positive codes, what lies between, the negative
      // codes, what lies below
      unsigned cs[kPer], c = 0;
      unsigned long long ms[kPer], m = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) cs[q] = 0;
      for (int r = 0; r < s.cl; ++r) {
        const unsigned* from = at_rank(&sm, r)->codes;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int e = tid * kPer + q;
          if (e < kN - 1 && e != kTable) cs[q] += from[e < kTable ? e : e - 1];
        }
      }
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int e = tid * kPer + q;
        ms[q] = 0;
        if (e == kTable || e == kN - 1) {
#pragma unroll 8
          for (int w = 0; w < warps; ++w) {
            cs[q] += static_cast<unsigned>(sm.list[4 * w + (e == kN - 1 ? 2 : 0)]);
            ms[q] += sm.list[4 * w + (e == kN - 1 ? 3 : 1)];
          }
        } else if (cs[q]) {
          ms[q] = cs[q] * code.weight(wt, e < kTable ? e : e - 1);
        }
        c += cs[q];
        m += ms[q];
      }
      unsigned c0 = 0u - c;
      unsigned long long m0 = 0ull - m;
      block_scan(sm, c, m);
      c0 += c;
      m0 += m;  // what lies before the thread's entries
      if (tid == kThreads - 1) {
        sm.picked = -1;
        sm.picked_c = c;
        sm.picked_m = m;
      }
      __syncthreads();
      unsigned long long Z = sm.picked_m;
      bool ok = true;
      // the entry that a cut falls on, and how many of its tokens are kept
      auto fall = [&](bool by_count, unsigned long long target) {
        unsigned bc = c0;
        unsigned long long bm = m0;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          if (by_count ? (bc < target && target <= bc + cs[q]) : (bm < target && target <= bm + ms[q])) {
            const int e = tid * kPer + q;
            const unsigned long long w = max(ms[q] / cs[q], 1ull);
            const unsigned n = by_count ? static_cast<unsigned>(target - bc)
                                        : static_cast<unsigned>((target - bm + w - 1) / w);
            sm.picked = e == kTable || e == kN - 1 ? -2 : e < kTable ? e : e - 1;
            sm.picked_n = n;
            sm.picked_m = ms[q] ? bm + n * w : bm;  // (an entry without a place: not used)
          }
          bc += cs[q];
          bm += ms[q];
        }
        __syncthreads();
        if (sm.picked == -2) ok = false;
        Z = sm.picked_m;
        __syncthreads();
      };
      const unsigned all = sm.picked_c;
      __syncthreads();
      if (rule.use_k && all > static_cast<unsigned>(rule.k)) fall(true, static_cast<unsigned long long>(rule.k));
      if (rule.use_p && ok && Z > 0) fall(false, rule.tp > 0.f ? ceil_share(rule.tp, Z) : 1ull);
      if (tid == 0) {
        ctl.bin = sm.picked;
        ctl.left = sm.picked < 0 ? 0 : sm.picked_n;
        ctl.refine = ok ? 0 : 1;
      }
    }
    s.sync();
    if (ctl.refine) return false;
    if (ctl.bin >= 0) v = code.value(ctl.bin);
  }
  // the weights of what is above the cut's code, and its ties
  for (int j = tid; j < 2 * kTable; j += kThreads) sm.weight[j] = code.value(j) > v ? code.weight(wt, j) : 0ull;
  __syncthreads();
  unsigned long long sum = 0;
  unsigned ties = 0;
  each_code(s, code,
            [&](float x, int, int j) {
              sum += sm.weight[j];
              ties += x == v;
            },
            [&](float x, int) { sum += x > v ? wt.weight44(x) : 0ull; });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(kFullMask, sum, o);
    ties += __shfl_xor_sync(kFullMask, ties, o);
  }
  if (lane == 0) {
    s.ls.wsum[s.gw] = sum;
    s.ls.wtot[s.gw] = ties;
  }
  s.sync();
  if (s.lead && tid == 0 && v > -INFINITY) {
    const unsigned long long w = wt.weight44(v);
    unsigned long long left = ctl.left;
    for (int k = 0; k < warps; ++k) {
      const unsigned long long n = min(left, sm.wtot[k]);
      sm.wsum[k] += n * w;
      sm.wtot[k] = n;
      left -= n;
    }
  }
  *value = v;
  return true;
}

// The kept tokens' mass per warp, left in the leader's wsum.
template <typename S>
__device__ void whole_sums(const S& s, const Weights& wt, unsigned long long keep) {
  unsigned long long sum = 0;
  const float kx = key50_value(keep);
  const bool any = keep == 0;
  each_weight(s, wt, [&](float x, int i, unsigned long long w) {
    if (any || (x >= kx && key50(x, i) >= keep)) sum += w;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
  if ((threadIdx.x & 31) == 0) s.ls.wsum[s.gw] = sum;
}

// top-p alone, or no cut: one exact pass over the row.
// A histogram of approximate class masses (in units of kMassUnit of the
// class's middle weight, one 32-bit sum: 2^18 tokens fit) tells the classes
// [c1, c2] in which the running mass passes top_p of the whole, with room for
// the masses' error.  The exact pass then sums all
// weights and those of the classes before c1, and gathers the tokens of c1 ..
// c2, among which the cut falls.  False if it does not, or if they are too
// many; else the kept tokens' mass per warp is in wsum.
template <typename S>
__device__ bool nucleus(const S& s, const Weights& wt, const Rule& rule, unsigned long long& keep) {
  Smem& sm = s.sm;
  Ctl& ctl = s.ls.ctl;
  const int tid = threadIdx.x, lane = tid & 31;
  keep = 0;
  if (!rule.use_p) {
    whole_sums(s, wt, keep);
    return true;
  }
  clear_classes(sm);
  if (s.lead && tid == 0) sm.list_n = 0;
  __syncthreads();
  s.each_value([&](float x, int) {
    const float y = wt.log2w(x);
    if (!(y >= kZeroBelow)) return;
    // (bin_of_log2's class, at most 920, and the mass by additions of 1.5 2^23
    // and 2^23: conversions are slower)
    const float z = fmaf(y, -kBinsPer2, kBinBig);
    const float w = ex2(fmaf(z - kBinBig, 1.f / kBinsPer2, y));  // 2^(-1/40) .. 2^(1/40)
    atomicAdd(&sm.mass_lo[__float_as_int(z) - __float_as_int(kBinBig)],
              __float_as_uint(fmaf(w, kMassUnit, 8388608.f)) & 0x7FFFFFu);
  });
  s.sync();
  if (s.lead) {
    constexpr int kPer = kBins / kThreads;
    float ms[kPer], m = 0.f;
    float cs[kPer];  // tokens, about
    static_assert(kPer == 4, "a thread's classes are one 16-byte load");
    unsigned units[kPer] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < kMaxCl; ++q) {  // (the CTAs' loads together)
      if (q >= s.cl) continue;
      const uint4 x = *reinterpret_cast<const uint4*>(&at_rank(&sm, q)->mass_lo[tid * kPer]);
      units[0] += x.x;
      units[1] += x.y;
      units[2] += x.z;
      units[3] += x.w;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      cs[j] = static_cast<float>(units[j]) * (1.f / kMassUnit);
      ms[j] = cs[j] * ex2(static_cast<float>(tid * kPer + j) * (-1.f / kBinsPer2));
      m += ms[j];
    }
    float inc = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(kFullMask, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sm.wval[tid >> 5] = inc;
    if (tid == 0) {
      ctl.bin = kBins;
      ctl.last = kBins;
    }
    __syncthreads();
    float before = inc - m, all = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (w < (tid >> 5)) before += sm.wval[w];
      all += sm.wval[w];
    }
    // (a token's mass is rounded by 2^-15 of itself, the fp32 sums add 2^-18 of
    // the whole)
    const float t1 = fmaxf(rule.tp, 0.f) * all - all * (1.f / 16384.f), t2 = t1 + all * (2.f / 16384.f);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = tid * kPer + j;
      const float after = before + ms[j];
      if (cs[j] > 0.f && after >= t1) atomicMin(&ctl.bin, c);
      if (cs[j] > 0.f && after >= t2) atomicMin(&ctl.last, c);
      before = after;
    }
    __syncthreads();
    unsigned members = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = tid * kPer + j;
      if (c >= ctl.bin && c <= ctl.last) members += static_cast<unsigned>(cs[j]);
    }
    atomicAdd(&sm.list_n, members);
    __syncthreads();
    if (tid == 0) {
      ctl.refine = sm.list_n > kList ? 1 : 0;
      sm.list_n = 0;
    }
  }
  s.sync();
  if (ctl.refine) return false;
  const int c1 = ctl.bin, c2 = ctl.last;
  unsigned long long above = 0, total = 0;
  each_weight(s, wt, [&](float x, int i, unsigned long long w) {
    const int b = bin_of(wt, x);
    total += w;
    if (b < c1) above += w;
    else if (b <= c2 && w != 0) {
      const unsigned at = atomicAdd(&s.ls.list_n, 1u);
      if (at < kList) s.ls.list[at] = key50(x, i);
    }
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    above += __shfl_xor_sync(kFullMask, above, o);
    total += __shfl_xor_sync(kFullMask, total, o);
  }
  if (lane == 0) {
    s.ls.wsum[s.gw] = above;
    s.ls.wtot[s.gw] = total;
  }
  s.sync();
  if (s.lead) {
    const int n = static_cast<int>(sm.list_n), warps = s.cl * kWarps;
    unsigned long long A = 0, Z = 0;
    for (int w = 0; w < warps; ++w) {
      A += sm.wsum[w];
      Z += sm.wtot[w];
    }
    const unsigned long long target = rule.tp > 0.f ? ceil_share(rule.tp, Z) : 1ull;
    const Source<true, typename S::Elem> l{sm, sm, s.row, 0, 0, 0, 0, n, 1, true, 0, 1};
    bool ok = n <= kList && target > A;
    if (ok) {
      fill_bins(l, wt, 0);
      unsigned count;
      unsigned long long in;
      all_classes(l, &count, &in);
      ok = target - A <= in;
      if (ok) {
        unsigned long long upto;
        cut(l, wt, false, target - A, keep, &upto);
        // the kept ones among them to their warps' masses
        clear_classes(sm);
        __syncthreads();
        l.each([&](float x, unsigned long long key) {
          if (key < keep) return;
          const int i = (1 << kIdxBits) - 1 - static_cast<int>(static_cast<unsigned>(key) & ((1u << kIdxBits) - 1));
          const int u = (i - s.row.head) / Row<typename S::Elem>::kPer;
          const int w = i < s.row.head ? 0 : u >= s.row.units ? warps - 1 : u / s.share;
          add_mass(sm, w, wt.weight44(x));
        });
        __syncthreads();
        for (int w = tid; w < warps; w += kThreads)
          sm.wsum[w] += (static_cast<unsigned long long>(sm.mass_hi[w]) << 32) + sm.mass_lo[w];
      }
    }
    __syncthreads();
    if (tid == 0) {
      ctl.keep = keep;
      ctl.refine = ok ? 0 : 1;
    }
  }
  s.sync();
  keep = ctl.keep;
  return ctl.refine == 0;
}

template <typename E>
__device__ bool from_list(const SampleParams& p, Smem& sm, int row, int n, unsigned long long bound_key,
                          unsigned long long tail, unsigned long long tail_err, const Weights& wt, const Rule& rule);

// top-k that the candidates did not decide (too many or fewer than k): a
// histogram of counts gives the class in which the k-th falls, and the tokens
// up to that class are the candidates.  False where they do not fit the list.
template <typename S>
__device__ bool k_list(const S& s, const SampleParams& p, int row, const Weights& wt, const Rule& rule) {
  Smem& sm = s.sm;
  Ctl& ctl = s.ls.ctl;
  clear_classes(sm);
  if (s.lead && threadIdx.x == 0) sm.list_n = 0;
  __syncthreads();
  s.each_value([&](float x, int) { atomicAdd(&sm.count[bin_of(wt, x)], 1u); });
  s.sync();
  if (s.lead) {
    unsigned total, c = 0, members = 0;
    unsigned long long none = 0;
    all_classes(s, &total, &none);
    const unsigned k = static_cast<unsigned>(rule.k);
    const int b = total > k ? pick_class(s, true, k, c, none, &members) : kBins;
    if (threadIdx.x == 0) {
      ctl.bin = b;
      ctl.refine = (total > k ? c + members : total) > kList;
    }
  }
  s.sync();
  if (ctl.refine) return false;
  const int b = ctl.bin;
  s.each_value([&](float x, int i) {
    if (bin_of(wt, x) <= b) s.ls.list[atomicAdd(&s.ls.list_n, 1u)] = key50(x, i);
  });
  s.sync();
  if (s.lead) {
    const int n = static_cast<int>(sm.list_n);
    unsigned long long least = ~0ull;
    for (int i = threadIdx.x; i < n; i += kThreads) least = min(least, sm.list[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(kFullMask, least, o));
    if ((threadIdx.x & 31) == 0) sm.scan_m[threadIdx.x >> 5] = least;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) least = min(least, sm.scan_m[w]);
    __syncthreads();
    // (all of the row's tokens, or the first k and some: nothing else is kept)
    if (b == kBins) least = static_cast<unsigned long long>(float_order(-INFINITY)) << kIdxBits;
    const bool ok = from_list<typename S::Elem>(p, sm, row, n, least, 0, 0, wt, rule);
    if (threadIdx.x == 0) {
      ctl.refine = ok ? 0 : 1;
      sm.cls_n = 0;
    }
  }
  s.sync();
  return ctl.refine == 0;
}

// The whole row, every decision on integer sums over it.
template <typename E>
__device__ void whole_row(const SampleParams& p, Smem& sm, Smem& ls, const E* src, int row, int cl, int rank,
                          const Weights& wt, const Rule& rule, bool greedy) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Row<E> rw(src, p.V);
  const int gw = rank * kWarps + warp, gn = cl * kWarps;
  const int share = (rw.units + gn - 1) / gn;
  const int ub = min(rw.units, gw * share), ue = min(rw.units, ub + share);
  const Source<false, E> s{sm, ls, rw, ub, ue, gw == 0, gw == gn - 1, 0, cl, rank == 0, gw, max(share, 1)};
  if (greedy) {  // the lowest index of the largest logit
    unsigned long long best = 0;
    s.each([&](float x, unsigned long long key) { best = max(best, key); });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
    if (lane == 0) ls.wsum[rank * kWarps + warp] = best;
    cluster_sync();
    if (s.lead && tid == 0) {
      for (int w = 0; w < cl * kWarps; ++w) best = max(best, sm.wsum[w]);
      p.token[row] = (1 << kIdxBits) - 1 - static_cast<int>(best & ((1u << kIdxBits) - 1));
      p.prob[row] = 1.f;
    }
    return;
  }
  unsigned long long keep = 0;
  float value = 0.f;
  bool coded = false;  // kept are the logits above `value` and the first of its ties
  if (rule.use_k && rule.k <= kList && k_list(s, p, row, wt, rule)) return;
  if constexpr (sizeof(E) == 2)
    coded = (rule.use_k || rule.use_p) && !(rule.mp > 0.f) && isfinite(wt.top) && code_cuts(s, wt, rule, &value);
  const bool quick = coded || (!rule.use_k && !(rule.mp > 0.f) && nucleus(s, wt, rule, keep));
  if (!quick) {
    keep = rule.mp > 0.f ? min_p_key(wt, rule.mp) : 0;
    if (rule.use_k || rule.use_p) {
      fill_bins(s, wt, keep);
      unsigned count = 0;
      unsigned long long Z = 0;
      if (s.lead) {
        all_classes(s, &count, &Z);
        if (tid == 0) ls.ctl.warp = rule.use_k && count > static_cast<unsigned>(rule.k);
      }
      cluster_sync();
      const bool refined = ls.ctl.warp && cut(s, wt, true, static_cast<unsigned long long>(rule.k), keep, &Z);
      if (rule.use_p) {
        unsigned long long upto;
        if (refined) fill_bins(s, wt, keep);
        cut(s, wt, false, rule.tp > 0.f && s.lead ? ceil_share(rule.tp, Z) : 1ull, keep, &upto);
      }
    }
    whole_sums(s, wt, keep);
  }
  cluster_sync();
  if (s.lead && warp == 0) {
    const int n = cl * kWarps;
    unsigned long long total = 0;
    for (int i = lane; i < n; i += 32) total += sm.wsum[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    if (lane == 0) {
      unsigned long long t = draw_mark(p.u[row], total);
      int w = 0;
      while (w < n - 1 && t >= sm.wsum[w]) t -= sm.wsum[w++];
      sm.ctl.warp = w;
      sm.ctl.left = t;
      sm.ctl.total = total;
    }
  }
  cluster_sync();
  if (ls.ctl.warp == rank * kWarps + warp) {
    // the warp's tokens in index order: the head, units of kPer tokens by the
    // lanes, the rest
    const unsigned long long t = ls.ctl.left, total = ls.ctl.total;
    unsigned long long before = 0;
    int ties = coded ? static_cast<int>(ls.wtot[gw]) : 0;  // that are still kept
    constexpr int kPer = Row<E>::kPer;
    auto step = [&](const float (&x)[kPer], int i0, int n) {  // the lane's n tokens from i0; true: found
      unsigned long long w[kPer], sum = 0;
      int tie = ties;  // that are still kept from the lane's first on
      if (coded) {
        int own = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) own += k < n && x[k] == value;
        int inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFullMask, inc, o);
          if (lane >= o) inc += y;
        }
        tie -= inc - own;
        ties -= __shfl_sync(kFullMask, inc, 31);
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        bool in = k < n && x[k] > -INFINITY;
        if (coded) in = in && (x[k] > value || (x[k] == value && tie-- > 0));
        else in = in && key50(x[k], i0 + k) >= keep;
        w[k] = in ? wt.weight44(x[k]) : 0ull;
        sum += w[k];
      }
      unsigned long long inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFullMask, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(kFullMask, before + inc > t);
      if (hit && lane == __ffs(hit) - 1) {
        unsigned long long c = before + inc - sum;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          if (c <= t && c + w[k] > t) {
            p.token[row] = i0 + k;
            p.prob[row] = share_of(w[k], total);
          }
          c += w[k];
        }
      }
      before += __shfl_sync(kFullMask, inc, 31);
      return hit != 0;
    };
    bool found = false;
    float x[kPer];
    if (gw == 0 && rw.head > 0) {
      x[0] = lane < rw.head ? logit<E>(src, lane) : -INFINITY;
      found = step(x, lane, lane < rw.head ? 1 : 0);
    }
    for (int b = ub; b < ue && !found; b += 32) {
      const int u = b + lane;
      if (u < ue) unpack<E>(rw.load(u), x);
      found = step(x, rw.index(u), u < ue ? kPer : 0);
    }
    const int rest = rw.index(rw.units);
    if (!found && gw == gn - 1 && rest < p.V) {
      x[0] = rest + lane < p.V ? logit<E>(src, rest + lane) : -INFINITY;
      step(x, rest + lane, rest + lane < p.V ? 1 : 0);
    }
  }
}

// The candidates in the leader's list (its block): all tokens whose logit is
// at least the bound's; the other tokens weigh `tail` together, at most
// tail_err off (units of 2^-44).  False where they do not decide the row.
template <typename E>
__device__ bool from_list(const SampleParams& p, Smem& sm, int row, int n, unsigned long long bound_key,
                          unsigned long long tail, unsigned long long tail_err, const Weights& wt, const Rule& rule) {
  const int tid = threadIdx.x;
  const Source<true, E> s{sm, sm, Row<E>(nullptr, 0), 0, 0, 0, 0, n, 1, true, 0, 1};
  unsigned long long keep = bound_key;
  bool all = key50_value(bound_key) == -INFINITY;  // nothing below `keep` is kept (the list has every token)
  if (rule.mp > 0.f) {
    const unsigned long long mk = min_p_key(wt, rule.mp);
    if (mk >= bound_key) {
      keep = mk;
      all = true;
    } else if (all) {
      keep = mk;
    }
  }
  fill_bins(s, wt, keep);
  unsigned count;
  unsigned long long Z;
  all_classes(s, &count, &Z);
  // (count is that of the tokens with a weight; the list may hold k with fewer)
  if (rule.use_k && n >= rule.k) {
    if (count > static_cast<unsigned>(rule.k)) {
      if (cut(s, wt, true, static_cast<unsigned long long>(rule.k), keep, &Z) && rule.use_p) fill_bins(s, wt, keep);
    }
    all = true;
  }
  // (top-k or min-p beyond the candidates, or nothing cut but the tail)
  if (!all && (rule.use_k || rule.mp > 0.f || !rule.use_p)) return false;
  if (all) tail = tail_err = 0;
  if (rule.use_p) {
    const unsigned long long lo = rule.tp > 0.f ? ceil_share(rule.tp, Z + tail - tail_err) : 1ull;
    const unsigned long long hi = rule.tp > 0.f ? ceil_share(rule.tp, Z + tail + tail_err) : 1ull;
    if (hi > Z) return false;
    cut(s, wt, false, lo, keep, &Z);
    if (hi > Z) return false;  // (the interval's other end falls on a later token)
  }
  // the draw: masses by index (256 to a class), then the class's tokens
  const unsigned long long t = draw_mark(p.u[row], Z);
  clear_classes(sm);
  __syncthreads();
  auto inverted = [](unsigned long long key) { return static_cast<unsigned>(key) & ((1u << kIdxBits) - 1); };
  s.each([&](float x, unsigned long long key) {
    if (key >= keep) add_mass(sm, 1023 - static_cast<int>(inverted(key) >> 8), wt.weight44(x));  // ascending index
  });
  __syncthreads();
  unsigned c0 = 0, members;
  unsigned long long before = 0;
  const unsigned c = pick_class(s, false, t + 1, c0, before, &members);
  s.each([&](float x, unsigned long long key) {
    if (key < keep || 1023 - (inverted(key) >> 8) != c) return;
    const unsigned at = atomicAdd(&sm.cls_n, 1u);  // (at most 256)
    sm.cls[at] = (static_cast<unsigned long long>(inverted(key)) << 32) | (key >> kIdxBits);
  });
  __syncthreads();
  const int m = static_cast<int>(sm.cls_n);  // (256 at most)
  unsigned long long mine = 0, w = 0;
  if (tid < m) {
    mine = sm.cls[tid];
    w = wt.weight44(order_float(static_cast<uint32_t>(mine)));
    sm.cls[kThreads + tid] = w;
  }
  __syncthreads();
  if (tid < m) {
#pragma unroll 4
    for (int j = 0; j < m; ++j) before += sm.cls[j] > mine ? sm.cls[kThreads + j] : 0ull;  // (lower indices)
    if (before <= t && before + w > t) {
      p.token[row] = (1 << kIdxBits) - 1 - static_cast<int>(mine >> 32);
      p.prob[row] = share_of(w, Z);
    }
  }
  return true;
}

// How long a request's rows take, roughly: 2 all weights exactly, 1 all
// weights, 0 the candidates'.  Only the rows' order depends on it.  (Whether
// top-p is decided by the candidates depends on the logits' spread over T, which
// is not known here: 0.9 stands for the spread that language models' logits
// have, where at T = 0.7 a few percent and at T = 1 most rows take whole-row
// passes.)
__device__ __forceinline__ int request_cost(const SampleParams& p, int req) {
  const float T = p.temperature ? p.temperature[req] : 1.f, tp = p.top_p ? p.top_p[req] : 1.f;
  const int k = p.top_k ? p.top_k[req] : 0;
  if (!(T > 0.f) || (k >= 1 && k < p.V)) return 0;
  if (p.min_p && p.min_p[req] > 0.f) return 0;
  return tp < 1.f && T < 0.9f ? 1 : 2;
}

template <typename E>
__global__ void __launch_bounds__(kThreads, 4) k_sample(const SampleParams p) {
  constexpr int kPer = Row<E>::kPer;
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  pdl_wait();
  pdl_trigger();
  unsigned cl_u, rank_u;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl_u));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_u));
  const int cl = static_cast<int>(cl_u), rank = static_cast<int>(rank_u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // requests that need their whole rows' weights first: their rows take several
  // times as long as the others', which then fill the SMs (2064 rows of 151936
  // in 16 requests of all kinds: an eighth to a third less time than in the rows'
  // order)
  int row = blockIdx.x / cl;
  const int requests = p.rows / p.rows_per_req;
  if (requests > 1 && requests <= kBins && requests * p.rows_per_req == p.rows) {
    for (int a = tid; a < requests; a += kThreads) sm.count[a] = request_cost(p, a);
    __syncthreads();
    if (warp == 0) {
      auto with = [&](int b, unsigned cost) {
        return __ballot_sync(kFullMask, b + lane < requests && sm.count[b + lane] == cost);
      };
      int place = row / p.rows_per_req;
      for (int cost = 2; cost >= 0; --cost) {
        for (int b = 0; b < requests; b += 32) {
          const unsigned in = with(b, cost);
          if (place >= 0 && place < __popc(in) && (in >> lane & 1) && __popc(in & ((1u << lane) - 1)) == place)
            sm.picked = b + lane;
          place -= __popc(in);
        }
      }
    }
    __syncthreads();
    row = sm.picked * p.rows_per_req + row % p.rows_per_req;
  }
  const int req = row / p.rows_per_req;
  const E* src = static_cast<const E*>(p.logits) + static_cast<size_t>(row) * p.row_stride;
  const bool lead = rank == 0;
  Smem& ls = *at_rank(&sm, 0);  // the leader's
  const Row<E> rw(src, p.V);
  const int gw = rank * kWarps + warp, gn = cl * kWarps;
  const int share = (rw.units + gn - 1) / gn;
  const int ub = min(rw.units, gw * share), ue = min(rw.units, ub + share);

  const float T = p.temperature ? p.temperature[req] : 1.f;
  Rule rule;
  rule.k = p.top_k ? p.top_k[req] : 0;
  rule.tp = p.top_p ? p.top_p[req] : 1.f;
  rule.mp = p.min_p && p.min_p[req] > 0.f ? fminf(p.min_p[req], 1.f) : 0.f;
  rule.use_k = rule.k >= 1 && rule.k < p.V;
  rule.use_p = rule.tp < 1.f;
  const bool greedy = !(T > 0.f);
  // log2(e) / T as a sum of two floats (fp64 divisions take a microsecond)
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-8f;
  const float ch = __fdiv_rn(kLog2e, T);
  const float ch_lo = isfinite(ch) && isfinite(T) ? __fdiv_rn(fmaf(-ch, T, kLog2e) + kLog2eLo, T) : 0.f;

  // (with no cut every token is in the draw, and the row's sums are needed)
  bool listed = greedy || rule.use_k || rule.use_p || rule.mp > 0.f;
  float bound = -INFINITY, bound2 = -INFINITY, off = 0.f;
  // (the table is waited for in front of the list)
  for (int i = tid; i < (1 << kExpBits) / 2; i += kThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sm.exp[2 * i])), "l"(g_exp.v + 4 * i)
                 : "memory");
  if (tid == 0) {
    sm.list_n = 0;
    sm.units_n = 0;
    sm.cls_n = 0;
    sm.ctl.done = 0;
  }
  // (waited for before the first access to another CTA's memory)
  if (cl > 1) cluster_arrive();
  if (listed) {
    // ---- 1. a sample: every thread one unit, evenly spread over the row (the
    // same in all of a cluster's CTAs: exchanging bounds of several samples
    // costs more than their better bound gives).  The bound is the r-th largest
    // of the units' maxima, with r / 256 the share of units that hold one of
    // the candidates wanted: 256 (1 - (1 - want / V)^kPer).  The order is that
    // of the maxima's upper 24 bits: any bound near it does.
    float m = -INFINITY;
    if (rw.units > 0) {
      float x[kPer];
      unpack<E>(rw.load(static_cast<int>(static_cast<long long>(tid) * rw.units / kThreads)), x);
      m = fmaxf(max_of(x), -INFINITY);
    }
    const unsigned mine = (float_order(m) & ~255u) | tid;
    sm.sample[tid] = mine;
    __syncthreads();
    const float want = rule.use_k ? fminf(fmaxf(2.f * rule.k, 0.5f * kWant), 1.2f * kWant) : kWant;
    const float share_out = fminf(want / static_cast<float>(p.V), 1.f);
    const int r = max(1, static_cast<int>(kThreads * (1.f - __powf(1.f - share_out, kPer)) + 0.5f));
    const int r2 = rule.use_k ? (2 * r + 2) / 3 : (r + 1) / 2;  // (should the list overflow)
    int above = 0;
    for (int q = 0; q < kThreads; q += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(&sm.sample[q]);
      above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    if (above == 0) sm.smax = m;
    if (above == r - 1) sm.sbound = m;
    if (above == r2 - 1) sm.sbound2 = m;
    __syncthreads();
    const float hi = sm.smax;
    bound = greedy ? hi : sm.sbound;
    bound2 = greedy ? hi : sm.sbound2;
    off = hi * ch;  // the reference of the sums
    if (!isfinite(off)) off = 0.f;
  } else {
    __syncthreads();
  }

  // ---- 2. one pass: units that reach the bound are noted; the weights of
  // the other tokens, 2^(x ch - off) <= 1, are summed where top-p needs them.
  // NaN makes the sum NaN, which sends the row to the whole-row path.
  float top = -INFINITY, sum = 0.f;
  const bool sums = rule.use_p && !rule.use_k && !greedy;
  auto pass = [&](auto mode) {
    constexpr int kMode = decltype(mode)::value;  // 0: largest logit, 1: and candidates, 2: and sums
    constexpr int kAhead = 4;
    auto take = [&](uint4 v, int u) {
      float x[kPer];
      unpack<E>(v, x);
      const float m = max_of(x);
      if constexpr (kMode == 0) {
        top = fmaxf(top, m);
        return 0.f;
      }
      if (m >= bound && m > -INFINITY) {
        top = fmaxf(top, m);
        const unsigned at = atomicAdd(&sm.units_n, 1u);
        if (at < kUnits) sm.unit[at] = static_cast<uint16_t>(u);
        return 0.f;
      }
      float w = 0.f;
      if constexpr (kMode == 2) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) w += ex2(fmaf(x[k], ch, -off));
      }
      return w;
    };
    int u = ub + lane;
    uint4 v[kAhead];
    auto full = [&](int at) { return at + 32 * (kAhead - 1) < ue; };
    if (full(u)) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) v[a] = rw.load(u + 32 * a);
    }
    for (; full(u); u += 32 * kAhead) {
      float w = 0.f;
      const bool more = full(u + 32 * kAhead);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const uint4 now = v[a];
        if (more) v[a] = rw.load(u + 32 * (kAhead + a));
        w += take(now, u + 32 * a);
      }
      sum += w;
    }
    for (; u < ue; u += 32) sum += take(rw.load(u), u);
  };
  if (!listed) pass(IntC<0>{});
  else if (!sums) pass(IntC<1>{});
  else pass(IntC<2>{});
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (cl > 1) cluster_wait();
  __syncthreads();
  // one token: to the leader's list, or into the sum
  auto token = [&](float x, int i) {
    if (!(x > -INFINITY)) return;  // (NaN, -inf)
    top = fmaxf(top, x);
    if (!listed) return;
    if (x >= bound) {
      const unsigned at = atomicAdd(&ls.list_n, 1u);
      if (at < kList) ls.list[at] = key50(x, i);
    } else {
      sum += ex2(fmaf(x, ch, -off));
    }
  };
  const float rest_sum = sum;
  for (;;) {
    if (listed) {
      const int n = min(static_cast<int>(sm.units_n), kUnits);
      for (int b = warp * 32; b < n; b += kThreads) {
        const int un = b + lane < n ? sm.unit[b + lane] : -1;
        unsigned in = 0;
        float x[kPer];
        if (un >= 0) {
          unpack<E>(rw.load(un), x);
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            if (!(x[k] > -INFINITY)) continue;  // (NaN, -inf)
            top = fmaxf(top, x[k]);
            if (x[k] >= bound) in |= 1u << k;
            else sum += ex2(fmaf(x[k], ch, -off));
          }
        }
        // the warp's candidates take their places by one addition
        int at = __popc(in);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFullMask, at, o);
          if (lane >= o) at += y;
        }
        unsigned base = 0;
        if (lane == 31) base = atomicAdd(&ls.list_n, static_cast<unsigned>(at));
        at += static_cast<int>(__shfl_sync(kFullMask, base, 31)) - __popc(in);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          if (!(in >> k & 1)) continue;
          if (at < kList) ls.list[at] = key50(x[k], rw.index(un) + k);
          ++at;
        }
      }
    }
    if (lead) {
      const int rest = rw.index(rw.units);
      if (tid < rw.head) token(logit<E>(src, tid), tid);
      if (tid < p.V - rest) token(logit<E>(src, rest + tid), rest + tid);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
      sum += __shfl_xor_sync(kFullMask, sum, o);
    }
    if (lane == 0) {
      sm.wmax[warp] = top;
      sm.wval[warp] = sum;
    }
    __syncthreads();
    if (tid == 0) {
      float t = sm.wmax[0], w = sm.wval[0];
      for (int k = 1; k < kWarps; ++k) {
        t = fmaxf(t, sm.wmax[k]);
        w += sm.wval[k];
      }
      ls.part[rank] = Part{t, w, off, sm.units_n > kUnits ? 1 : 0};
    }
    if (cl > 1) cluster_sync();
    else __syncthreads();
    // too many candidates: once more among the noted units, with the higher bound
    if (!(ls.list_n > kList && bound2 > bound)) break;
    if (cl > 1) cluster_sync();
    else __syncthreads();
    bound = bound2;
    sum = rest_sum;
    if (tid == 0) sm.list_n = 0;
    if (cl > 1) cluster_sync();
    else __syncthreads();
  }

  // ---- 3. the leader decides the row by the list, or the cluster by the row
  Weights wt;
  wt.exp = sm.exp;
  wt.ch = ch;
  wt.cl = ch_lo;
  if (lead) {
    float all = 0.f;
    bool lost = false;
    top = -INFINITY;
    for (int q = 0; q < cl; ++q) {
      top = fmaxf(top, sm.part[q].top);
      all += sm.part[q].sum;
      lost |= sm.part[q].lost != 0;
    }
    wt.top = top;
    const int n = static_cast<int>(sm.list_n);
    bool done = false;
    if (top == -INFINITY) {
      if (tid == 0) {
        p.token[row] = -1;
        p.prob[row] = 0.f;
      }
      done = true;
    } else if (greedy) {
      if (!lost && n <= kList) {
        unsigned long long best = 0;
        for (int i = tid; i < n; i += kThreads) best = max(best, sm.list[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
        if (lane == 0) sm.scan_m[warp] = best;
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kWarps; ++w) best = max(best, sm.scan_m[w]);
          p.token[row] = (1 << kIdxBits) - 1 - static_cast<int>(best & ((1u << kIdxBits) - 1));
          p.prob[row] = 1.f;
        }
        done = true;
      }
    } else if (listed && !lost && n <= kList && isfinite(top) && isfinite(all) && isfinite(top * ch)) {
      // the sums, relative to the largest logit: 2^(off - top ch) of what
      // they are, off by (|x ch - off| <= 46 where a weight counts, and so
      // is |off - top ch|) 2^-19 for each argument's rounding, 2^-19 for
      // ch's, 2^-21 for two ex2 and 2^-17 for some 100 additions: below
      // 2^-16; the weights' own rounding to whole units is half a unit per
      // token
      const unsigned long long tail =
          static_cast<unsigned long long>(all * ex2(fmaf(-top, ch, off)) * 17592186044416.f);
      done = from_list<E>(p, sm, row, n, static_cast<unsigned long long>(float_order(bound)) << kIdxBits, tail,
                          (tail >> 16) + static_cast<unsigned long long>(p.V), wt, rule);
    }
    if (tid == 0) {
      sm.ctl.done = done ? 1 : 0;
      sm.ctl.top = top;
      sm.cls_n = 0;
    }
  }
  if (cl > 1) cluster_sync();
  else __syncthreads();
  if (!ls.ctl.done) {
    wt.top = ls.ctl.top;
    whole_row<E>(p, sm, ls, src, row, cl, rank, wt, rule, greedy);
  }
  if (cl > 1) cluster_sync();  // (no CTA leaves while another reads the leader's memory)
}

}  // namespace
}  // namespace dt

extern "C" dartree_status dartree_sample(const void* logits, int32_t bf16, int64_t row_stride, int32_t V,
                                         int32_t rows, int32_t rows_per_req, const float* temperature,
                                         const int32_t* top_k, const float* top_p, const float* min_p,
                                         const float* u, int32_t* token, float* prob, void* stream) {
  using namespace dt;
  if (!logits || !u || !token || !prob) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (V < 1 || rows < 1 || rows_per_req < 1 || row_stride < V)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "bad V, rows, rows_per_req or row_stride");
  if (V > (1 << kIdxBits)) return cache_fail(DARTREE_ERR_UNSUPPORTED, "V must be at most 2^18");
  const SampleParams p{logits, row_stride, V, rows, rows_per_req, temperature, top_k, top_p, min_p, u, token, prob};
  // one cluster per row: as many CTAs as the SMs hold (four each)
  int cl = 1;
  while (cl < kMaxCl && static_cast<long long>(rows) * cl * 2 <= 608 && V / cl > 4096) cl *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (static_cast<long long>(rows) * cl > 0x7FFFFFFFll) return cache_fail(DARTREE_ERR_UNSUPPORTED, "too many rows");
  const dim3 grid(static_cast<unsigned>(rows) * cl);
  static std::atomic<uint64_t> done_bf16{0}, done_f32{0};
  cudaError_t e = bf16 ? opt_in_smem(k_sample<uint16_t>, &done_bf16) : opt_in_smem(k_sample<float>, &done_f32);
  if (e == cudaSuccess)
    e = launch_kernel_cluster(bf16 ? k_sample<uint16_t> : k_sample<float>, grid, dim3(kThreads), sizeof(Smem), st,
                              true, cl, p);
  return cache_launched(e);
}
