// A row of logits as whole numbers: its weights in units of 2^-44, the order of
// its tokens as keys, and the cuts (top-k, min-p, top-p) of a row that a
// thread-block cluster works on.
//
// The functions take the including kernel's shared memory as Mem: the classes
// (mass_lo, mass_hi, count [kBins]), a class's members (cls [kClass], cls_n), the
// codes' counts (codes [2 kTable]), a list, the scans (scan_m, scan_c [warps]),
// picked, picked_n, picked_c, picked_m, ctl, kThreads, the block's threads, and
// kWideSums, whether sums over the cluster's CTAs take all their loads together.
#pragma once
#include <cuda_bf16.h>

#include "block.cuh"
#include "cache.cuh"
#include "ptx.cuh"

namespace dt {

constexpr int kBins = 1024;
constexpr float kBinsPer2 = 20.f;    // classes per power of two
constexpr int kClass = 1024;         // members of a class that are sorted
constexpr int kRanked = 128;         // members of a class that are ranked by comparisons
constexpr int kIdxBits = 18;
constexpr float kZeroBelow = -46.f;  // 2^-46 rounds to 0 in units of 2^-44
constexpr int kExpBits = 10;
constexpr int kTable = 768;          // bf16 logits of a sign whose weights are tabled

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

// weight44 as a call, where it is rare or not what takes the time (its code is some
// 70 instructions, and kernels that have it in a dozen places take minutes to
// compile).
static __device__ __noinline__ unsigned long long weight44_call(float x, float top, float ch, float cl,
                                                                const float2* exp) {
  return Weights{top, ch, cl, exp}.weight44(x);
}
struct CalledWeights : Weights {
  __device__ __forceinline__ explicit CalledWeights(const Weights& w) : Weights(w) {}
  __device__ __forceinline__ unsigned long long weight44(float x) const { return weight44_call(x, top, ch, cl, exp); }
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
template <typename Mem>
__device__ __forceinline__ void block_scan(Mem& sm, unsigned& c, unsigned long long& m) {
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
template <bool LIST, typename E, typename Mem_>
struct RowSource {
  using Mem = Mem_;
  Mem& sm;
  Mem& ls;
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
      for (int i = threadIdx.x; i < n; i += Mem::kThreads) {
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
    // (all CTAs' loads together, where the kernel has the registers: one after the
    // other 8 CTAs' take 3 us)
    constexpr int kAhead = !LIST && Mem::kWideSums ? 8 : 1;
    for (int q0 = 0; q0 < (LIST ? 1 : cl); q0 += kAhead) {
#pragma unroll
      for (int q = q0; q < q0 + kAhead; ++q) {
        if (q >= (LIST ? 1 : cl)) continue;
        const Mem* o = LIST ? &sm : at_rank(&sm, q);
        *c += o->count[b];
        *m += (static_cast<unsigned long long>(o->mass_hi[b]) << 32) + o->mass_lo[b];
      }
    }
  }
};

// A 64-bit sum in shared memory from two 32-bit atomics (shared memory has
// no 64-bit add): the low word's add that wraps carries.
template <typename Mem>
__device__ __forceinline__ void add_mass(Mem& sm, int b, unsigned long long w) {
  const unsigned lo = static_cast<unsigned>(w);
  const unsigned old = atomicAdd(&sm.mass_lo[b], lo);
  const unsigned hi = static_cast<unsigned>(w >> 32) + (old + lo < old ? 1u : 0u);
  if (hi) atomicAdd(&sm.mass_hi[b], hi);
}

template <typename Mem>
__device__ __forceinline__ void clear_classes(Mem& sm) {
  for (int i = threadIdx.x; i < kBins; i += Mem::kThreads) {
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
  constexpr int kThreads = S::Mem::kThreads, kPer = kBins / kThreads;
  auto& sm = s.sm;
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
template <typename S, typename W>
__device__ bool cut(const S& s, const W& wt, bool by_count, unsigned long long target,
                    unsigned long long& keep, unsigned long long* upto) {
  constexpr int kThreads = S::Mem::kThreads;
  auto& sm = s.sm;
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
template <typename W>
__device__ unsigned long long min_p_key(const W& wt, float mp) {
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

// Count and mass over all classes (leader's block).
template <typename S>
__device__ void all_classes(const S& s, unsigned* count, unsigned long long* mass) {
  constexpr int kThreads = S::Mem::kThreads, kPer = kBins / kThreads;
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
  template <typename W>
  __device__ __forceinline__ unsigned long long weight(const W& wt, int j) const {
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

// top-k and top-p of a bf16 row by counts of its codes: they and the codes'
// weights give the running counts and masses exactly, so a cut falls on a code
// and a number of its ties, the first in index order.  Left for the cluster: the
// code's place ctl.bin (-1: nothing is cut), its ties that are kept ctl.left, all
// of them ctl.last, and the kept mass ctl.total.  False where a cut falls on a
// logit without a place.  The leader's list is used (4 numbers per warp).
// kLeast: tokens below `least` are out (min-p's).
template <bool kLeast = false, typename S, typename W>
__device__ __forceinline__ bool code_cut(const S& s, const W& wt, const Rule& rule, const Codes& code,
                                         float least = -INFINITY) {
  auto& sm = s.sm;
  Ctl& ctl = s.ls.ctl;
  constexpr int kThreads = S::Mem::kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warps = s.cl * (kThreads / 32);
  constexpr int kN = 2 * kTable + 2, kPer = (kN + kThreads - 1) / kThreads;
  for (int j = tid; j < 2 * kTable; j += kThreads) sm.codes[j] = 0;
  __syncthreads();
  unsigned between = 0, below = 0;
  unsigned long long between_m = 0, below_m = 0;
  auto other = [&](float x, int) {
    const unsigned long long w = wt.weight44(x);
    const bool low = code.below(x);
    between += !low;
    below += low;
    between_m += low ? 0ull : w;
    below_m += low ? w : 0ull;
  };
  each_code(s, code,
            [&](float x, int, int j) {
              if (!kLeast || x >= least) atomicAdd(&sm.codes[j], 1u);
            },
            [&](float x, int i) {
              if (!kLeast || x >= least) other(x, i);
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
    // (what lies between and below: warp v adds up the warps' v-th number)
    if constexpr (S::Mem::kWideSums) {
      const int v = tid >> 5;
      if (v < 4) {
        unsigned long long x = 0;
        for (int w = lane; w < warps; w += 32) x += sm.list[4 * w + v];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFullMask, x, o);
        if (lane == 0) sm.list[4 * warps + v] = x;
      }
    }
    constexpr int kAhead = S::Mem::kWideSums ? 8 : 1;
    for (int r0 = 0; r0 < s.cl; r0 += kAhead) {
#pragma unroll
      for (int r = r0; r < r0 + kAhead; ++r) {
        if (r >= s.cl) continue;
        const unsigned* from = at_rank(&sm, r)->codes;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int e = tid * kPer + q;
          if (e < kN - 1 && e != kTable) cs[q] += from[e < kTable ? e : e - 1];
        }
      }
    }
    if constexpr (S::Mem::kWideSums) __syncthreads();
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int e = tid * kPer + q;
      ms[q] = 0;
      if (e == kTable || e == kN - 1) {
        const int v = e == kN - 1 ? 2 : 0;
        if constexpr (S::Mem::kWideSums) {
          cs[q] = static_cast<unsigned>(sm.list[4 * warps + v]);
          ms[q] = sm.list[4 * warps + v + 1];
        } else {
#pragma unroll 8
          for (int w = 0; w < warps; ++w) {
            cs[q] += static_cast<unsigned>(sm.list[4 * w + v]);
            ms[q] += sm.list[4 * w + v + 1];
          }
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
          sm.picked_c = cs[q];
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
      ctl.last = static_cast<int>(sm.picked_c);
      ctl.total = Z;
      ctl.refine = ok ? 0 : 1;
    }
  }
  s.sync();
  return ctl.refine == 0;
}

}  // namespace dt
