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
#include "row_cuts.cuh"

namespace dt {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kMassUnit = 16000.f; // 2^18 2^(1/40) units fit 32 bits
constexpr int kList = 2944;          // candidates
constexpr float kWant = 1800.f;      // candidates aimed at
constexpr int kUnits = 4096;         // 16-byte units of a CTA that may hold candidates
constexpr int kMaxCl = 8;

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

struct Part {            // a CTA's share of the pass, for the leader
  float top, sum, off;
  int lost;              // more units than kUnits
};

struct Smem {
  static constexpr int kThreads = kWarps * 32;
  static constexpr bool kWideSums = false;
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

template <bool LIST, typename E>
using Source = RowSource<LIST, E, Smem>;

// w / z to fp32, for w <= z: both as sums of two floats (49 bits or more), the
// quotient of the upper ones corrected once.  (An fp64 division: 0.7 us.)
__device__ __forceinline__ float share_of(unsigned long long w, unsigned long long z) {
  const float wh = __ull2float_rn(w), zh = __ull2float_rn(z);
  const float wl = __ll2float_rn(static_cast<long long>(w - __float2ull_rn(wh)));
  const float zl = __ll2float_rn(static_cast<long long>(z - __float2ull_rn(zh)));
  const float q = __fdiv_rn(wh, zh);
  return q + __fdiv_rn(fmaf(-q, zh, wh) + fmaf(-q, zl, wl), zh);
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

// floor(u total) for the draw, below total.
__device__ __forceinline__ unsigned long long draw_mark(float u, unsigned long long total) {
  unsigned long long t = 0;
  if (u > 0.f)
    t = u >= 1.f ? total : __umul64hi(fraction64(u), total);
  return t < total ? t : total - 1;
}

// The row's classes: counts and masses of what is above `keep`.
template <typename S, typename W>
__device__ void fill_bins(const S& s, const W& wt, unsigned long long keep) {
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
  const Codes code(wt.top);
  if (!code.sound()) return false;
  if (!code_cut(s, wt, rule, code)) return false;
  const float v = ctl.bin >= 0 ? code.value(ctl.bin) : -INFINITY;
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
