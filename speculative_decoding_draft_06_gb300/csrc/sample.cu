// Tokens drawn from rows of logits (dartree_sample).
//
// A row is the work of one thread-block cluster: CTA k, warp w reads the
// (16 k + w)-th contiguous share of the vocabulary.  Every cut (top-k,
// min-p, top-p) keeps a prefix of the order (logit desc, index asc), so the
// kept tokens are those whose 50-bit key (ordered logit, inverted index) is
// at least one threshold.
//
// The weights w = 2^((l - max) log2(e) / T) are integers in units of 2^-44
// (weight44): sums of them are exact whatever their order, so the shared
// histograms may be filled by atomics, and "mass >= top_p Z" and "running
// sum > u Z" are decided on whole numbers.  32-bit sums would not do: a row
// of 150 000 tokens has as many borders, and a running sum that is off by
// 2^-20 of the total moves the draw over one of them every few rows.
//
// 1. the largest key (max, arg max);
// 2. with top-k or top-p: a histogram of counts and masses over 1536 bins of
//    -log2 w (1/32 each, monotone in the logit); the bin in which the cut
//    falls is gathered (refined by digits of the key while it holds more
//    than kList), sorted, and the cut element found in it;
// 3. the kept tokens' sums per warp, the warp in which u Z falls, and in
//    that warp the token.
#include <cuda_bf16.h>

#include "block.cuh"
#include "cache.cuh"

namespace dt {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 1536;        // 48 powers of two, 32 bins each
constexpr float kBinsPer2 = 32.f;
constexpr int kList = 2048;
constexpr int kMaxCl = 8;
constexpr int kIdxBits = 18;
constexpr float kZeroBelow = -46.f;  // 2^-46 rounds to 0 in units of 2^-44
constexpr int kExpBits = 10;

// 2^(j / 1024) as the sum of two floats.
struct ExpTable {
  float hi[1 << kExpBits], lo[1 << kExpBits];
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
    t.hi[j] = static_cast<float>(x);
    t.lo[j] = static_cast<float>(x - static_cast<double>(t.hi[j]));
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
  int bin;
  int refine;            // 1: another digit, 0: gather
  int warp;              // draw: the warp (of the cluster)
};

struct Smem {
  float2 exp[1 << kExpBits];
  unsigned long long mass[kBins];
  unsigned count[kBins];
  unsigned long long list[kList];
  unsigned long long wsum[kMaxCl * kWarps];
  unsigned long long best[kMaxCl];
  unsigned long long scan_m[kWarps];
  unsigned scan_c[kWarps];
  unsigned list_n;
  Ctl ctl;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same object in CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T* at_rank(T* p, int rank) {
  uint64_t out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(out);
}

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
    const float n = rintf(p * 1024.f);    // p = (n + f) / 1024, |f| <= 1/2, exact
    const float t = fmaf(n, -1.f / 1024.f, p);
    const int ni = static_cast<int>(n);
    const float2 T = exp[ni & 1023];
    const int sh = 44 + (ni >> 10);       // the integer part, up to the table's
    constexpr float kL1 = 0.693147182464599609375f;  // ln 2 = kL1 + kL1lo
    constexpr float kL1lo = -1.904654299957768e-9f;
    const float a = t * kL1;
    float b = fmaf(t, kL1, -a);
    b = fmaf(t, kL1lo, b);
    b = fmaf(e * kL1, fmaf(t, kL1, 1.f), b);  // 2^(t+e) - 2^t
    b = fmaf(t * t, fmaf(t, 0.05550410866f, 0.24022650696f), b);  // 2^t - 1 = a + b
    const float m = T.x * a;
    float lo = fmaf(T.x, a, -m);
    lo = fmaf(T.x, b, lo);
    lo = fmaf(T.y, a, lo);
    lo += T.y;                            // T (1 + a + b) = T.x + m + lo
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);  // 2^sh, sh >= -2
    const long long w = __float2ll_rn(T.x * up) + __float2ll_rn(m * up) + __float2ll_rn(lo * up);
    return w > 0 ? static_cast<unsigned long long>(w) : 0ull;
  }
};

__device__ __forceinline__ unsigned long long key50(float x, int idx) {
  return (static_cast<unsigned long long>(float_order(x)) << kIdxBits) |
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

// ceil(p z) for p in (0, 1) (fp32) and z < 2^63, at least 1.
__device__ __forceinline__ unsigned long long ceil_share(float p, unsigned long long z) {
  const unsigned long long f = static_cast<unsigned long long>(ldexp(static_cast<double>(p), 63));
  const unsigned long long hi = __umul64hi(f, z), lo = f * z;
  const unsigned long long q = (hi << 1) | (lo >> 63);
  const unsigned long long c = q + ((lo << 1) != 0ull ? 1ull : 0ull);
  return c > 0ull ? c : 1ull;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  unsigned cl_u, rank_u;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl_u));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_u));
  const int cl = static_cast<int>(cl_u), rank = static_cast<int>(rank_u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / cl, req = row / p.rows_per_req;
  const E* src = static_cast<const E*>(p.logits) + static_cast<size_t>(row) * p.row_stride;
  const bool lead = rank == 0;
  Smem& ls = *at_rank(&sm, 0);  // the leader's

  const int share = (p.V + cl * kWarps - 1) / (cl * kWarps);
  const int begin = min(p.V, (rank * kWarps + warp) * share), end = min(p.V, begin + share);

  // ---- 1. the largest key
  unsigned long long best = 0;
  for (int i = begin + lane; i < end; i += 32) {
    const unsigned long long k = key50(logit<E>(src, i), i);
    best = k > best ? k : best;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long y = __shfl_xor_sync(kFullMask, best, o);
    best = y > best ? y : best;
  }
  if (lane == 0) sm.scan_m[warp] = best;
  for (int i = tid; i < (1 << kExpBits); i += kThreads) sm.exp[i] = make_float2(g_exp.hi[i], g_exp.lo[i]);
  for (int i = tid; i < kBins; i += kThreads) {
    sm.mass[i] = 0;
    sm.count[i] = 0;
  }
  if (tid == 0) sm.list_n = 0;
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? sm.scan_m[lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long y = __shfl_xor_sync(kFullMask, best, o);
      best = y > best ? y : best;
    }
    if (lane < cl) at_rank(&sm, lane)->best[rank] = best;
  }
  cluster_sync();
  best = sm.best[0];
  for (int k = 1; k < cl; ++k) best = sm.best[k] > best ? sm.best[k] : best;
  const float top = key50_value(best);
  const float T = p.temperature ? p.temperature[req] : 1.f;
  const bool greedy = !(T > 0.f);
  if (top == -INFINITY || greedy) {  // (the same in the whole cluster)
    if (lead && tid == 0) {
      const bool none = top == -INFINITY;
      p.token[row] = none ? -1 : (1 << kIdxBits) - 1 - static_cast<int>(best & ((1u << kIdxBits) - 1));
      p.prob[row] = none ? 0.f : 1.f;
    }
    return;  // (no CTA reads another's memory after the barrier above)
  }
  const double c2 = 1.4426950408889634074 / static_cast<double>(T);
  Weights wt;
  wt.top = top;
  wt.ch = static_cast<float>(c2);
  wt.cl = isinf(wt.ch) ? 0.f : static_cast<float>(c2 - static_cast<double>(wt.ch));
  wt.exp = sm.exp;
  const int k = p.top_k ? p.top_k[req] : 0;
  const float tp = p.top_p ? p.top_p[req] : 1.f;
  const float mp = p.min_p ? fminf(p.min_p[req], 1.f) : 0.f;
  const bool use_k = k >= 1 && k < p.V, use_p = tp < 1.f;
  unsigned long long keep = 0;  // threshold key so far

  // ---- 2. the cuts
  if (mp > 0.f) {
    // the smallest ordered logit whose weight is at least min_p: 32 probes a
    // round (every warp finds the same)
    const unsigned long long need = static_cast<unsigned long long>(ceil(ldexp(static_cast<double>(mp), 44)));
    unsigned lo = 0, hi = float_order(top);  // the answer lies in (lo, hi]
    while (hi - lo > 1) {
      const unsigned step = (hi - lo + 31) / 32;
      const unsigned long long at = static_cast<unsigned long long>(lo) + static_cast<unsigned long long>(lane + 1) * step;
      const bool in = at >= hi || wt.weight44(order_float(static_cast<unsigned>(at))) >= need;
      const int f = __ffs(__ballot_sync(kFullMask, in)) - 1;  // (the last probe is at or behind hi)
      const unsigned long long nhi = static_cast<unsigned long long>(lo) + static_cast<unsigned long long>(f + 1) * step;
      lo += static_cast<unsigned>(f) * step;
      hi = nhi < hi ? static_cast<unsigned>(nhi) : hi;
    }
    keep = static_cast<unsigned long long>(hi) << kIdxBits;
  }
  if (use_k || use_p) {
    auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>(wt.log2w(x) * -kBinsPer2)); };
    for (int i = begin + lane; i < end; i += 32) {
      const float x = logit<E>(src, i);
      if (key50(x, i) < keep) continue;
      const unsigned long long w = wt.weight44(x);
      if (w == 0) continue;
      const int b = bin_of(x);
      atomicAdd(&sm.count[b], 1u);
      atomicAdd(&sm.mass[b], w);
    }
    cluster_sync();
    // the leader keeps the bins' sums of the whole row
    constexpr int kPer = kBins / kThreads;
    unsigned row_c[kPer];
    unsigned long long row_m[kPer];
    if (lead) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        row_c[j] = 0;
        row_m[j] = 0;
        for (int q = 0; q < cl; ++q) {
          const Smem* o = at_rank(&sm, q);
          row_c[j] += o->count[tid * kPer + j];
          row_m[j] += o->mass[tid * kPer + j];
        }
      }
    }
    unsigned long long Z = 0;  // mass of what is kept so far (leader)
    // find the element at which the running count (by_count) or mass reaches
    // `target`; what lies before it counts.  All CTAs call it together; on
    // return sm.ctl.keep of the leader is its key, and in the leader `got`
    // the mass up to and with it.
    auto cut = [&](bool by_count, unsigned long long target, unsigned long long* got) {
      unsigned c_before = 0;
      unsigned long long m_before = 0;
      // the class that holds the element among n_cls = kPer * kThreads (or
      // 1024) classes whose sums the leader's threads hold
      auto pick = [&](int per, const unsigned* cs, const unsigned long long* ms, int shift) {
        unsigned c = 0;
        unsigned long long m = 0;
        for (int j = 0; j < per; ++j) {
          c += cs[j];
          m += ms[j];
        }
        const unsigned c0 = c;
        const unsigned long long m0 = m;
        block_scan(sm, c, m);
        unsigned bc = c_before + c - c0;
        unsigned long long bm = m_before + m - m0;
        for (int j = 0; j < per; ++j) {
          const bool here = by_count ? (bc < target && target <= bc + cs[j]) : (bm < target && target <= bm + ms[j]);
          if (here) {
            if (shift < 0) {
              sm.ctl.bin = tid * per + j;
              sm.ctl.prefix = sm.ctl.mask = 0;
            } else {  // digits run from the largest
              sm.ctl.prefix |= static_cast<unsigned long long>(1023 - (tid * per + j)) << shift;
              sm.ctl.mask |= 1023ull << shift;
            }
            sm.ctl.refine = cs[j] > kList;
            sm.scan_c[0] = bc;
            sm.scan_m[0] = bm;
          }
          bc += cs[j];
          bm += ms[j];
        }
        __syncthreads();
        c_before = sm.scan_c[0];
        m_before = sm.scan_m[0];
        __syncthreads();
      };
      if (lead) pick(kPer, row_c, row_m, -1);
      cluster_sync();
      for (int shift = 40; ls.ctl.refine; shift -= 10) {
        for (int i = tid; i < 1024; i += kThreads) {
          sm.mass[i] = 0;
          sm.count[i] = 0;
        }
        const int bin = ls.ctl.bin;
        const unsigned long long pre = ls.ctl.prefix, msk = ls.ctl.mask;
        __syncthreads();
        for (int i = begin + lane; i < end; i += 32) {
          const float x = logit<E>(src, i);
          const unsigned long long key = key50(x, i);
          if (key < keep || (key & msk) != pre) continue;
          const unsigned long long w = wt.weight44(x);
          if (w == 0 || bin_of(x) != bin) continue;
          const int d = 1023 - static_cast<int>((key >> shift) & 1023);
          atomicAdd(&sm.count[d], 1u);
          atomicAdd(&sm.mass[d], w);
        }
        cluster_sync();
        if (lead) {
          unsigned cs[2];
          unsigned long long ms[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            cs[j] = 0;
            ms[j] = 0;
            for (int q = 0; q < cl; ++q) {
              const Smem* o = at_rank(&sm, q);
              cs[j] += o->count[tid * 2 + j];
              ms[j] += o->mass[tid * 2 + j];
            }
          }
          pick(2, cs, ms, shift);
        }
        cluster_sync();
      }
      // the class's members to the leader
      {
        const int bin = ls.ctl.bin;
        const unsigned long long pre = ls.ctl.prefix, msk = ls.ctl.mask;
        for (int i = begin + lane; i < end; i += 32) {
          const float x = logit<E>(src, i);
          const unsigned long long key = key50(x, i);
          if (key < keep || (key & msk) != pre || bin_of(x) != bin || wt.weight44(x) == 0) continue;
          const unsigned at = atomicAdd(&ls.list_n, 1u);
          if (at < kList) ls.list[at] = key;
        }
      }
      cluster_sync();
      if (lead) {
        const int n = min(static_cast<int>(sm.list_n), kList);
        const int n2 = pow2_at_least(n);
        for (int i = n + tid; i < n2; i += kThreads) sm.list[i] = 0;
        __syncthreads();
        block_sort_desc(reinterpret_cast<uint64_t*>(sm.list), n2);
        constexpr int kQ = kList / kThreads;
        unsigned cs[kQ];
        unsigned long long ms[kQ];
        unsigned c = 0;
        unsigned long long m = 0;
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
          const int i = tid * kQ + j;
          cs[j] = i < n ? 1u : 0u;
          ms[j] = i < n ? wt.weight44(key50_value(sm.list[i])) : 0ull;
          c += cs[j];
          m += ms[j];
        }
        const unsigned c0 = c;
        const unsigned long long m0 = m;
        block_scan(sm, c, m);
        unsigned bc = c_before + c - c0;
        unsigned long long bm = m_before + m - m0;
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
          if (cs[j] && (by_count ? bc + 1 == target : (bm < target && target <= bm + ms[j]))) {
            sm.ctl.keep = sm.list[tid * kQ + j];
            sm.ctl.left = bm + ms[j];
          }
          bc += cs[j];
          bm += ms[j];
        }
        if (tid == 0) sm.list_n = 0;
        __syncthreads();
        *got = sm.ctl.left;
      }
      cluster_sync();
      keep = ls.ctl.keep;
    };
    // the leader tells whether each cut is needed
    if (lead) {
      unsigned c = 0;
      unsigned long long m = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        c += row_c[j];
        m += row_m[j];
      }
      block_scan(sm, c, m);
      if (tid == kThreads - 1) {
        sm.ctl.total = m;
        sm.ctl.warp = use_k && c > static_cast<unsigned>(k);
      }
      __syncthreads();
      Z = sm.ctl.total;
    }
    cluster_sync();
    if (ls.ctl.warp) cut(true, static_cast<unsigned long long>(k), &Z);
    if (use_p) {
      unsigned long long got;
      cut(false, tp > 0.f && lead ? ceil_share(tp, Z) : 1ull, &got);
    }
  }

  // ---- 3. the kept tokens' mass per warp, and the draw
  unsigned long long sum = 0;
  for (int i = begin + lane; i < end; i += 32) {
    const float x = logit<E>(src, i);
    if (key50(x, i) >= keep) sum += wt.weight44(x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
  if (lane == 0) ls.wsum[rank * kWarps + warp] = sum;
  cluster_sync();
  if (lead && warp == 0) {
    const int n = cl * kWarps;
    unsigned long long total = 0;
    for (int i = lane; i < n; i += 32) total += sm.wsum[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    if (lane == 0) {
      const float u = p.u[row];
      unsigned long long t = 0;
      if (u > 0.f)
        t = u >= 1.f ? total : __umul64hi(static_cast<unsigned long long>(ldexp(static_cast<double>(u), 64)), total);
      t = t < total ? t : total - 1;
      int w = 0;
      while (w < n - 1 && t >= sm.wsum[w]) t -= sm.wsum[w++];
      sm.ctl.warp = w;
      sm.ctl.left = t;
      sm.ctl.total = total;
    }
  }
  cluster_sync();
  const int win = ls.ctl.warp;
  if (win == rank * kWarps + warp) {
    const unsigned long long t = ls.ctl.left, total = ls.ctl.total;
    unsigned long long before = 0;
    for (int b = begin; b < end; b += 32) {
      const int i = b + lane;
      unsigned long long w = 0;
      if (i < end) {
        const float x = logit<E>(src, i);
        if (key50(x, i) >= keep) w = wt.weight44(x);
      }
      unsigned long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFullMask, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned hit = __ballot_sync(kFullMask, before + inc > t);
      if (hit) {
        if (lane == __ffs(hit) - 1) {
          p.token[row] = i;
          p.prob[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(total));
        }
        break;
      }
      before += __shfl_sync(kFullMask, inc, 31);
    }
  }
  cluster_sync();  // (no CTA leaves while another reads the leader's memory)
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
  // one cluster per row: as many CTAs as fill the SMs twice over
  int cl = 1;
  while (cl < kMaxCl && static_cast<long long>(rows) * cl < 304 && V / cl > 4096) cl *= 2;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (static_cast<long long>(rows) * cl > 0x7FFFFFFFll) return cache_fail(DARTREE_ERR_UNSUPPORTED, "too many rows");
  const dim3 grid(static_cast<unsigned>(rows) * cl);
  cudaError_t e = set_max_dynamic_smem(bf16 ? k_sample<uint16_t> : k_sample<float>);
  if (e == cudaSuccess)
    e = launch_kernel_cluster(bf16 ? k_sample<uint16_t> : k_sample<float>, grid, dim3(kThreads), sizeof(Smem), st,
                              false, cl, p);
  return cache_launched(e);
}
