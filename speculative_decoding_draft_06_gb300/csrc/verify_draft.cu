// Verification of drafted tokens against the target's probabilities
// (dartree_verify).
//
// At a node with target p and draft q the children's tokens were drawn from q
// one after the other without replacement.  Child x is accepted with
// probability min(1, P(x) / Q(x)), P and Q what is left of p and q; otherwise P
// becomes the normalised max(P - Q, 0), and Q loses x.  Nested, that is
//   P_k ~ max(p - A_k q, 0),   A_{k+1} = A_k + N_k / Z_k,
//   N_k = sum_i max(p_i - A_k q_i, 0),   Z_k = 1 - q(x_1) - ... - q(x_k),
// (max(max(p - a q, 0) - b q, 0) = max(p - (a + b) q, 0), and a rejected token
// has p - A q <= 0 from then on), so a rejection costs one pass for one sum.
//
// A request is the work of one thread-block cluster, which walks from the root:
// only the rows of the path are read.  Its warps have contiguous shares of a row,
// in index order.  Per node:
//   1. largest logits and sums of both rows in fp32, one pass each.  Where the
//      first child's test is not within 2^-12 of its border these decide it;
//   2. (a rejection, a border, the draw) a pass in whole numbers: weights in units
//      of 2^-44 (row_cuts.cuh), summed over the tokens with p > A q, and over all.
//      32-bit sums would not do for the draw: a row has as many borders as tokens;
//   3. no child accepted: the draw, by the warps' sums and within one warp's share.
// top-k, min-p and top-p cut the target's row first, as dartree_sample does.
#include "row_cuts.cuh"

namespace dt {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCl = 8;
constexpr int kKids = DARTREE_MAX_B;

struct VerifyParams {
  const int32_t *parent, *token, *n_out;
  const void *logits, *draft;
  long long req_stride, row_stride, draft_req_stride, draft_row_stride;
  int V, R, B, draft_rows;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *draft_temperature, *u;
  int max_len;
  int32_t *accept_len, *accept_nodes, *bonus;
  float* prob;
};

// A warp's sums of a pass, in units of 2^-44 of the rows' largest weights: p and
// q over all tokens, and over those with p > A q.
struct Sums {
  unsigned long long p, q, over_p, over_q;
};

struct Smem {
  static constexpr int kThreads = kWarps * 32;
  __align__(16) float2 exp[1 << kExpBits];
  unsigned mass_lo[kBins], mass_hi[kBins], count[kBins];
  unsigned long long cls[kClass];
  unsigned long long list[1];  // (row_cuts' lists are not used)
  // the exchange: a slot per warp of the cluster, in every CTA.  Its halves take
  // turns: when one is written again, every CTA has come to the barrier behind the
  // other's writing, and so has read it
  union Slot {
    Sums sums;
    float4 stats;
    unsigned long long best;
  };
  __align__(16) Slot slot[2][kMaxCl * kWarps];
  unsigned long long scan_m[kWarps];
  unsigned scan_c[kWarps];
  unsigned cls_n;
  int picked;
  unsigned picked_n, picked_c;
  unsigned long long picked_m;
  Ctl ctl;
  int kids[kKids], tokens[kKids];
  int kid_count[kWarps];
};

// kN consecutive logits from src + at (NaN as -inf; `wide`: 16-byte loads).
template <typename E, int kN>
__device__ __forceinline__ void load_logits(const E* src, int at, bool wide, float (&x)[kN]) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));
  if (wide) {
    if constexpr (kN >= kPer) {
#pragma unroll
      for (int k = 0; k < kN; k += kPer) {
        float y[kPer];
        unpack<E>(__ldg(reinterpret_cast<const uint4*>(src + at + k)), y);
#pragma unroll
        for (int j = 0; j < kPer; ++j) x[k + j] = y[j];
      }
    } else {  // four of 16 bits
      static_assert(kN * sizeof(E) == 8, "half a unit");
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + at));
      x[0] = __uint_as_float(v.x << 16);
      x[1] = __uint_as_float(v.x & 0xFFFF0000u);
      x[2] = __uint_as_float(v.y << 16);
      x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = logit<E>(src, at + k);
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) x[k] = fmaxf(x[k], -INFINITY);
}

// log2(e) / T as a sum of two floats.
__device__ __forceinline__ void set_temperature(Weights& wt, float T) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-8f;
  wt.ch = __fdiv_rn(kLog2e, T);
  wt.cl = isfinite(wt.ch) && isfinite(T) ? __fdiv_rn(fmaf(-wt.ch, T, kLog2e) + kLog2eLo, T) : 0.f;
}

// (m, s): the largest logit and the sum of 2^((x - m) ch) of two shares, joined.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2, float ch) {
  const float t = fmaxf(m, m2);
  if (t > -INFINITY) s = s * ex2((m - t) * ch) + s2 * ex2((m2 - t) * ch);
  m = t;
}

// The same of a warp's share of a row (a lane's part of it).
template <typename E>
__device__ __forceinline__ void row_stats(const Row<E>& row, int ub, int ue, bool first, bool last, float ch, float& m,
                                          float& s) {
  constexpr int kPer = Row<E>::kPer, kAhead = 4;
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  s = 0.f;
  auto take = [&](uint4 v) {
    float x[kPer];
    unpack<E>(v, x);
    const float t = fmaxf(max_of(x), -INFINITY);
    if (t > m) {
      s *= ex2((m - t) * ch);
      m = t;
    }
    if (m > -INFINITY) {
      float w = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) w += ex2((fmaxf(x[k], -INFINITY) - m) * ch);
      s += w;
    }
  };
  for (int u = ub + lane; u < ue; u += 32 * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (u + 32 * a < ue) v[a] = row.load(u + 32 * a);
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (u + 32 * a < ue) take(v[a]);
  }
  auto one = [&](int i) {
    const float x = logit<E>(row.src, i);
    if (x > -INFINITY) join_stats(m, s, x, 1.f, ch);
  };
  if (first && lane < row.head) one(lane);
  const int rest = row.index(row.units);
  if (last && lane < row.V - rest) one(rest + lane);
}

// c q^ in whole units for the tokens with p^ > c q^ (about: at most p^): c = m 2^-s.
struct Scale {
  unsigned long long m;
  int s;
  __device__ __forceinline__ explicit Scale(double c) {
    const int e = c > 0. ? ilogb(c) : 0;
    m = c > 0. ? static_cast<unsigned long long>(scalbn(c, 62 - e)) : 0ull;  // [2^62, 2^63)
    s = 62 - e;
  }
  __device__ __forceinline__ unsigned long long of(unsigned long long q, unsigned long long most) const {
    // q < 2^45: (q 2^18) m / 2^64 = c q 2^(s - 46)
    const unsigned long long h = __umul64hi(q << 18, m);
    const int down = s - 46;
    const unsigned long long x = down >= 64 ? 0ull : down >= 0 ? h >> down : down > -64 ? h << -down : most;
    return min(x, most);
  }
};

template <typename E, typename F>
__global__ void __launch_bounds__(kThreads) k_verify(const VerifyParams p) {
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
  const int r = blockIdx.x / cl;
  const int gw = rank * kWarps + warp, gn = cl * kWarps;
  Smem& ls = *at_rank(&sm, 0);
  const bool lead = rank == 0;

  const float T = p.temperature ? p.temperature[r] : 1.f;
  const float Td = p.draft_temperature && p.draft_temperature[r] > 0.f ? p.draft_temperature[r] : 1.f;
  Rule rule;
  rule.k = p.top_k ? p.top_k[r] : 0;
  rule.tp = p.top_p ? p.top_p[r] : 1.f;
  rule.mp = p.min_p && p.min_p[r] > 0.f ? fminf(p.min_p[r], 1.f) : 0.f;
  rule.use_k = rule.k >= 1 && rule.k < p.V;
  rule.use_p = rule.tp < 1.f;
  const bool greedy = !(T > 0.f);
  Weights wp, wq;
  wp.exp = wq.exp = sm.exp;
  set_temperature(wp, greedy ? 1.f : T);
  set_temperature(wq, Td);
  for (int i = tid; i < (1 << kExpBits); i += kThreads)
    sm.exp[i] = make_float2(__ldg(g_exp.v + 2 * i), __ldg(g_exp.v + 2 * i + 1));
  if (tid == 0) sm.cls_n = 0;

  const float* u = p.u + static_cast<size_t>(r) * (p.B + 1);
  const int32_t* token = p.token + static_cast<size_t>(r) * p.B;
  const int32_t* parent = p.parent ? p.parent + static_cast<size_t>(r) * p.B : nullptr;
  const int n = max(0, min(p.n_out[r], p.B));
  int par = 0;  // which half of the exchange is next
  int cur = 0, len = 0;
  cluster_sync();  // (every CTA's memory is there)

  for (;;) {
    const E* prow = static_cast<const E*>(p.logits) + static_cast<size_t>(r) * p.req_stride +
                    static_cast<size_t>(cur) * p.row_stride;
    const F* qrow = static_cast<const F*>(p.draft) + static_cast<size_t>(r) * p.draft_req_stride +
                    static_cast<size_t>(cur) * p.draft_row_stride;
    // ---- the node's children in order; of several with one token the first
    int kids = 0;
    if (!parent) {
      kids = cur < n ? 1 : 0;
      if (tid == 0 && kids) {
        sm.kids[0] = cur;
        sm.tokens[0] = token[cur];
      }
      __syncthreads();
    } else {
      for (int b = cur; b < n; b += kThreads) {
        const int i = b + tid;
        const bool mine = i < n && parent[i] == cur - 1;
        const unsigned in = __ballot_sync(kFullMask, mine);
        if (lane == 0) sm.kid_count[warp] = __popc(in);
        __syncthreads();
        int at = kids;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) at += sm.kid_count[w];
          kids += sm.kid_count[w];
        }
        if (mine) {
          at += __popc(in & ((1u << lane) - 1u));
          sm.kids[at] = i;
          sm.tokens[at] = token[i];
        }
        __syncthreads();
      }
    }
    if (cur >= p.draft_rows) kids = 0;  // (no draft distribution: nothing was drawn there)

    // ---- 1. the rows' largest logits and sums
    const Row<E> row(prow, p.V);
    const int share = (row.units + gn - 1) / gn;
    const int ub = min(row.units, gw * share), ue = min(row.units, ub + share);
    unsigned long long total_p = 0, total_q = 0;  // exact, once they are known
    float top_p, sum_p, top_q = -INFINITY, sum_q = 0.f;
    {
      row_stats<E>(row, ub, ue, gw == 0, gw == gn - 1, wp.ch, top_p, sum_p);
      if (kids > 0 && !greedy) {
        const Row<F> qr(qrow, p.V);
        const int qs = (qr.units + gn - 1) / gn, qb = min(qr.units, gw * qs), qe = min(qr.units, qb + qs);
        row_stats<F>(qr, qb, qe, gw == 0, gw == gn - 1, wq.ch, top_q, sum_q);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        join_stats(top_p, sum_p, __shfl_xor_sync(kFullMask, top_p, o), __shfl_xor_sync(kFullMask, sum_p, o), wp.ch);
        join_stats(top_q, sum_q, __shfl_xor_sync(kFullMask, top_q, o), __shfl_xor_sync(kFullMask, sum_q, o), wq.ch);
      }
      if (lane < cl) at_rank(&sm, lane)->slot[par][gw].stats = make_float4(top_p, sum_p, top_q, sum_q);
      cluster_sync();
      top_p = top_q = -INFINITY;
      sum_p = sum_q = 0.f;
      for (int w = lane; w < gn; w += 32) {
        const float4 x = sm.slot[par][w].stats;
        join_stats(top_p, sum_p, x.x, x.y, wp.ch);
        join_stats(top_q, sum_q, x.z, x.w, wq.ch);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        join_stats(top_p, sum_p, __shfl_xor_sync(kFullMask, top_p, o), __shfl_xor_sync(kFullMask, sum_p, o), wp.ch);
        join_stats(top_q, sum_q, __shfl_xor_sync(kFullMask, top_q, o), __shfl_xor_sync(kFullMask, sum_q, o), wq.ch);
      }
      // (a join's rounding depends on its order, which is not the same in all lanes;
      // what is decided has to be)
      sum_p = __shfl_sync(kFullMask, sum_p, 0);
      sum_q = __shfl_sync(kFullMask, sum_q, 0);
      par ^= 1;
    }
    wp.top = top_p;
    wq.top = top_q;
    if (top_p == -INFINITY) {  // nothing to choose from
      if (lead && tid == 0) {
        p.bonus[r] = -1;
        p.prob[r] = 0.f;
      }
      break;
    }
    if (greedy) {  // the lowest index of the largest logit
      const RowSource<false, E, Smem> s{sm, ls, row, ub, ue, gw == 0, gw == gn - 1, 0, cl, lead, gw, max(share, 1)};
      unsigned long long best = 0;
      s.each_value([&](float x, int i) {
        if (x == top_p) best = max(best, key50(x, i));
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
      if (lane < cl) at_rank(&sm, lane)->slot[par][gw].best = best;
      cluster_sync();
      best = 0;
      for (int w = lane; w < gn; w += 32) best = max(best, sm.slot[par][w].best);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
      par ^= 1;
      const int x = (1 << kIdxBits) - 1 - static_cast<int>(best & ((1u << kIdxBits) - 1));
      int next = -1;
      for (int k = kids - 1; k >= 0; --k)
        if (sm.tokens[k] == x) next = sm.kids[k];
      __syncthreads();  // (the children may be written again)
      if (next < 0) {
        if (lead && tid == 0) {
          p.bonus[r] = x;
          p.prob[r] = 1.f;
        }
        break;
      }
      if (lead && tid == 0 && len < p.max_len) p.accept_nodes[static_cast<size_t>(r) * p.max_len + len] = next;
      ++len;
      cur = next + 1;
      continue;
    }

    // ---- the cuts: kept are the tokens whose key reaches `keep`
    unsigned long long keep = 0;
    if (rule.use_k || rule.use_p || rule.mp > 0.f) {
      const RowSource<false, E, Smem> s{sm, ls, row, ub, ue, gw == 0, gw == gn - 1, 0, cl, lead, gw, max(share, 1)};
      keep = rule.mp > 0.f ? min_p_key(wp, rule.mp) : 0;
      fill_bins(s, wp, keep);
      unsigned count = 0;
      unsigned long long Z = 0;
      if (lead) {
        all_classes(s, &count, &Z);
        if (tid == 0) {
          ls.ctl.warp = rule.use_k && count > static_cast<unsigned>(rule.k);
          ls.ctl.total = Z;
        }
      }
      cluster_sync();
      if (ls.ctl.warp) {
        const bool refined = cut(s, wp, true, static_cast<unsigned long long>(rule.k), keep, &Z);
        if (refined && rule.use_p) fill_bins(s, wp, keep);
      }
      if (rule.use_p) {
        unsigned long long upto = 0;
        cut(s, wp, false, rule.tp > 0.f && lead ? ceil_share(rule.tp, Z) : 1ull, keep, &upto);
        Z = upto;
      }
      if (lead && tid == 0) ls.ctl.total = Z;
      cluster_sync();
      total_p = ls.ctl.total;
    }
    const float keep_x = keep ? key50_value(keep) : -INFINITY;

    // ---- 2. a pass in whole numbers, for the A given
    double A = 0., N = 1.;
    bool sums_for_A = false;  // slot[par ^ 1] has the sums of A
    unsigned long long over_p = 0, over_q = 0;
    auto each_pair = [&](bool with_q, auto f) {  // f(p's logit, q's, index)
      const bool wide = with_q && ((reinterpret_cast<uintptr_t>(qrow + row.head) &
                                    (sizeof(F) < sizeof(E) ? 7 : 15)) == 0);
      auto one = [&](int i) {
        const float x = logit<E>(prow, i);
        f(x, with_q ? logit<F>(qrow, i) : -INFINITY, i);
      };
      if (gw == 0 && lane < row.head) one(lane);
      const int rest = row.index(row.units);
      if (gw == gn - 1 && lane < p.V - rest) one(rest + lane);
      for (int a = ub + lane; a < ue; a += 32) {
        float x[kPer], y[kPer];
        unpack<E>(row.load(a), x);
        if (with_q) {
          load_logits<F, kPer>(qrow, row.index(a), wide, y);
        } else {
#pragma unroll
          for (int k = 0; k < kPer; ++k) y[k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) f(fmaxf(x[k], -INFINITY), y[k], row.index(a) + k);
      }
    };
    // p's weight of a kept token, in log2 (0 for the largest)
    auto kept = [&](float x, int i) { return x > keep_x || (x == keep_x && key50(x, i) >= keep); };
    // log2 of c = A sum_p / sum_q, where q's weights are to be compared with p's
    auto log2_c = [&]() {
      const float sp = total_p ? __ull2float_rn(total_p) * 0x1p-44f : sum_p;
      const float sq = total_q ? __ull2float_rn(total_q) * 0x1p-44f : sum_q;
      return A > 0. ? log2f(static_cast<float>(A)) + log2f(sp) - log2f(sq) : -INFINITY;
    };
    auto pass = [&](bool with_q) {
      const float lc = log2_c();
      const bool all = total_q == 0 || total_p == 0;  // the rows' totals are wanted too
      Sums t{0, 0, 0, 0};
      each_pair(with_q, [&](float x, float y, int i) {
        const bool in = kept(x, i);
        const float a = in ? wp.log2w(x) : -INFINITY, b = with_q ? wq.log2w(y) : -INFINITY;
        const bool over = a > -INFINITY && a > b + lc;
        if (!all && !over) return;
        const unsigned long long v = in ? wp.weight44(x) : 0ull, w = with_q ? wq.weight44(y) : 0ull;
        t.p += v;
        t.q += w;
        if (over) {
          t.over_p += v;
          t.over_q += w;
        }
      });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t.p += __shfl_xor_sync(kFullMask, t.p, o);
        t.q += __shfl_xor_sync(kFullMask, t.q, o);
        t.over_p += __shfl_xor_sync(kFullMask, t.over_p, o);
        t.over_q += __shfl_xor_sync(kFullMask, t.over_q, o);
      }
      if (lane < cl) at_rank(&sm, lane)->slot[par][gw].sums = t;
      cluster_sync();
      t = Sums{0, 0, 0, 0};
      for (int w = lane; w < gn; w += 32) {
        const Sums x = sm.slot[par][w].sums;
        t.p += x.p;
        t.q += x.q;
        t.over_p += x.over_p;
        t.over_q += x.over_q;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t.p += __shfl_xor_sync(kFullMask, t.p, o);
        t.q += __shfl_xor_sync(kFullMask, t.q, o);
        t.over_p += __shfl_xor_sync(kFullMask, t.over_p, o);
        t.over_q += __shfl_xor_sync(kFullMask, t.over_q, o);
      }
      if (all) {
        total_p = t.p;
        if (with_q) total_q = t.q;
      }
      over_p = t.over_p;
      over_q = t.over_q;
      par ^= 1;
      sums_for_A = true;
    };

    // ---- the children's tests
    int next = -1;
    unsigned long long tried = 0;  // q's weight of the rejected ones
    for (int k = 0; k < kids && next < 0; ++k) {
      const int x = sm.tokens[k], node = sm.kids[k];
      bool dead = x < 0 || x >= p.V;
      for (int j = 0; j < k; ++j) dead = dead || sm.tokens[j] == x;
      if (dead) continue;
      const float lq = logit<F>(qrow, x), lp = logit<E>(prow, x);
      const unsigned long long q = top_q > -INFINITY ? wq.weight44(lq) : 0ull;
      if (q == 0) continue;  // it cannot have been drawn
      const unsigned long long w = kept(lp, x) ? wp.weight44(lp) : 0ull;
      const double ux = static_cast<double>(u[node + 1]), qd = static_cast<double>(q), pd = static_cast<double>(w);
      bool yes = false;
      if (A == 0.) {
        const bool exact = total_p != 0 && total_q != 0;
        if (!exact) {
          const float sp = total_p ? __ull2float_rn(total_p) * 0x1p-44f : sum_p;
          const float lhs = u[node + 1] * static_cast<float>(qd) * sp, rhs = static_cast<float>(pd) * sum_q;
          const float gap = fabsf(lhs - rhs);
          if (!(isfinite(lhs) && isfinite(rhs) && gap > rhs * (1.f / 4096.f))) pass(true);
          yes = lhs < rhs;
        }
        if (total_p != 0 && total_q != 0)
          yes = ux * qd * static_cast<double>(total_p) < pd * static_cast<double>(total_q);
      } else if (N > 0.) {
        const double np = static_cast<double>(total_p), nq = static_cast<double>(total_q);
        const double left = total_q > tried ? static_cast<double>(total_q - tried) : 0.;
        // (Z = left / nq; nothing left of q: it cannot have been drawn)
        if (left <= 0.) continue;
        const double a = N * nq / left;
        yes = ux * a * (qd / nq) < pd / np - A * (qd / nq);
      }
      if (yes) {
        next = node;
        break;
      }
      if (N <= 0.) continue;
      const double z = A == 0. ? 1. : static_cast<double>(total_q - tried) / static_cast<double>(total_q);
      A += N / z;
      tried += q;
      pass(true);
      N = static_cast<double>(over_p) / static_cast<double>(total_p) -
          A * (static_cast<double>(over_q) / static_cast<double>(total_q));
      if (!(N > 0x1p-40)) N = 0.;  // (nothing but rounding)
    }
    if (next >= 0) {
      __syncthreads();  // (the children may be written again)
      if (lead && tid == 0 && len < p.max_len) p.accept_nodes[static_cast<size_t>(r) * p.max_len + len] = next;
      ++len;
      cur = next + 1;
      continue;
    }

    // ---- 3. the draw from max(p - A q, 0), from p where that is nothing
    if (N <= 0.) A = 0.;
    const bool with_q = A > 0.;
    if (!sums_for_A || !with_q) {
      total_p = 0;
      pass(false);
    }
    const double c = with_q ? A * static_cast<double>(total_p) / static_cast<double>(total_q) : 0.;
    const int from = par ^ 1;
    constexpr int kEach = kMaxCl * kWarps / 32;
    double mine[kEach], sum = 0.;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int w = lane * kEach + k;
      mine[k] = 0.;
      if (w < gn) {
        const Sums x = sm.slot[from][w].sums;
        mine[k] = fmax(static_cast<double>(x.over_p) - c * static_cast<double>(x.over_q), 0.);
      }
      sum += mine[k];
    }
    double inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(kFullMask, inc, o);
      if (lane >= o) inc += y;
    }
    const double total = __shfl_sync(kFullMask, inc, 31);
    const double u0 = static_cast<double>(u[0]);
    const double mark = u0 > 0. ? fmin(u0, 1.) * total : 0.;
    // the warp in whose share the running sum passes the mark; behind all of
    // them, the last that has any
    double before = inc - sum, left = 0.;
    int owner = -1, last = -1;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (owner < 0 && mine[k] > 0. && before + mine[k] > mark) {
        owner = lane * kEach + k;
        left = mark - before;
      }
      if (mine[k] > 0.) last = lane * kEach + k;
      before += mine[k];
    }
    const unsigned hit = __ballot_sync(kFullMask, owner >= 0);
    if (hit) {
      const int src = __ffs(hit) - 1;
      owner = __shfl_sync(kFullMask, owner, src);
      left = __shfl_sync(kFullMask, left, src);
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(kFullMask, last, o));
      owner = last;
      left = 0x1p63;
    }
    if (owner == gw) {
      const unsigned long long t = left > 0. ? (left < 0x1p63 ? static_cast<unsigned long long>(left) : ~0ull) : 0ull;
      const Scale sc(c);
      const float lc = log2_c();
      unsigned long long run = 0, last_w = 0;
      int last_i = -1;
      bool found = false;
      const bool wide = (reinterpret_cast<uintptr_t>(qrow + row.head) & (sizeof(F) < sizeof(E) ? 7 : 15)) == 0;
      auto residual = [&](float x, float y, int i) -> unsigned long long {
        if (!kept(x, i)) return 0ull;
        if (with_q && !(wp.log2w(x) > wq.log2w(y) + lc)) return 0ull;
        const unsigned long long v = wp.weight44(x);
        return with_q ? v - sc.of(wq.weight44(y), v) : v;
      };
      auto emit = [&](int i, unsigned long long w) {
        p.bonus[r] = i;
        p.prob[r] = static_cast<float>(static_cast<double>(w) / total);
      };
      // the lane's tokens i0 .. i0 + m - 1 of a step, in index order over the lanes
      auto step = [&](const float (&x)[kPer], const float (&y)[kPer], int i0, int m) {
        unsigned long long w[kPer], own = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          w[k] = k < m ? residual(x[k], y[k], i0 + k) : 0ull;
          own += w[k];
          if (w[k]) {
            last_i = i0 + k;
            last_w = w[k];
          }
        }
        unsigned long long upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long z = __shfl_up_sync(kFullMask, upto, o);
          if (lane >= o) upto += z;
        }
        const unsigned hits = __ballot_sync(kFullMask, run + upto > t);
        if (hits && lane == __ffs(hits) - 1) {
          unsigned long long at = run + upto - own;
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            if (at <= t && at + w[k] > t) emit(i0 + k, w[k]);
            at += w[k];
          }
        }
        run += __shfl_sync(kFullMask, upto, 31);
        found = hits != 0;
      };
      float x[kPer], y[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[k] = y[k] = -INFINITY;
      auto single = [&](int i, bool on) {
        if (on) {
          x[0] = logit<E>(prow, i);
          if (with_q) y[0] = logit<F>(qrow, i);
        }
        step(x, y, i, on ? 1 : 0);
      };
      if (gw == 0 && row.head > 0) single(lane, lane < row.head);
      for (int b = ub; b < ue && !found; b += 32) {
        const int a = b + lane;
        if (a < ue) {
          unpack<E>(row.load(a), x);
#pragma unroll
          for (int k = 0; k < kPer; ++k) x[k] = fmaxf(x[k], -INFINITY);
          if (with_q) load_logits<F, kPer>(qrow, row.index(a), wide, y);
        }
        step(x, y, row.index(a), a < ue ? kPer : 0);
      }
      const int rest = row.index(row.units);
      if (!found && gw == gn - 1 && rest < p.V) single(rest + lane, rest + lane < p.V);
      if (!found) {  // (the running sum ends below the mark by its rounding)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const int i2 = __shfl_xor_sync(kFullMask, last_i, o);
          const unsigned long long w2 = __shfl_xor_sync(kFullMask, last_w, o);
          if (i2 > last_i) {
            last_i = i2;
            last_w = w2;
          }
        }
        if (lane == 0) emit(last_i, last_w);
      }
    }
    break;
  }
  if (lead) {
    if (tid == 0) p.accept_len[r] = len;
    for (int i = len + tid; i < p.max_len; i += kThreads) p.accept_nodes[static_cast<size_t>(r) * p.max_len + i] = -1;
  }
  cluster_sync();  // (no CTA leaves while another reads or writes its memory)
}

template <typename E, typename F>
cudaError_t launch_verify(const VerifyParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(k_verify<E, F>, &done);
  if (e != cudaSuccess) return e;
  // a request's rows over as many CTAs as the SMs hold (two each)
  int cl = 1;
  while (cl < kMaxCl && static_cast<long long>(p.R) * cl * 2 <= 304 && p.V / cl > 4096) cl *= 2;
  return launch_kernel_cluster(k_verify<E, F>, dim3(static_cast<unsigned>(p.R) * cl), dim3(kThreads), sizeof(Smem), st,
                               true, cl, p);
}

}  // namespace
}  // namespace dt

extern "C" dartree_status dartree_verify(const int32_t* parent, const int32_t* token, const int32_t* n_out,
                                         const void* logits, int32_t bf16, int64_t req_stride, int64_t row_stride,
                                         const void* draft, int32_t draft_bf16, int64_t draft_req_stride,
                                         int64_t draft_row_stride, int32_t draft_rows, int32_t V, int32_t R, int32_t B,
                                         const float* temperature, const int32_t* top_k, const float* top_p,
                                         const float* min_p, const float* draft_temperature, const float* u,
                                         int32_t max_len, int32_t* accept_len, int32_t* accept_nodes, int32_t* bonus,
                                         float* prob, void* stream) {
  using namespace dt;
  if (!token || !n_out || !logits || !draft || !u || !accept_len || !accept_nodes || !bonus || !prob)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (V < 1 || R < 1 || B < 1 || draft_rows < 1 || max_len < 1)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "bad V, R, B, draft_rows or max_len");
  if (row_stride < V || draft_row_stride < V || req_stride < 0 || draft_req_stride < 0)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "rows are V logits, one after the other");
  if (V > (1 << kIdxBits)) return cache_fail(DARTREE_ERR_UNSUPPORTED, "V must be at most 2^18");
  if (B > DARTREE_MAX_B) return cache_fail(DARTREE_ERR_UNSUPPORTED, "a tree has at most 1024 nodes");
  if (R > (1 << 24)) return cache_fail(DARTREE_ERR_UNSUPPORTED, "verify takes at most 2^24 requests");
  const uintptr_t odd = (reinterpret_cast<uintptr_t>(logits) & (bf16 ? 1 : 3)) |
                        (reinterpret_cast<uintptr_t>(draft) & (draft_bf16 ? 1 : 3));
  if (odd) return cache_fail(DARTREE_ERR_INVALID_ARG, "logits and draft must be aligned to their type");
  const VerifyParams p{parent, token, n_out, logits, draft, req_stride, row_stride, draft_req_stride, draft_row_stride,
                       V, R, B, draft_rows, temperature, top_k, top_p, min_p, draft_temperature, u,
                       max_len, accept_len, accept_nodes, bonus, prob};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? (draft_bf16 ? launch_verify<uint16_t, uint16_t>(p, st) : launch_verify<uint16_t, float>(p, st))
                             : (draft_bf16 ? launch_verify<float, uint16_t>(p, st) : launch_verify<float, float>(p, st));
  return cache_launched(e);
}
