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
// in index order.  The children's tests take sums in fp32 with a bound of their
// error: a pass for the rows' largest logits and sums, one per rejection.  Whole
// numbers (weights in units of 2^-44, row_cuts.cuh; a table of bf16's codes) decide
// where a test lies within the bound, and the draw at the path's end: there 32-bit
// sums would not do, a row has as many borders as tokens.  One pass gives them for
// up to kLevels rejections: what enters N_k are the sums of p and of q over the
// tokens with p > A_k q, which the logarithms and the approximate A_k tell apart to
// 2^-14 (kBorder); the exact A_k follow from them.  Where the tokens that lie nearer
// to the border could matter to N_k (a target that is its draft but for a few tokens),
// one more pass takes those in whole numbers, by the exact A_k.
// top-k, min-p and top-p cut the target's row first, as dartree_sample does; a bf16
// row by counts of its codes.
//
// Bound by latency: a path's nodes wait for one another, and each is a chain of
// passes, barriers of the cluster and scalar steps, 4 us at the least; the pass in
// whole numbers by issue and by its table's bank conflicts (two look-ups a token).
// One chain of 8 over 32000 fp32 logits 30 to 38 us (by its path); 16 trees of 128 nodes
// over 151936 in bf16 101 to 117 us, 64 chains of 7 with settings of their own 258 to
// 351 us (both to the end of their longest paths; the rows of all paths read once would
// take 10 and 20 us).  Steps for the trees (the chains; by other draws than these):
// every sum in whole numbers 210 us (837); tests in fp32, one pass in whole numbers per
// path, its fp64 in one warp 147 (440, top-p); floors and lists for top-k, the pass at
// the draw in line 137 (385); acceptance before the cut 140 (318); a node's state and
// the cuts' arguments in registers, copies of them for the calls, 136 to 104 (301 to
// 266).  The passes as calls cost 7%, two CTAs of 512 threads to an SM (64 registers) 20
// to 40%, copies in registers inside the calls of a Node too 3 to 10%.  The tokens at the
// border p = A q in whole numbers cost 1%.
#include "row_cuts.cuh"

namespace dt {

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

namespace {

constexpr int kThr = 512;
constexpr int kMaxCl = 8;
constexpr int kLevels = 4;           // rejections of a pass in whole numbers
constexpr int kNotes = 256;           // tokens that a warp notes in a scan
constexpr int kFew = 512;            // tokens of a list on which top-k is decided by comparing all
constexpr float kBorder = 0x1p-14f;  // what log2 p - log2 A q may be off by: two logarithms below 46, three
                                     // roundings each, 2^-15.9; A by 2^-17 and the rows' sums by 2^-18, 2^-15.5
constexpr float kSumError = 0x1p-15f;  // relative error of a sum in fp32: a lane's 130 additions one after the
                                       // other (2^18 tokens, one CTA) 2^-17; logits' differences times log2(e) / T
                                       // below 46, three roundings, 2^-17.4; 128 new largest logits, each an ex2
                                       // (2^-22) for half of the sum, 2^-16

// A warp's sums of a pass, in units of 2^-44 of the rows' largest weights: p and
// q over all tokens, and over those with p > A_k q.
struct Sums {
  unsigned long long p, q, over_p[kLevels], over_q[kLevels];
};

struct VerifySmem {
  static constexpr int kThreads = kThr, kWarps = kThr / 32, kListMost = 2048;
  static constexpr bool kWideSums = true;
  __align__(16) float2 exp[1 << kExpBits];
  union {  // the cuts; behind them the weights of bf16's codes
    struct {
      union {
        struct {
          unsigned mass_lo[kBins], mass_hi[kBins], count[kBins];
        };
        unsigned codes[2 * kTable];
      };
      unsigned long long cls[kClass];
      unsigned long long list[kListMost];
    };
    struct {
      unsigned long long table_p[2 * kTable], table_q[2 * kTable];
    };
  };
  // the exchange: a slot per warp of the cluster, in every CTA.  Its halves take
  // turns: when one is written again, every CTA has come to the barrier behind the
  // other's writing, and so has read it
  union Slot {
    Sums sums;
    float4 stats;
    unsigned long long best;
  };
  __align__(16) Slot slot[2][kMaxCl * kWarps];
  unsigned long long near[2];      // p over the tokens within kBorder of a level's border (as slot; 0 between its uses)
  uint16_t notes[kWarps][kNotes];  // of a scan
  unsigned long long scan_m[kWarps];
  unsigned scan_c[kWarps];
  unsigned long long part[kWarps];
  unsigned cls_n, list_n;  // (list_n is 0 between its uses)
  float floor;
  int picked;
  unsigned picked_n, picked_c;
  unsigned long long picked_m;
  Ctl ctl;
  int kid_count[kWarps];
  // In 64 bits, by the first warp alone (the GPU has few units for them: each of
  // these numbers in all threads cost 10 us a node)
  struct {
    unsigned long long p, q;     // the rows' sums
    double A, N, Z;              // behind `settled` rejections
    unsigned long long gone;     // q's weight of their children
    int settled, level;          // level: whose sums slot[..] has
    int yes, drawn;              // a test's result
    double total;                // the draw: the whole residual
    unsigned long long left;     // the mark within the owner's share
    int owner;                   // the warp that has it
    unsigned long long scale_m;  // A sum_p / sum_q
    int scale_s;
    int border;                  // the next pass takes the tokens at the border in whole numbers, by it
  } ex;
};

// Behind it, B + 1 entries each.
struct TreeSmem {
  int* at;
  int n;
  static constexpr int kArrays = 8;
  __device__ __forceinline__ TreeSmem(void* from, int B) : at(static_cast<int*>(from)), n(B + 1) {}
  __device__ __forceinline__ float* floats(int k) const { return reinterpret_cast<float*>(at + k * n); }
  __device__ __forceinline__ int* parent() const { return at; }  // the request's tree and random numbers
  __device__ __forceinline__ int* token() const { return at + n; }
  __device__ __forceinline__ float* u() const { return floats(2); }
  __device__ __forceinline__ int* kids() const { return at + 3 * n; }  // the node's children
  __device__ __forceinline__ float* kid_p() const { return floats(4); }  // their logits (q -inf: passed over)
  __device__ __forceinline__ float* kid_q() const { return floats(5); }
  __device__ __forceinline__ float* reject_a() const { return floats(6); }  // the rejected ones: A behind them,
  __device__ __forceinline__ float* reject_q() const { return floats(7); }  // about, and their logits under q
};

// Weights of a row's tokens: bf16's codes from a table.
template <typename E, typename W>
struct Weigh {
  const W& w;
  const unsigned long long* table;
  Codes codes;
  __device__ __forceinline__ Weigh(const W& weights, const unsigned long long* t)
      : w(weights), table(t), codes(weights.top) {}
  __device__ __forceinline__ unsigned long long operator()(float x) const {
    if constexpr (sizeof(E) == 2) {
      const int j = codes.place(x);
      return j >= 0 ? table[j] : weight44_call(x, w.top, w.ch, w.cl, w.exp);
    } else {
      return w.weight44(x);
    }
  }
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

// log2(e) / T as a sum of two floats (of an infinite T the smallest float: 0 times the
// distance of a logit of -inf would be NaN).
__device__ __forceinline__ void set_temperature(Weights& wt, float T) {
  constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLo = 1.9259629911266175e-8f;
  wt.ch = T == INFINITY ? 0x1p-149f : __fdiv_rn(kLog2e, T);
  wt.cl = isfinite(wt.ch) && isfinite(T) ? __fdiv_rn(fmaf(-wt.ch, T, kLog2e) + kLog2eLo, T) : 0.f;
}

// (m, s): the largest logit and the sum of 2^((x - m) ch) of two shares, joined.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2, float ch) {
  const float t = fmaxf(m, m2);
  if (t > -INFINITY) s = s * ex2((m - t) * ch) + s2 * ex2((m2 - t) * ch);
  m = t;
}

// The same over a warp's lanes: the largest first, then one sum (in each lane
// the same up to its last bits).
__device__ __forceinline__ void warp_stats(float& m, float& s, float& m2, float& s2, float ch, float ch2) {
  float t = m, t2 = m2;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t = fmaxf(t, __shfl_xor_sync(kFullMask, t, o));
    t2 = fmaxf(t2, __shfl_xor_sync(kFullMask, t2, o));
  }
  s = m > -INFINITY ? s * ex2((m - t) * ch) : 0.f;
  s2 = m2 > -INFINITY ? s2 * ex2((m2 - t2) * ch2) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(kFullMask, s, o);
    s2 += __shfl_xor_sync(kFullMask, s2, o);
  }
  m = t;
  m2 = t2;
}

// The largest of a unit's logits (NaN counts as nothing).
[[maybe_unused]] __device__ __forceinline__ float unit_max(uint4 v, float) {
  return fmaxf(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))),
               -INFINITY);
}
[[maybe_unused]] __device__ __forceinline__ float unit_max(uint4 v, uint16_t) {
  const auto pair = [](uint32_t x) { return *reinterpret_cast<const __nv_bfloat162*>(&x); };
  const __nv_bfloat162 m = __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w)));
  return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
}

// The same of a warp's share of a row (a lane's part of it).  A NaN among the
// logits makes the sum NaN (and the row's tests take whole numbers).  x ch - m ch
// is one rounding, with m ch as a sum of two floats.
template <typename E>
__device__ __forceinline__ void row_stats(const Row<E>& row, int ub, int ue, bool first, bool last, float ch, float& m,
                                          float& s) {
  constexpr int kPer = Row<E>::kPer, kAhead = 4;
  const int lane = threadIdx.x & 31;
  float mc = 0.f, mcl = 0.f;
  m = -INFINITY;
  s = 0.f;
  auto take = [&](uint4 v) {
    const float t = unit_max(v, E{});
    if (t > m) {
      s *= ex2(fmaf(m - t, ch, -mcl));
      m = t;
      mc = t * ch;
      mcl = fmaf(t, ch, -mc);
    }
    if (m > -INFINITY) {
      float x[kPer], w[2] = {0.f, 0.f};
      unpack<E>(v, x);
#pragma unroll
      for (int k = 0; k < kPer; ++k) w[k & 1] += ex2(fmaf(x[k], ch, -mc));
      s += w[0] + w[1];
    }
  };
  // (the next units on their way while these are taken)
  int a = ub + lane;
  uint4 next[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (a + 32 * k < ue) next[k] = row.load(a + 32 * k);
#pragma unroll 1
  for (; a < ue; a += 32 * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) v[k] = next[k];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (a + 32 * (kAhead + k) < ue) next[k] = row.load(a + 32 * (kAhead + k));
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (a + 32 * k < ue) take(v[k]);
  }
  if (m > -INFINITY) s *= ex2(-mcl);
  auto one = [&](int i) {
    const float x = logit<E>(row.src, i);
    if (x > -INFINITY) join_stats(m, s, x, 1.f, ch);
  };
  if (first && lane < row.head) one(lane);
  const int rest = row.index(row.units);
  if (last && lane < row.V - rest) one(rest + lane);
}

// floor(c q), or `most` where that is less, for c = m 2^-s > 0.  Exact: where the sum of some
// tokens' p is above that of their q, one of them is above its own.
struct Scale {
  unsigned long long m;
  int s;
  static __device__ __forceinline__ Scale from(double c) {
    const int e = c > 0. ? ilogb(c) : 0;
    return Scale{c > 0. ? static_cast<unsigned long long>(scalbn(c, 62 - e)) : 0ull, 62 - e};  // [2^62, 2^63)
  }
  __device__ __forceinline__ unsigned long long of(unsigned long long q, unsigned long long most) const {
    const unsigned long long hi = __umul64hi(q, m), lo = q * m;
    unsigned long long x;
    if (s >= 64) x = s >= 128 ? 0ull : hi >> (s - 64);
    else if (s > 0) x = hi >> s ? most : hi << (64 - s) | lo >> s;
    else x = s == 0 && !hi ? lo : q ? most : 0ull;
    return min(x, most);
  }
};

// floor(u z) for u in (0, 1), z below 2^63.
__device__ __forceinline__ unsigned long long floor_share(float u, unsigned long long z) {
  const unsigned bits = __float_as_uint(u);
  const int exponent = static_cast<int>(bits >> 23), down = 150 - max(exponent, 1);  // u = factor 2^-down
  const unsigned long long factor = (bits & 0x7FFFFFu) | (exponent ? 0x800000u : 0u);
  const unsigned long long hi = __umul64hi(z, factor), lo = z * factor;
  return down >= 128 ? 0ull : down >= 64 ? hi >> (down - 64) : hi << (64 - down) | lo >> down;
}

// A row's tokens from a floor on, in no particular order: a warp notes them as it
// goes over its units, and takes the notes 32 at a time (what is done with a token
// costs ten times the look at it, and nearly every 32 tokens have one to be taken).
template <typename E, typename Mem>
struct FloorSource : RowSource<false, E, Mem> {
  float floor;
  __device__ __forceinline__ FloorSource(const RowSource<false, E, Mem>& s, float f) : RowSource<false, E, Mem>(s), floor(f) {}
  // f(logit, index); with `rest` -> the lane's part of the others' weights in fp32
  template <typename F>
  __device__ __forceinline__ float scan(const Weights& wt, bool rest, F f) const {
    constexpr int kPer = Row<E>::kPer;
    const Row<E>& row = this->row;
    const int lane = threadIdx.x & 31, ub = this->ub, ue = this->ue, base = row.index(ub);
    uint16_t* notes = this->sm.notes[threadIdx.x >> 5];
    int n = 0;
    float skipped = 0.f;
    auto flush = [&]() {
      __syncwarp();
#pragma unroll 1
      for (int b = lane; b < n; b += 32) {
        const int i = base + notes[b];
        f(logit<E>(row.src, i), i);
      }
      __syncwarp();
      n = 0;
    };
    auto one = [&](int i) {
      const float x = logit<E>(row.src, i);
      if (x >= floor && x > -INFINITY) f(x, i);
      else if (rest) skipped += ex2(wt.log2w(x));
    };
    if (this->first && lane < row.head) one(lane);
    const int end = row.index(row.units);
    if (this->last && lane < row.V - end) one(end + lane);
    uint4 next = ub + lane < ue ? row.load(ub + lane) : make_uint4(0, 0, 0, 0);
#pragma unroll 1
    for (int b = ub; b < ue; b += 32) {
      const uint4 v = next;
      const bool on = b + lane < ue;
      if (b + 32 + lane < ue) next = row.load(b + 32 + lane);
      const float top = on ? unit_max(v, E{}) : -INFINITY;
      const bool any = __any_sync(kFullMask, top >= floor && top > -INFINITY);
      if (!any && !rest) continue;
      float x[kPer];
      unpack<E>(v, x);
      if (any) {
        const int at = row.index(b + lane) - base;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const bool in = on && x[k] >= floor && x[k] > -INFINITY;
          const unsigned who = __ballot_sync(kFullMask, in);
          if (in) {
            notes[n + __popc(who & ((1u << lane) - 1u))] = static_cast<uint16_t>(at + k);
            x[k] = -INFINITY;
          }
          n += __popc(who);
          if (n > kNotes - 32) flush();
        }
      }
      if (rest && on) {
        float w = 0.f;
#pragma unroll
        for (int k = 0; k < kPer; ++k) w += ex2(wt.log2w(x[k]));
        skipped += w;
      }
    }
    flush();
    return skipped;
  }
  template <typename F>
  __device__ __forceinline__ void each_value(F f) const {
    scan(Weights{}, false, f);
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    each_value([&](float x, int i) { f(x, key50(x, i)); });
  }
};

// A value that the row's k-th largest logit reaches: the k-th largest of the warps'
// largest, or a little below the k-th largest of the lanes' (by classes, with two
// barriers of the cluster).
template <typename S>
__device__ __noinline__ float kth_floor(const S& given, const Weights& its_wp, int k, float lane_top, int half) {
  const S src(given);
  const Weights wp(its_wp);
  using Mem = typename S::Mem;
  Mem& sm = src.sm;
  const int warps = src.cl * Mem::kWarps, tid = threadIdx.x;
  if (k <= warps) {
    if (tid < warps) {
      const float mine = sm.slot[half][tid].stats.x;
      int above = 0;
#pragma unroll 4
      for (int w = 0; w < warps; ++w) {
        const float x = sm.slot[half][w].stats.x;
        above += x > mine || (x == mine && w < tid);
      }
      if (above == k - 1) sm.floor = mine;
    }
    __syncthreads();
    return sm.floor;
  }
  clear_classes(sm);
  __syncthreads();
  if (lane_top > -INFINITY) atomicAdd(&sm.count[bin_of(wp, lane_top)], 1u);
  cluster_sync();
  Ctl& ctl = src.ls.ctl;
  if (src.lead) {
    unsigned lanes, c = 0, members = 0;
    unsigned long long none = 0;
    all_classes(src, &lanes, &none);
    none = 0;
    const int b = lanes >= static_cast<unsigned>(k) ? pick_class(src, true, k, c, none, &members) : kBins;
    if (tid == 0) ctl.bin = b;
  }
  cluster_sync();
  // (class b ends half a step below its middle)
  return ctl.bin < kBins - 1 ? wp.top - (static_cast<float>(ctl.bin) + 1.f) / (kBinsPer2 * wp.ch) : -INFINITY;
}

// The cuts of the few tokens in the leader's list (its block; every token that
// reaches the list's least is in it, k of them at least): each against all.
template <typename S>
__device__ __noinline__ void list_cut(const S& given, const Weights& its_wp, const Rule& its_rule, unsigned long long least, int n) {
  const S src(given);
  const Weights wp(its_wp);
  const Rule rule(its_rule);
  auto& sm = src.sm;
  const CalledWeights called(wp);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = S::Mem::kWarps, kPer = kFew / S::Mem::kThreads;
  unsigned long long key[kPer], w[kPer], before[kPer], top = 0, end = ~0ull;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int i = tid + q * S::Mem::kThreads;
    key[q] = i < n ? sm.list[i] : 0ull;
    w[q] = i < n ? called.weight44(key50_value(key[q])) : 0ull;
    before[q] = 0;
    sm.cls[i] = w[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    unsigned rank = 0;
    if (key[q] != 0) {
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const bool above = sm.list[j] > key[q];
        rank += above;
        before[q] += above ? sm.cls[j] : 0ull;
      }
    }
    if (key[q] == 0 || key[q] < least || rank >= static_cast<unsigned>(rule.k)) key[q] = 0;
    else {
      top = max(top, before[q] + w[q]);
      end = min(end, key[q]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top = max(top, __shfl_xor_sync(kFullMask, top, o));
    end = min(end, __shfl_xor_sync(kFullMask, end, o));
  }
  if (lane == 0) {
    sm.scan_m[warp] = top;
    sm.part[warp] = end;
  }
  __syncthreads();
  for (int k = 0; k < kWarps; ++k) {
    top = max(top, sm.scan_m[k]);
    end = min(end, sm.part[k]);
  }
  if (!rule.use_p) {
    if (tid == 0) {
      sm.ctl.keep = end;
      sm.ctl.total = top;
    }
    return;
  }
  const unsigned long long target = rule.tp > 0.f ? ceil_share(rule.tp, top) : 1ull;
#pragma unroll
  for (int q = 0; q < kPer; ++q)
    if (key[q] != 0 && before[q] < target && target <= before[q] + w[q]) {
      sm.ctl.keep = key[q];
      sm.ctl.total = before[q] + w[q];
    }
}

// ceil(p (z + rest)), at least 1, for z and a mass that is known in fp32 only (in units of the largest
// weight; off by 2^-17.4 for its terms' arguments and 2^-17 for a lane's 140 additions, together below
// 2^-16): the least and the largest that it may be.
__device__ __forceinline__ void share_between(float p, unsigned long long z, float rest, int tokens,
                                              unsigned long long* lo, unsigned long long* hi) {
  if (!(p > 0.f)) {
    *lo = *hi = 1ull;
    return;
  }
  if (!(rest > 0.f)) {
    *lo = *hi = ceil_share(p, z);
    return;
  }
  const unsigned long long r = static_cast<unsigned long long>(rest * 17592186044416.f);
  const unsigned long long off = (r >> 16) + static_cast<unsigned long long>(tokens);
  *lo = ceil_share(p, z + (r > off ? r - off : 0ull));
  *hi = ceil_share(p, z + r + off);
}

// The cuts of a row by classes of its weights -> whether they are made: the key that
// the kept tokens reach in *keep (on entry what they reach at least), their mass in
// ctl.total.  With `rest` the tokens below the source's floor are part of what
// top-p's share is of, and the cut may stay open.
template <typename S>
__device__ __noinline__ bool class_cut(const S& given, const Weights& its_wp, const Rule& its_rule, bool rest,
                                       unsigned long long* keep_io) {
  const S src(given);
  const Weights wp(its_wp);
  const Rule rule(its_rule);
  auto& sm = src.sm;
  const CalledWeights called(wp);
  unsigned long long keep = *keep_io;
  const int tid = threadIdx.x, lane = tid & 31;
  float skipped = 0.f;
  auto fill = [&]() {
    clear_classes(sm);
    __syncthreads();
    skipped = src.scan(wp, rest, [&](float x, int i) {
      if (key50(x, i) < keep) return;
      const unsigned long long w = called.weight44(x);
      if (w == 0) return;
      const int b = bin_of(wp, x);
      atomicAdd(&sm.count[b], 1u);
      add_mass(sm, b, w);
    });
  };
  fill();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) skipped += __shfl_xor_sync(kFullMask, skipped, o);
  if (lane == 0) src.ls.list[src.gw] = __float_as_uint(skipped);
  cluster_sync();
  unsigned count = 0;
  unsigned long long Z = 0;
  Ctl& ctl = src.ls.ctl;
  if (src.lead) {
    all_classes(src, &count, &Z);
    if (tid == 0) {
      ctl.warp = rule.use_k && count > static_cast<unsigned>(rule.k);
      ctl.total = Z;
    }
  }
  cluster_sync();
  bool open = false;
  for (int by_mass = ctl.warp ? 0 : 1; by_mass < (rule.use_p ? 2 : 1); ++by_mass) {
    unsigned long long target = static_cast<unsigned long long>(rule.k), hi = 0;
    if (by_mass) {
      target = 1;
      if (src.lead) {
        float sum = 0.f;
        if (rest) {
          for (int w = lane; w < src.cl * S::Mem::kWarps; w += 32)
            sum += __uint_as_float(static_cast<unsigned>(sm.list[w]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
        }
        share_between(rule.tp, Z, sum, src.row.V, &target, &hi);
        // (behind the floor: any place, it does not count)
        open = target > Z;
        if (open) target = Z;
      }
    }
    unsigned long long upto = 0;
    const bool refined = cut(src, called, !by_mass, target, keep, &upto);
    Z = upto;
    open = open || (by_mass && hi > Z);
    if (refined && !by_mass && rule.use_p) {
      fill();
      cluster_sync();
    }
  }
  if (src.lead && tid == 0) {
    ctl.total = Z;
    ctl.done = open ? 0 : 1;
  }
  cluster_sync();
  *keep_io = keep;
  return ctl.done != 0;
}

// A bit per token of a bf16 unit whose logit is both halves of v, in index order.
[[maybe_unused]] __device__ __forceinline__ unsigned tie_bits(uint4 u, __nv_bfloat162 v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  unsigned bits = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const unsigned m = __heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), v);
    bits |= (m & (1u << 2 * k)) | (m >> 16 & (2u << 2 * k));
  }
  return bits;
}

// The key of the want-th token, in index order, whose bf16 logit is v (not zero): the
// warps' numbers of them, then the warp in whose share it lies.  Written to ctl.keep;
// a barrier of the cluster has to follow.
template <typename S>
__device__ __noinline__ void nth_tie(const S& given, float v, unsigned want) {
  const S src(given);
  auto& sm = src.sm;
  const auto& row = src.row;
  const int lane = threadIdx.x & 31, rest = row.index(row.units);
  const unsigned before_lane = (1u << lane) - 1u;
  const __nv_bfloat162 vv = __float2bfloat162_rn(v);
  const bool head = src.first && lane < row.head && logit<uint16_t>(row.src, lane) == v;
  const bool tail = src.last && lane < row.V - rest && logit<uint16_t>(row.src, rest + lane) == v;
  const unsigned heads = __ballot_sync(kFullMask, head), tails = __ballot_sync(kFullMask, tail);
  constexpr int kAhead = 4;
  unsigned mine = 0;
#pragma unroll 1
  for (int a = src.ub + lane; a < src.ue; a += 32 * kAhead) {
    uint4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (a + 32 * k < src.ue) u[k] = row.load(a + 32 * k);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (a + 32 * k < src.ue) mine += __popc(tie_bits(u[k], vv));
  }
  mine = __reduce_add_sync(kFullMask, mine) + __popc(heads) + __popc(tails);
  if (lane < src.cl) at_rank(&sm, lane)->list[src.gw] = mine;
  cluster_sync();
  unsigned before = 0;
  for (int w = lane; w < src.gw; w += 32) before += static_cast<unsigned>(sm.list[w]);
  before = __reduce_add_sync(kFullMask, before);
  if (want <= before || want > before + mine) return;
  unsigned left = want - before;  // of the warp's own
  auto emit = [&](int i) { src.ls.ctl.keep = key50(v, i); };
  if (left <= static_cast<unsigned>(__popc(heads))) {
    if (head && __popc(heads & before_lane) == left - 1) emit(lane);
    return;
  }
  left -= __popc(heads);
  auto load = [&](int q) { return q < src.ue ? row.load(q) : make_uint4(0, 0, 0, 0); };
  uint4 next = load(src.ub + lane);
#pragma unroll 1
  for (int b = src.ub + lane; b - lane < src.ue; b += 32) {
    unsigned bits = b < src.ue ? tie_bits(next, vv) : 0u;
    next = load(b + 32);
    const unsigned n = __popc(bits);
    unsigned upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += x;
    }
    const unsigned all = __shfl_sync(kFullMask, upto, 31);
    if (left <= all) {
      if (upto - n < left && left <= upto) {
        for (unsigned k = left - (upto - n); k > 1; --k) bits &= bits - 1;
        emit(row.index(b) + __ffs(bits) - 1);
      }
      return;
    }
    left -= all;
  }
  if (tail && __popc(tails & before_lane) == left - 1) emit(rest + lane);
}

// The cuts of a row -> the key that the kept tokens reach (0: all are), their mass
// in *mass (0: not known).  sum: the row's sum in fp32; half: which slots have the
// warps' largest logits.
template <typename S>
__device__ __noinline__ unsigned long long cut_row(const S& given, const Weights& its_wp, const Rule& its_rule, float lane_top,
                                                   float sum, int half, unsigned long long* mass) {
  const S src(given);
  const Weights wp(its_wp);
  const Rule rule(its_rule);
  using E = typename S::Elem;
  using Mem = typename S::Mem;
  Mem &sm = src.sm, &ls = src.ls;
  const int tid = threadIdx.x;
  const CalledWeights called(wp);
  const unsigned long long least = rule.mp > 0.f ? min_p_key(called, rule.mp) : 0;
  if (!rule.use_k && !rule.use_p) return least;
  const float least_x = least ? key50_value(least) : -INFINITY;
  unsigned long long keep = least;
  bool done = false;
  if (rule.use_k && rule.k <= kFew / 2) {  // few: by a list of those above the k-th's floor
    const float floor = fmaxf(least_x, kth_floor(S(src), Weights(wp), rule.k, lane_top, half));
    FloorSource<E, Mem>(src, floor).each_value([&](float x, int i) {
      const unsigned at = atomicAdd(&ls.list_n, 1u);
      if (at < kFew) ls.list[at] = key50(x, i);
    });
    cluster_sync();
    const int n = static_cast<int>(ls.list_n);
    done = n <= kFew;
    if (done && src.lead) list_cut(S(src), Weights(wp), Rule(rule), least, n);
    cluster_sync();
    if (src.lead && tid == 0) sm.list_n = 0;  // (the next to add to it comes behind another barrier)
    if (done) keep = ls.ctl.keep;
  }
  if constexpr (sizeof(E) == 2) {
    const Codes code(wp.top);
    if (!done && isfinite(wp.top) && code.sound()) {
      done = least ? code_cut<true>(src, called, rule, code, least_x) : code_cut(src, called, rule, code);
      const int bin = ls.ctl.bin;
      const unsigned want = static_cast<unsigned>(ls.ctl.left), ties = static_cast<unsigned>(ls.ctl.last);
      if (done && bin >= 0) {
        const float v = code.value(bin);
        keep = static_cast<unsigned long long>(float_order(v + 0.f)) << kIdxBits;
        if (want < ties) {  // the first of them in index order
          // (few: by a list, a barrier less, 3 to 5 us at 150 thousand tokens)
          if (ties <= kFew) {
            FloorSource<E, Mem>(src, v).each_value([&](float x, int i) {
              if (x == v) ls.list[atomicAdd(&ls.list_n, 1u)] = key50(x, i);
            });
            cluster_sync();
            if (src.lead) {
              for (unsigned i = tid; i < ties; i += Mem::kThreads) {
                const unsigned long long mine = sm.list[i];
                unsigned above = 0;
#pragma unroll 4
                for (unsigned j = 0; j < ties; ++j) above += sm.list[j] > mine;
                if (above == want - 1) sm.ctl.keep = mine;
              }
              if (tid == 0) sm.list_n = 0;
            }
          } else {
            nth_tie(S(src), v, want);
          }
          cluster_sync();
          keep = ls.ctl.keep;
        }
      }
    }
  }
  // By classes, fp32's: of the tokens above a floor where one is known.  k-th's; for
  // top-p alone, of all V tokens those that weigh less than half of (1 - p) / V of the
  // whole are together less than what it leaves out
  float floor = least_x;
  bool rest = false;
  if (!done) {
    keep = least;
    if (rule.use_k && rule.k <= 1024) {
      cluster_sync();  // (ctl may be written again)
      floor = fmaxf(floor, kth_floor(S(src), Weights(wp), rule.k, lane_top, half));
      // (what lies below it is out, also where k tokens are left)
      if (floor > -INFINITY) keep = max(keep, static_cast<unsigned long long>(float_order(floor + 0.f)) << kIdxBits);
    } else if (!rule.use_k && least == 0 && rule.tp > 0.f) {
      const float y = __log2f(0.5f * (1.f - rule.tp) * sum / static_cast<float>(src.row.V));
      rest = y > kZeroBelow && isfinite(wp.top + y / wp.ch);
      if (rest) floor = wp.top + y / wp.ch;
    }
  }
  for (int round = 0; round < 2 && !done; ++round) {
    cluster_sync();  // (ctl and the classes' memory may be written again)
    unsigned long long kept = keep;
    done = class_cut(FloorSource<E, Mem>(src, floor), Weights(wp), Rule(rule), rest, &kept);
    keep = done ? kept : least;
    floor = -INFINITY;
    rest = false;
  }
  *mass = ls.ctl.total;
  cluster_sync();
  return keep;
}

// A node's rows and what the cluster's threads know of them.  The seldom steps are
// calls, with a copy of it: an object whose address a call is given lies in memory, and
// 512 threads' of them do not stay in L1.
template <typename E, typename F>
struct Node {
  VerifySmem& sm;
  TreeSmem tree;
  Weights wp, wq;
  Row<E> row;            // the target's
  const F* qrow;
  int ub, ue;            // the warp's units
  int gw, gn, cl;        // the warp in the cluster, its warps, its CTAs
  int par;               // which half of the exchange is next
  unsigned long long keep;  // kept are the tokens whose key reaches it,
  float keep_x;             // its logit
  float sum_p, sum_q;       // the rows' sums in units of their largest weights, about
  unsigned long long total_p, total_q;  // in whole numbers, once they are known
  bool tables;           // the codes' weights are in shared memory
  bool exact;            // sm.ex counts
  int tried;             // rejected children

  __device__ __forceinline__ bool kept(float x, int i) const { return x > keep_x || (x == keep_x && key50(x, i) >= keep); }
  __device__ __forceinline__ float near_p() const { return total_p ? __ull2float_rn(total_p) * 0x1p-44f : sum_p; }
  __device__ __forceinline__ float near_q() const { return total_q ? __ull2float_rn(total_q) * 0x1p-44f : sum_q; }
  // log2 of A sum_p / sum_q: what q's weights are multiplied by next to p's
  __device__ __forceinline__ float log2_c(float A) const {
    return A > 0.f ? __log2f(A) + __log2f(near_p()) - __log2f(near_q()) : -INFINITY;
  }

  // f(p's logit, q's, index, place in its unit) for the warp's tokens
  template <bool kQ, typename G>
  __device__ __forceinline__ void each_pair(G f) const {
    constexpr int kPer = Row<E>::kPer;
    const int lane = threadIdx.x & 31;
    const bool wide = (reinterpret_cast<uintptr_t>(qrow + row.head) & (sizeof(F) < sizeof(E) ? 7 : 15)) == 0;
    auto one = [&](int i) { f(logit<E>(row.src, i), kQ ? logit<F>(qrow, i) : -INFINITY, i, 0); };
    if (gw == 0 && lane < row.head) one(lane);
    const int rest = row.index(row.units);
    if (gw == gn - 1 && lane < row.V - rest) one(rest + lane);
    // (the next unit on its way while one is taken)
    uint4 v = make_uint4(0, 0, 0, 0);
    float y[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) y[k] = -INFINITY;
    int a = ub + lane;
    if (a < ue) {
      v = row.load(a);
      if constexpr (kQ) load_logits<F, kPer>(qrow, row.index(a), wide, y);
    }
#pragma unroll 1
    while (a < ue) {
      const int i = row.index(a);
      float x[kPer], z[kPer];
      unpack<E>(v, x);
#pragma unroll
      for (int k = 0; k < kPer; ++k) z[k] = y[k];
      a += 32;
      if (a < ue) {
        v = row.load(a);
        if constexpr (kQ) load_logits<F, kPer>(qrow, row.index(a), wide, y);
      }
#pragma unroll
      for (int k = 0; k < kPer; ++k) f(fmaxf(x[k], -INFINITY), z[k], i + k, k);
    }
  }

  // sum max(p - A q, 0) in fp32, in units of p's largest weight (four sums a lane)
  __device__ __forceinline__ float near_pass(float A) {
    const int lane = threadIdx.x & 31;
    float part[4] = {0.f, 0.f, 0.f, 0.f};
    if (A > 0.f) {
      const float lc = log2_c(A);
      each_pair<true>([&](float x, float y, int i, int k) {
        const float a = wp.log2w(x), b = wq.log2w(y) + lc;
        if (kept(x, i)) part[k & 3] += fmaxf(ex2(a) - ex2(b), 0.f);
      });
    } else {
      each_pair<false>([&](float x, float, int i, int k) {
        if (kept(x, i)) part[k & 3] += ex2(wp.log2w(x));
      });
    }
    float sum = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    if (lane < cl) at_rank(&sm, lane)->slot[par][gw].stats = make_float4(sum, 0.f, 0.f, 0.f);
    cluster_sync();
    sum = 0.f;
    for (int w = lane; w < gn; w += 32) sum += sm.slot[par][w].stats.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    par ^= 1;
    return __shfl_sync(kFullMask, sum, 0);
  }

  // Whether top-p alone certainly keeps token xi (logit xp) with a share of at least
  // `need` of what is kept: by the mass before it, which has to be below p of the
  // whole, and the kept mass, p of the whole and less than the last kept token's more.
  // That one weighs no more than xi, and less than a 16th or a 256th of it where the
  // tokens that weigh as much are less than p together.
  __device__ __forceinline__ bool surely_kept(float xp, int xi, float top_p, float need) {
    const int lane = threadIdx.x & 31;
    const float yx = wp.log2w(xp);
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
    each_pair<false>([&](float x, float, int i, int) {
      const float y = wp.log2w(x), w = ex2(y);
      s0 += x > xp || (x == xp && i < xi) ? w : 0.f;
      s1 += y >= yx - 4.f ? w : 0.f;
      s2 += y >= yx - 8.f ? w : 0.f;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(kFullMask, s0, o);
      s1 += __shfl_xor_sync(kFullMask, s1, o);
      s2 += __shfl_xor_sync(kFullMask, s2, o);
    }
    if (lane < cl) at_rank(&sm, lane)->slot[par][gw].stats = make_float4(s0, s1, s2, 0.f);
    cluster_sync();
    s0 = s1 = s2 = 0.f;
    for (int w = lane; w < gn; w += 32) {
      const float4 x = sm.slot[par][w].stats;
      s0 += x.x;
      s1 += x.y;
      s2 += x.z;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s0 += __shfl_xor_sync(kFullMask, s0, o);
      s1 += __shfl_xor_sync(kFullMask, s1, o);
      s2 += __shfl_xor_sync(kFullMask, s2, o);
    }
    par ^= 1;
    // (512 additions a lane, 2^-15, and the arguments: below 2 kSumError)
    constexpr float kLow = 1.f - 4.f * kSumError, kHigh = 1.f + 4.f * kSumError;
    const float target = top_p * sum_p, below = target * kLow, w = ex2(yx);
    const float last = s2 < below ? w * (1.f / 256.f) : s1 < below ? w * (1.f / 16.f) : w;
    const bool sure = s0 < below && w * kLow > need * kHigh * (target * kHigh + last);
    return __shfl_sync(kFullMask, static_cast<int>(sure), 0) != 0;
  }

  // The kept tokens' sum.
  __device__ __forceinline__ float near_kept() {
    Node n = *this;
    const float sum = kept_call(&n);
    par = n.par;
    return sum;
  }
  static __device__ __noinline__ float kept_call(Node* n) { return n->near_pass(0.f); }

  template <int kMost, bool kExactBorder = false>
  __device__ __forceinline__ void sum_up(const float (&lc)[kLevels], Sums& t) {
    const int lane = threadIdx.x & 31;
    const Weigh<E, Weights> weigh_p(wp, sm.table_p);
    const Weigh<F, Weights> weigh_q(wq, sm.table_q);
    t = Sums{};
    float near = 0.f;
    each_pair<(kMost > 0)>([&](float x, float y, int i, int) {
      const unsigned long long v = kept(x, i) ? weigh_p(x) : 0ull;
      t.p += v;
      if constexpr (kMost > 0) {
        const unsigned long long w = weigh_q(y);
        t.q += w;
        const float gap = v ? wp.log2w(x) - wq.log2w(y) : -INFINITY;
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
          const float by = gap - lc[k];
          bool over = by > 0.f;
          if (fabsf(by) < kBorder) {
            if constexpr (kExactBorder) over = Scale{sm.ex.scale_m, sm.ex.scale_s}.of(w, v) < v;
            else near += __ull2float_rn(v);
          }
          if (over) {
            t.over_p[k] += v;
            t.over_q[k] += w;
          }
        }
      }
    });
    auto reduce = [&]() {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t.p += __shfl_xor_sync(kFullMask, t.p, o);
        if constexpr (kMost > 0) t.q += __shfl_xor_sync(kFullMask, t.q, o);
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
          t.over_p[k] += __shfl_xor_sync(kFullMask, t.over_p[k], o);
          t.over_q[k] += __shfl_xor_sync(kFullMask, t.over_q[k], o);
        }
      }
    };
    reduce();
    if (kMost == 0) t.over_p[0] = t.p;
    if (kMost > 0 && !kExactBorder && __any_sync(kFullMask, near > 0.f)) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) near += __shfl_xor_sync(kFullMask, near, o);
      // (a whole number: the same in every CTA, in whatever order the warps come)
      const unsigned long long mine = __float2ull_rn(__shfl_sync(kFullMask, near, 0));
      if (lane < cl) atomicAdd(&at_rank(&sm, lane)->near[par], mine);
    }
    if (lane < cl) {
      Sums& to = at_rank(&sm, lane)->slot[par][gw].sums;
      to.p = t.p;
      to.q = t.q;
#pragma unroll
      for (int k = 0; k < (kMost ? kMost : 1); ++k) {
        to.over_p[k] = t.over_p[k];
        to.over_q[k] = t.over_q[k];
      }
    }
    cluster_sync();
    if (threadIdx.x < 32) {
      t = Sums{};
      for (int w = lane; w < gn; w += 32) {
        const Sums& x = sm.slot[par][w].sums;
        t.p += x.p;
        t.q += x.q;
#pragma unroll
        for (int k = 0; k < kMost; ++k) {
          t.over_p[k] += x.over_p[k];
          t.over_q[k] += x.over_q[k];
        }
      }
      reduce();
    }
  }

  // The sums in whole numbers.  levels 0: p's alone; above: for the rejected
  // children from `done` on (or, behind all of them, only the rows' totals), whose As
  // in reject_a tell the tokens' sides.  Where one of them or the rows' sums turn out
  // too far off, or the tokens at the border too many, it is settled with the next
  // pass (kExactBorder: one level, whose scale is known).  The warps' sums are left in
  // slot[par ^ 1].
  template <bool kExactBorder = false>
  __device__ __forceinline__ void exact_pass(int levels, int done) {
    const int lane = threadIdx.x & 31;
    if (!tables && sizeof(E) + sizeof(F) < 8) {
      const Codes cp(wp.top), cq(wq.top);
      const CalledWeights called_p(wp), called_q(wq);
#pragma unroll 1
      for (int j = threadIdx.x; j < 2 * kTable; j += kThr) {
        if (sizeof(E) == 2) sm.table_p[j] = cp.weight(called_p, j);
        if (sizeof(F) == 2) sm.table_q[j] = wq.top > -INFINITY ? cq.weight(called_q, j) : 0ull;
      }
      __syncthreads();
      tables = true;
    }
    const int m = min(levels, tried - done);
    float lc[kLevels];
#pragma unroll
    for (int k = 0; k < kLevels; ++k) lc[k] = k < m ? log2_c(tree.reject_a()[done + k]) : INFINITY;
    Sums t;
    if constexpr (kExactBorder) sum_up<1, true>(lc, t);
    else if (levels == 0) sum_up<0>(lc, t);
    else if (levels == 1) sum_up<1>(lc, t);
    else sum_up<kLevels>(lc, t);
    par ^= 1;
    if (threadIdx.x < 32) {
      int at = 0;
      bool border = false;
      if (m > 0) {
        const unsigned long long weight = lane < m ? CalledWeights(wq).weight44(tree.reject_q()[done + lane]) : 0ull;
        const double inv_np = 1. / static_cast<double>(t.p), inv_nq = 1. / static_cast<double>(t.q);
        double a = sm.ex.A, n = sm.ex.N, z = sm.ex.Z;
        unsigned long long gone = sm.ex.gone;
        // (the sums that the sides were told by: exact ones from the next pass on)
        const float p44 = __ull2float_rn(t.p), q44 = __ull2float_rn(t.q), near = __ull2float_rn(sm.near[par ^ 1]);
        const bool sound = fabsf(near_p() * 0x1p44f - p44) <= 0x1p-18f * p44 && fabsf(near_q() * 0x1p44f - q44) <= 0x1p-18f * q44;
#pragma unroll
        for (int k = 0; k < kLevels; ++k) {
          if (k >= m || at < k || !sound || border) continue;
          const double next_a = a == 0. ? 1. : z > 0. ? a + n / z : a;
          if (fabs(next_a - static_cast<double>(tree.reject_a()[done + k])) > 0x1p-17 * next_a) {
            __syncwarp();
            if (lane == 0) tree.reject_a()[done + k] = static_cast<float>(next_a);
            continue;
          }
          const double next_n = static_cast<double>(t.over_p[k]) * inv_np - next_a * (static_cast<double>(t.over_q[k]) * inv_nq);
          // (a token on the wrong side takes less than 2^-14 of its p from the sum: more than 2^-25 of it all?)
          if (!kExactBorder && near > 0x1p-11f * static_cast<float>(next_n) * p44) {
            border = true;
            const Scale c = Scale::from(next_a * static_cast<double>(t.p) * inv_nq);
            if (lane == 0) {
              sm.ex.scale_m = c.m;
              sm.ex.scale_s = c.s;
            }
            continue;
          }
          a = next_a;
          gone += __shfl_sync(kFullMask, weight, k);
          z = t.q > gone ? static_cast<double>(t.q - gone) * inv_nq : 0.;
          n = next_n > 0x1p-40 ? next_n : 0.;  // (below: nothing but rounding)
          at = k + 1;
        }
        __syncwarp();
        if (lane == 0) {
          sm.near[par ^ 1] = 0;
          sm.ex.A = a;
          sm.ex.N = n;
          sm.ex.Z = z;
          sm.ex.gone = gone;
          sm.ex.settled = done + at;
        }
      }
      if (lane == 0) {
        sm.ex.level = levels == 0 ? 0 : at - 1;
        sm.ex.border = border;
        sm.ex.p = t.p;
        sm.ex.q = t.q;
      }
    }
    __syncthreads();
    total_p = sm.ex.p;
    if (levels > 0) total_q = sm.ex.q;
  }

  __device__ __forceinline__ void begin_exact() {
    if (exact) return;
    if (threadIdx.x == 0) {
      sm.ex.A = 0.;
      sm.ex.N = sm.ex.Z = 1.;
      sm.ex.gone = 0;
      sm.ex.settled = 0;
      sm.ex.level = -1;
      sm.ex.border = 0;
    }
    __syncthreads();
    exact = true;
  }

  // sm.ex behind all rejected children (seldom before the draw).
  __device__ __forceinline__ void settle() {
    Node n = *this;
    settle_call(&n);
    par = n.par;
    total_p = n.total_p;
    total_q = n.total_q;
    tables = n.tables;
    exact = n.exact;
  }
  static __device__ __noinline__ void settle_call(Node* n) {
    bool totals = !n->exact && n->tried == 0;
    n->begin_exact();
    for (int done = n->sm.ex.settled; done < n->tried || totals; done = n->sm.ex.settled) {
      if (n->sm.ex.border) n->template exact_pass<true>(1, done);
      else n->exact_pass(n->tried - done > 1 ? kLevels : 1, done);
      totals = false;
    }
  }

  // A test in whole numbers: child `tried`'s logits, p's only if it is kept.
  __device__ __forceinline__ void exact_test(float xp, float xq, bool in, float u) const {
    const Node n = *this;
    test_call(&n, xp, xq, in, u);
  }
  static __device__ __noinline__ void test_call(const Node* n, float xp, float xq, bool in, float u) {
    n->test(xp, xq, in, u);
  }
  __device__ __forceinline__ void test(float xp, float xq, bool in, float u) const {
    __syncthreads();  // (the test before has been read)
    if (threadIdx.x < 32) {
      const double np = static_cast<double>(total_p), nq = static_cast<double>(total_q), z = sm.ex.Z;
      const double q = static_cast<double>(CalledWeights(wq).weight44(xq)) / nq;
      const double p = in ? static_cast<double>(CalledWeights(wp).weight44(xp)) / np : 0.;
      const bool left = z > 0.;  // (nothing left of q but what the children before it had)
      const double a = left ? sm.ex.N / z : 0.;
      const bool ok = left && static_cast<double>(u) * a * q < p - sm.ex.A * q;
      if (threadIdx.x == 0) {
        sm.ex.yes = ok;
        sm.ex.drawn = left;
        tree.reject_a()[tried] = static_cast<float>(sm.ex.A + a);
      }
    }
    __syncthreads();
  }
};

template <typename E, typename F>
__global__ void __launch_bounds__(kThr, 1) k_verify(const VerifyParams p) {
  using Mem = VerifySmem;
  constexpr int kWarps = Mem::kWarps;
  extern __shared__ __align__(16) uint8_t raw[];
  Mem& sm = *reinterpret_cast<Mem*>(raw);
  const TreeSmem tree(raw + sizeof(Mem), p.B);
  pdl_wait();
  pdl_trigger();
  unsigned cl_u, rank_u;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl_u));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_u));
  const int cl = static_cast<int>(cl_u), rank = static_cast<int>(rank_u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.x / cl;
  const int gw = rank * kWarps + warp, gn = cl * kWarps;
  Mem& ls = *at_rank(&sm, 0);
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
  for (int i = tid; i < (1 << kExpBits); i += kThr)
    sm.exp[i] = make_float2(__ldg(g_exp.v + 2 * i), __ldg(g_exp.v + 2 * i + 1));
  if (tid == 0) sm.cls_n = sm.list_n = 0, sm.near[0] = sm.near[1] = 0;
  const int n = max(0, min(p.n_out[r], p.B));
  for (int i = tid; i < n; i += kThr) {
    tree.parent()[i] = p.parent ? p.parent[static_cast<size_t>(r) * p.B + i] : i - 1;
    tree.token()[i] = p.token[static_cast<size_t>(r) * p.B + i];
  }
  for (int i = tid; i <= n; i += kThr) tree.u()[i] = p.u[static_cast<size_t>(r) * (p.B + 1) + i];
  int par = 0, cur = 0, len = 0;
  cluster_sync();  // (every CTA's memory is there)

  for (;;) {
    const E* prow = static_cast<const E*>(p.logits) + static_cast<size_t>(r) * p.req_stride +
                    static_cast<size_t>(cur) * p.row_stride;
    const F* qrow = static_cast<const F*>(p.draft) + static_cast<size_t>(r) * p.draft_req_stride +
                    static_cast<size_t>(cur) * p.draft_row_stride;
    // ---- the node's children in order
    int kids = 0;
    if (cur < p.draft_rows)  // (else no draft distribution: nothing was drawn there)
      for (int b = cur; b < n; b += kThr) {
        const int i = b + tid;
        const bool mine = i < n && tree.parent()[i] == cur - 1;
        const unsigned in = __ballot_sync(kFullMask, mine);
        if (lane == 0) sm.kid_count[warp] = __popc(in);
        __syncthreads();
        int at = kids;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) at += sm.kid_count[w];
          kids += sm.kid_count[w];
        }
        if (mine) tree.kids()[at + __popc(in & ((1u << lane) - 1u))] = i;
        __syncthreads();
      }
    // a thread per child: its logits (on their way during the pass below)
    auto kid_logits = [&](int k, float* lp, float* lq) {
      const int x = tree.token()[tree.kids()[k]];
      *lp = *lq = -INFINITY;
      if (x >= 0 && x < p.V) {
        *lp = logit<E>(prow, x);
        *lq = logit<F>(qrow, x);
      }
    };
    float lp, lq;
    if (tid < kids) kid_logits(tid, &lp, &lq);

    // ---- the rows' largest logits and sums
    const Row<E> row(prow, p.V);
    const int share = (row.units + gn - 1) / gn;
    const int ub = min(row.units, gw * share), ue = min(row.units, ub + share);
    float top_p, sum_p, lane_top, top_q = -INFINITY, sum_q = 0.f;
    {
      row_stats<E>(row, ub, ue, gw == 0, gw == gn - 1, wp.ch, top_p, sum_p);
      lane_top = top_p;
      if (kids > 0 && !greedy) {
        const Row<F> qr(qrow, p.V);
        const int qs = (qr.units + gn - 1) / gn, qb = min(qr.units, gw * qs), qe = min(qr.units, qb + qs);
        row_stats<F>(qr, qb, qe, gw == 0, gw == gn - 1, wq.ch, top_q, sum_q);
      }
      warp_stats(top_p, sum_p, top_q, sum_q, wp.ch, wq.ch);
      if (lane < cl) at_rank(&sm, lane)->slot[par][gw].stats = make_float4(top_p, sum_p, top_q, sum_q);
      for (int k = tid; k < kids; k += kThr) {
        if (k != tid) kid_logits(k, &lp, &lq);
        // (of several with one token the first counts)
        const int x = tree.token()[tree.kids()[k]];
        bool twice = false;
        for (int j = 0; j < k; ++j) twice |= tree.token()[tree.kids()[j]] == x;
        tree.kid_p()[k] = lp;
        tree.kid_q()[k] = twice ? -INFINITY : lq;
      }
      cluster_sync();
      top_p = top_q = -INFINITY;
      sum_p = sum_q = 0.f;
      for (int w = lane; w < gn; w += 32) {
        const float4 x = sm.slot[par][w].stats;
        join_stats(top_p, sum_p, x.x, x.y, wp.ch);
        join_stats(top_q, sum_q, x.z, x.w, wq.ch);
      }
      warp_stats(top_p, sum_p, top_q, sum_q, wp.ch, wq.ch);
      // (what is decided has to be the same in all threads, to the last bit)
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
    auto accept = [&](int node) {
      __syncthreads();  // (the children may be written again)
      if (lead && tid == 0 && len < p.max_len) p.accept_nodes[static_cast<size_t>(r) * p.max_len + len] = node;
      ++len;
      cur = node + 1;
    };
    const RowSource<false, E, Mem> src{sm, ls, row, ub, ue, gw == 0, gw == gn - 1, 0, cl, lead, gw, max(share, 1)};
    if (greedy) {  // the lowest index of the largest logit
      unsigned long long best = 0;
      if (__any_sync(kFullMask, lane_top == top_p))
        src.each_value([&](float x, int i) {
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
        if (tree.token()[tree.kids()[k]] == x) next = tree.kids()[k];
      if (next < 0) {
        if (lead && tid == 0) {
          p.bonus[r] = x;
          p.prob[r] = 1.f;
        }
        break;
      }
      accept(next);
      continue;
    }

    Node<E, F> node{sm, tree, wp, wq, row, qrow, ub, ue, gw, gn, cl, par, 0ull, -INFINITY,
                          sum_p, sum_q, 0ull, 0ull, false, false, 0};
    // ---- the cuts (top-p alone: often the first child is accepted whatever it
    // cuts off, at a quarter of its cost)
    if (rule.use_p && !rule.use_k && !(rule.mp > 0.f) && rule.tp > 0.f) {
      // (the first that may have been drawn; one of a weight near zero is left to the tests)
      int k = 0;
      while (k < kids && !(tree.kid_q()[k] > -INFINITY && wq.log2w(tree.kid_q()[k]) >= kZeroBelow)) ++k;
      if (k < kids && wq.log2w(tree.kid_q()[k]) >= kZeroBelow + 2.f && isfinite(sum_p) && isfinite(sum_q) &&
          tree.kid_p()[k] > -INFINITY) {
        const int kid = tree.kids()[k];
        const float need = tree.u()[kid + 1] * ex2(wq.log2w(tree.kid_q()[k])) / sum_q;
        if (node.surely_kept(tree.kid_p()[k], tree.token()[kid], rule.tp, need)) {
          par = node.par;
          accept(kid);
          continue;
        }
      }
    }
    if (rule.use_k || rule.use_p || rule.mp > 0.f) {
      const auto its_src = src;  // (copies, as Node's)
      const Weights its_wp = wp;
      const Rule its_rule = rule;
      unsigned long long mass = 0;
      node.keep = cut_row(its_src, its_wp, its_rule, lane_top, sum_p, par ^ 1, &mass);
      node.total_p = mass;
      node.keep_x = node.keep ? key50_value(node.keep) : -INFINITY;
      if (node.keep && node.total_p == 0) node.sum_p = node.near_kept();  // (min-p alone)
    }

    // ---- the children's tests.  A, N, Z and what they may be off by, in fp32;
    // once node.exact, those of sm.ex count
    float A = 0.f, N = 1.f, Z = 1.f, off_a = 0.f, off_n = 0.f, off_z = 0.f;
    int next = -1;
    const float near_p = node.near_p(), inv_p = 1.f / near_p, inv_q = 1.f / sum_q;
    for (int k = 0; k < kids; ++k) {
      if (node.exact && !(sm.ex.N > 0.)) break;
      const int kid = tree.kids()[k];
      const float xq = tree.kid_q()[k], xp = tree.kid_p()[k], yq = wq.log2w(xq);
      // (it cannot have been drawn)
      if (!(xq > -INFINITY) || !(yq >= kZeroBelow)) continue;
      if (yq < kZeroBelow + 2.f && CalledWeights(wq).weight44(xq) == 0) continue;
      const bool in = node.kept(xp, tree.token()[kid]);
      const float ux = tree.u()[kid + 1], qx = ex2(yq) * inv_q;
      bool yes = false, drawn = true;
      if (!node.exact) {
        const float px = in ? ex2(wp.log2w(xp)) * inv_p : 0.f, a = N / Z;
        const float left = ux * a * qx, right = px - A * qx;
        const float off = qx * (ux * (off_n + a * off_z) / Z + off_a) + kSumError * (px + (A + ux * a) * qx);
        yes = left < right;
        // (not with NaN, infinities, or where q may be used up)
        if (!(fabsf(left - right) > 2.f * off && Z > 4.f * off_z)) node.settle();
      }
      if (node.exact) {
        node.exact_test(xp, xq, in, ux);
        yes = sm.ex.yes != 0;
        drawn = sm.ex.drawn != 0;
      }
      if (!drawn) continue;
      if (yes) {
        next = kid;
        break;
      }
      off_a += (off_n + N / Z * off_z) / Z;
      A += N / Z;
      Z -= qx;
      off_z += kSumError * qx;
      if (tid == 0) {
        if (!node.exact) tree.reject_a()[node.tried] = A;
        tree.reject_q()[node.tried] = xq;
      }
      ++node.tried;
      __syncthreads();
      if (node.exact) {
        node.settle();
      } else {
        bool more = false;  // another child to be tested (the draw takes whole numbers)
        for (int j = k + 1; j < kids; ++j) more |= tree.kid_q()[j] > -INFINITY;
        if (!more) break;
        N = node.near_pass(A) * inv_p;
        off_n = kSumError * (1.f + A) + off_a;
        if (!(N > 8.f * off_n)) node.settle();
      }
    }
    if (next >= 0) {
      par = node.par;
      accept(next);
      continue;
    }

    // ---- the draw from max(p - A q, 0), from p where that is nothing
    // (settle(), and p's sums alone where they are to be had)
    bool with_q = node.tried > 0;
    if (with_q) node.begin_exact();
    for (;;) {
      const int done = with_q ? sm.ex.settled : 0, more = with_q ? node.tried - done : 0;
      if (with_q && more == 0) {
        if (sm.ex.N > 0.) break;
        with_q = false;
      }
      node.exact_pass(more > 1 ? kLevels : more, done);
      if (!with_q) break;
      if (sm.ex.border) node.settle();
    }
    // the warp in whose share the running sum passes the mark; behind all of
    // them, the last that has any
    if (warp == 0) {
      const int from = node.par ^ 1, level = sm.ex.level;
      // (in whole numbers: fp64 took 1.5 us more)
      const Scale sc = Scale::from(
          with_q ? sm.ex.A * static_cast<double>(node.total_p) / static_cast<double>(node.total_q) : 0.);
      constexpr int kEach = (kMaxCl * kWarps + 31) / 32;
      unsigned long long mine[kEach], sum = 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int w = lane * kEach + k;
        mine[k] = 0;
        if (w < gn) {
          const Sums& x = sm.slot[from][w].sums;
          mine[k] = x.over_p[level];
          if (with_q) mine[k] -= sc.of(x.over_q[level], mine[k]);
        }
        sum += mine[k];
      }
      unsigned long long inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(kFullMask, inc, o);
        if (lane >= o) inc += y;
      }
      const unsigned long long total = __shfl_sync(kFullMask, inc, 31);
      const float u0 = tree.u()[0];
      const unsigned long long mark = !(u0 > 0.f) ? 0ull : u0 < 1.f ? floor_share(u0, total) : total;
      unsigned long long before = inc - sum, left = 0;
      int owner = -1, last = -1;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        if (owner < 0 && before + mine[k] > mark && mine[k] > 0) {
          owner = lane * kEach + k;
          left = mark - before;  // (of the first lane that has one)
        }
        if (mine[k] > 0) last = lane * kEach + k;
        before += mine[k];
      }
      const unsigned hit = __ballot_sync(kFullMask, owner >= 0);
      if (hit) {
        const int who = __ffs(hit) - 1;
        owner = __shfl_sync(kFullMask, owner, who);
        left = __shfl_sync(kFullMask, left, who);
      } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(kFullMask, last, o));
        owner = max(last, 0);
        left = ~0ull;
      }
      if (lane == 0) {
        sm.ex.owner = owner;
        sm.ex.left = left;
        sm.ex.total = static_cast<double>(total);
        sm.ex.scale_m = sc.m;
        sm.ex.scale_s = sc.s;
      }
    }
    __syncthreads();
    const int owner = sm.ex.owner;
    if (owner / kWarps == rank) {
      // its tokens over the CTA's threads, in pieces in index order
      unsigned long long t = sm.ex.left;
      const CalledWeights called_p(wp), called_q(wq);
      const Weigh<E, CalledWeights> weigh_p(called_p, sm.table_p);
      const Weigh<F, CalledWeights> weigh_q(called_q, sm.table_q);
      const Scale sc{sm.ex.scale_m, sm.ex.scale_s};
      const float lc = with_q ? node.log2_c(static_cast<float>(sm.ex.A)) : 0.f;
      auto residual = [&](int i) -> unsigned long long {
        const float x = logit<E>(prow, i);
        if (!node.kept(x, i)) return 0ull;
        const float y = with_q ? logit<F>(qrow, i) : -INFINITY;
        // (at the border in whole numbers, whatever the pass took it for)
        if (with_q && wp.log2w(x) - wq.log2w(y) < lc - 2.f * kBorder) return 0ull;
        const unsigned long long v = weigh_p(x);
        return with_q ? v - sc.of(weigh_q(y), v) : v;
      };
      const int ob = min(row.units, owner * share), oe = min(row.units, ob + share);
      const int b = owner == 0 ? 0 : row.index(ob), e = owner == gn - 1 ? p.V : row.index(oe);
      const int each = (e - b + kThr - 1) / kThr;
      const int mb = min(e, b + tid * each), me = min(e, mb + each);
      unsigned long long own = 0;
#pragma unroll 1
      for (int i = mb; i < me; ++i) own += residual(i);
      unsigned long long upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(kFullMask, upto, o);
        if (lane >= o) upto += x;
      }
      if (lane == 31) sm.part[warp] = upto;
      __syncthreads();
      unsigned long long all = 0;
      for (int w = 0; w < kWarps; ++w) {
        if (w == warp) upto += all;
        all += sm.part[w];
      }
      // (the share's sum is above 0, so one of its tokens is; the mark may lie behind them by rounding)
      t = min(t, all - 1);
      auto emit = [&](int i, unsigned long long z) {
        p.bonus[r] = i;
        p.prob[r] = static_cast<float>(static_cast<double>(z) / sm.ex.total);
      };
      const unsigned hit = __ballot_sync(kFullMask, upto > t && upto - own <= t);
      if (hit) {  // the thread's piece once more, by the warp
        const int who = __ffs(hit) - 1, pe = __shfl_sync(kFullMask, me, who);
        unsigned long long run = __shfl_sync(kFullMask, upto - own, who);
        bool found = false;
        for (int i0 = __shfl_sync(kFullMask, mb, who); i0 < pe && !found; i0 += 32) {
          const int i = i0 + lane;
          const unsigned long long z = i < pe ? residual(i) : 0ull;
          unsigned long long sum = z;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long x = __shfl_up_sync(kFullMask, sum, o);
            if (lane >= o) sum += x;
          }
          const unsigned at = __ballot_sync(kFullMask, run + sum > t);
          found = at != 0;
          if (found && lane == __ffs(at) - 1) emit(i, z);
          run += __shfl_sync(kFullMask, sum, 31);
        }
      }
    }
    break;
  }
  if (lead) {
    if (tid == 0) p.accept_len[r] = len;
    for (int i = len + tid; i < p.max_len; i += kThr) p.accept_nodes[static_cast<size_t>(r) * p.max_len + i] = -1;
  }
  cluster_sync();  // (no CTA leaves while another reads or writes its memory)
}

}  // namespace

// One object per pair of types (DT_E, DT_F: 0 fp32, 1 bf16), the checks with the first.
template <int kE, int kF>
cudaError_t launch_verify(const VerifyParams& p, int cl, cudaStream_t st);

#if DT_E
using E_ = uint16_t;
#else
using E_ = float;
#endif
#if DT_F
using F_ = uint16_t;
#else
using F_ = float;
#endif

template <>
cudaError_t launch_verify<DT_E, DT_F>(const VerifyParams& p, int cl, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(k_verify<E_, F_>, &done);
  if (e != cudaSuccess) return e;
  const size_t smem = sizeof(VerifySmem) + TreeSmem::kArrays * sizeof(int) * (static_cast<size_t>(p.B) + 1);
  return launch_kernel_cluster(k_verify<E_, F_>, dim3(static_cast<unsigned>(p.R) * cl), dim3(kThr), smem, st, true, cl, p);
}

}  // namespace dt

#if !DT_E && !DT_F

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
  // A request's rows over several CTAs.  15 clusters of 8, 36 of 4 and 76 of 2 find
  // room at once; paths differ in length, so a few more than that still gain (those
  // that wait start long before the longest ends).  Chains of 7 over 151936 bf16
  // logits without cuts (with settings of their own), us: 16 of them by 8 CTAs 82
  // (128), by 4 93 (153); 24 110 (178), 89 (160); 40 by 4 127 (174), by 2 151 (243);
  // 64 168 (238), 152 (283); 100 by 2 216 (296), by 1 264 (487); 150 294 (416), 276
  // (581).
  const int most = R <= 16 ? kMaxCl : R <= 40 ? 4 : R <= 152 ? 2 : 1;
  int cl = 1;
  while (cl < most && V / cl > 4096) cl *= 2;
  const VerifyParams p{parent, token, n_out, logits, draft, req_stride, row_stride, draft_req_stride, draft_row_stride,
                       V, R, B, draft_rows, temperature, top_k, top_p, min_p, draft_temperature, u,
                       max_len, accept_len, accept_nodes, bonus, prob};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bf16 ? (draft_bf16 ? launch_verify<1, 1>(p, cl, st) : launch_verify<1, 0>(p, cl, st))
                             : (draft_bf16 ? launch_verify<0, 1>(p, cl, st) : launch_verify<0, 0>(p, cl, st));
  return cache_launched(e);
}

#endif
