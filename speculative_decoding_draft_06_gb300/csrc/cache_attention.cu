// Attention of single tokens and draft trees over the paged 4-bit cache
// (dartree_cache_attention).
//
// Rows (queries) of a key/value head: q = node * g + query head within the
// group, g = Hq / Hkv.  A CTA takes up to 16 rows of one request and one
// key/value head and a share of its keys (the keys are split over CTAs until
// the GPU is full; a second kernel joins the shares).  Its four warps are
// independent: each takes every fourth 64-key tile of the share, brings the
// tile's codes and scales into its own two stages in shared memory with bulk
// copies (one for a 64-token page), and has a softmax state and an output of
// its own until the end.
//
// Both products are mma m16n8k16 in fp16 with fp32 sums and the keys' side as
// the 16-row operand: S^T = K Q^T (16 keys x 8 rows x 16 dims), O^T += V^T
// P^T (16 dims x 8 rows x 16 keys).  A code times its scale has 6 significant
// bits and lies between 2^-10 and 2688: exact in fp16.  The queries are
// scaled per row by a power of two to at most 2 before they become fp16, so
// all that rounds is fp32 sums, P (2^-12 of a weight, with its reference maximum
// at 2^6 so that weights down to 2^-20 of the largest keep all their bits; the
// normaliser sums them before they are rounded, in fp32) and the output, whose
// rounding to bf16 (2^-9) is the largest.
//
// The k index of a product may run over the dims (or keys) in any order, and
// so may the row index: the orders are chosen so that a lane's codes lie
// together and its loads meet no bank twice.  In S^T, lane (r = lane / 4, c =
// lane % 4) holds the dims [c dh/4, (c + 1) dh/4) of its keys: one 16-byte
// (dh = 128) load each.  Row index i of S^T is key i/2 + 4 (i % 2) of its
// eight; in O^T, rows r and r + 8 of dim tile j are the dims r dh/8 + 2 j and
// + 1: a lane's dims of a key are 8 (4) bytes.  P^T is S^T's accumulator
// transposed within the warp (movmatrix).
//
// Bound by memory where there are many keys: 64 single tokens over 1 to 16001
// tokens, 32 heads over 8 of 128: 144 us, 5.1 TB/s, 77% of a copy's rate; one
// over 131072 tokens 36 us, 4.2 TB/s (the join and the ramp: a warp has 9
// tiles); over 1000 tokens 6.9 us, latency.  Steps:
// a producer warp and rows as the 16-row operand 315 us for the 64; warps with
// rings of their own and keys as that operand 246; four code bytes to a
// conversion 198; stages of 64 keys and no scaling in front 145.
#include <cstdlib>

#include "cache_attn.cuh"

namespace dt {
namespace {

constexpr int kTileKeys = 64;   // keys of a stage
constexpr int kStep = 32;       // keys between two looks at the maximum
constexpr int kStages = 2;
constexpr int kMaxCluster = 8;  // splits that join in a cluster's shared memory
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

__device__ int g_cache_err;  // error word when the caller passes none

// Bits of x where the mask has ones, of y where it has zeros.
__device__ __forceinline__ uint32_t bit_select(uint32_t mask, uint32_t x, uint32_t y) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(mask), "r"(x), "r"(y));
  return d;
}

// Bytes of one tile in shared memory: key codes, key scales, value codes,
// value scales of 64 tokens (a 64-token page's chunk, byte for byte).
template <int DH>
struct Tile {
  static constexpr int kCodes = kTileKeys * DH / 2, kScales = kTileKeys * DH / 16;
  static constexpr int kV = kCodes + kScales;
  static constexpr int kBytes = 2 * kV;
};

template <int DH, int NQ>
struct __align__(128) AttnSmem {
  union {
    uint8_t stage[kWarps][kStages][Tile<DH>::kBytes];
    struct {
      float red[kWarps][8 * NQ][DH + 4];
      float recv[8 * NQ + kMaxCluster][DH + 4];  // a cluster's shares of the rows that this CTA joins
    };
  };
  uint64_t full[kWarps][kStages];
  uint64_t valid[kWarps][kStages];  // bit k: key k of the tile is there
  float2 ml[kWarps][8 * NQ];
  float2 recv_ml[8 * NQ + kMaxCluster];
};

template <int DH, int NQ>
__device__ __forceinline__ void attend_rows(const CacheAttnParams& p) {
  constexpr int kSteps = DH / 16;   // k-steps of S^T, dim tiles of O^T
  constexpr int kRows = 8 * NQ;
  using T = Tile<DH>;
  extern __shared__ __align__(128) uint8_t raw[];
  AttnSmem<DH, NQ>& sm = *reinterpret_cast<AttnSmem<DH, NQ>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, hk = blockIdx.y, r = blockIdx.z;
  Span sp;
  if (!request_span(p, r, &sp)) return;
  // rows q0 .. q0 + live - 1
  int q0 = 0, live = (sp.n + 1) * p.g;
  if (p.tail) {
    q0 = live;
    live = tail_rows(live);
    if (live == 0) return;
    q0 -= live;
  }
  const int t_all = row_tile_keys(p, sp, 0);
  const int t_beg = split * p.split_tiles;
  const int nt = min(t_all, t_beg + p.split_tiles) - t_beg;
  // (one split: rows without keys are written as 0; a cluster's CTAs all stay)
  if (nt <= 0 && !p.cluster && !(split == 0 && p.n_split == 1)) return;
  const int mine = nt > warp ? (nt - warp + kWarps - 1) / kWarps : 0;  // the warp's tiles

  if (lane < kStages) mbar_init(&sm.full[warp][lane], 1);
  fence_mbar_init();
  __syncwarp();
  if (threadIdx.x == 0 && split == 0 && hk == 0 && !p.tail && static_cast<long long>(p.lens[r]) + sp.n > p.max_len)
    atomicOr(p.err, DT_ERR_BAD_INDEX);

  // ---- the warp's copies: lane (piece, segment) has one of a tile's (a
  // piece: min(page, 64) tokens; segments: key codes, key scales, values', or
  // all of a 64-token page at once)
  const int P = 1 << p.c.log_page;
  const int piece = P < kTileKeys ? P : kTileKeys;
  const int pieces = kTileKeys / piece, segs = P == kTileKeys ? 1 : 4;
  const int pc = lane / segs, seg = lane % segs;
  const bool copies = pc < pieces;
  const int32_t* trow = p.table + static_cast<size_t>(r) * p.max_pages;
  const int unit = (seg & 1) ? DH / 16 : DH / 2;  // bytes of a token in the segment
  const uint32_t bytes = static_cast<uint32_t>(segs == 1 ? T::kBytes : piece * unit);
  const int seg_tile = (seg >> 1) * T::kV + ((seg & 1) ? T::kCodes : 0) + (segs == 1 ? 0 : pc * piece * unit);
  const uint8_t* seg_base = p.c.pool + static_cast<size_t>(hk) * p.c.chunk + (seg >> 1) * (p.c.chunk >> 1) +
                            ((seg & 1) ? P * DH / 2 : 0);
  auto first_key = [&](int i) { return (t_beg + warp + i * kWarps) * kTileKeys; };
  auto page_of = [&](int i) {  // the lane's piece's page: -1 none, -2 bad
    const int key = first_key(i) + pc * piece;
    if (i >= mine || !copies || key >= sp.L) return -1;
    const int slot = key >> p.c.log_page;
    const int page = slot < p.max_pages ? trow[slot] : -2;
    return page < 0 || page >= p.c.pages ? -2 : page;
  };
  auto issue = [&](int i, int page) {
    if (i >= mine) return;
    const int st = i % kStages, key0 = first_key(i);
    const unsigned got = __ballot_sync(kFullMask, page >= 0);
    if (page == -2 && seg == 0) atomicOr(p.err, DT_ERR_BAD_INDEX);
    if (lane == 0) {
      uint64_t v = ~0ull;
      if (got != (segs == 1 ? 1u : (pieces == 1 ? 0xFu : pieces == 2 ? 0xFFu : 0xFFFFu))) {
        v = 0;
        for (int k = 0; k < pieces; ++k)
          if ((got >> (segs * k)) & 1u) v |= (piece == 64 ? ~0ull : ((1ull << piece) - 1ull) << (k * piece));
      }
      const int left = sp.L - key0;
      if (left < kTileKeys) v &= (1ull << left) - 1ull;
      sm.valid[warp][st] = v;
      mbar_arrive_expect_tx(&sm.full[warp][st], static_cast<uint32_t>(__popc(got) / segs * piece * (DH / 8 * 9)));
    }
    __syncwarp();
    if (page >= 0) {
      const int tok = (key0 + pc * piece) & (P - 1);
      bulk_load(&sm.stage[warp][st][seg_tile], seg_base + static_cast<size_t>(page) * p.c.page_bytes + tok * unit, bytes,
                &sm.full[warp][st]);
    }
  };
  int page[kStages];
#pragma unroll
  for (int i = 0; i < kStages; ++i) page[i] = page_of(i);
#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i, page[i]);
  int next_page = page_of(kStages);

  // ---- queries: column r of row group n is row 8 n + r, dims [c DH/4, ..)
  const int rr = lane >> 2, c = lane & 3;
  uint32_t qb[NQ][kSteps][2];
  float fac[NQ][2];                 // of rows 8 n + 2 c, + 1
  int node[NQ][2];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const bool on = 8 * n + rr < live;
    const int q = on ? q0 + 8 * n + rr : 0, nd = q / p.g;
    uint32_t w[DH / 8];
    const uint4* src = reinterpret_cast<const uint4*>(
        p.Q + (static_cast<size_t>(r) * (p.B + 1) + nd) * p.q_stride +
        static_cast<size_t>(hk * p.g + (on ? q - nd * p.g : 0)) * DH + c * (DH / 4));
#pragma unroll
    for (int k = 0; k < DH / 32; ++k) {
      const uint4 x = on ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      w[4 * k] = x.x;
      w[4 * k + 1] = x.y;
      w[4 * k + 2] = x.z;
      w[4 * k + 3] = x.w;
    }
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < DH / 8; ++k)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
    top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
    top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
    float down;
    const float f = row_exponent(p, top, &down);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fac[n][i] = __shfl_sync(kFullMask, f, (2 * c + i) * 4);
      node[n][i] = __shfl_sync(kFullMask, nd, (2 * c + i) * 4);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const uint32_t x = w[2 * s], y = w[2 * s + 1];  // dims 4s, 4s+1 | 4s+2, 4s+3 of the lane's
      qb[n][s][0] = pack_f16(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
      qb[n][s][1] = pack_f16(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xFFFF0000u) * down);
    }
  }
  float o[NQ][kSteps][4];           // dim tile j: dims rr DH/8 + 2 j, + 1 of rows 8 n + 2 c, + 1
  float m[NQ][2], l[NQ][2];         // reference maximum (a score, before its factor), sum
  float limit[NQ][2];               // the score above which m rises
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n][0] = m[n][1] = limit[n][0] = limit[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
  }

  // One step of 32 keys: `at` their first in the tile, key0 its position,
  // valid their bits.  kAll: every row sees every key.
  auto step = [&](auto all_seen, const uint8_t* tile, int at, int key0, uint32_t valid) {
    constexpr bool kAll = decltype(all_seen)::value != 0;
    // ---- S^T of the two halves of 16 keys
    float s[2][NQ][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) s[h][n][0] = s[h][n][1] = s[h][n][2] = s[h][n][3] = 0.f;
      uint32_t w[2][DH / 32], sc[2][2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = at + 16 * h + 8 * t + (rr >> 1) + 4 * (rr & 1);
        if constexpr (DH == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + key * 64 + c * 16);
          w[t][0] = x.x;
          w[t][1] = x.y;
          w[t][2] = x.z;
          w[t][3] = x.w;
          const uint32_t two = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(tile + T::kCodes + key * 8 + c * 2));
          sc[t][0] = __byte_perm(two, two, 0x1010);
          sc[t][1] = __byte_perm(two, two, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(tile + key * 32 + c * 8);
          w[t][0] = x.x;
          w[t][1] = x.y;
          const uint32_t b = tile[T::kCodes + key * 4 + c];
          sc[t][0] = sc[t][1] = e4m3x2_to_f16x2(b | (b << 8));
        }
      }
#pragma unroll
      for (int k2 = 0; k2 < kSteps / 2; ++k2) {  // a word: two k-steps
        uint32_t x[2][4];
        e2m1x8_to_f16(w[0][k2], x[0]);
        e2m1x8_to_f16(w[1][k2], x[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a[4] = {h2mul(x[0][2 * k], sc[0][k2 >> 1]), h2mul(x[1][2 * k], sc[1][k2 >> 1]),
                                 h2mul(x[0][2 * k + 1], sc[0][k2 >> 1]), h2mul(x[1][2 * k + 1], sc[1][k2 >> 1])};
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma_f16(s[h][n], a, qb[n][2 * k2 + k][0], qb[n][2 * k2 + k][1]);
        }
      }
    }
    // ---- x = 2 t + i: key 16 h + 8 t + perm(rr), row 8 n + 2 c + i.  The
    // scores stay as they are (a row's factor to base 2 multiplies their
    // distance from the reference); the reference rises where one passes `limit`
    bool up = false;
    float top[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      if constexpr (!kAll) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int i2 = x & 1, kk = 16 * h + 8 * (x >> 1) + (rr >> 1) + 4 * (rr & 1), pos = key0 + kk;
            bool seen = (valid >> kk) & 1u;
            if (seen && pos >= sp.Lp) {
              const int j = pos - sp.Lp;
              seen = node[n][i2] > 0 &&
                     ((__ldg(p.mask + (static_cast<size_t>(r) * p.B + node[n][i2] - 1) * p.words + (j >> 5)) >>
                       (j & 31)) & 1u);
            }
            if (!seen) s[h][n][x] = -INFINITY;
          }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[n][x] = fmaxf(fmaxf(s[0][n][x], s[0][n][x + 2]), fmaxf(s[1][n][x], s[1][n][x + 2]));
        up |= top[n][x] > limit[n][x];
      }
    }
    if (__any_sync(kFullMask, up)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float al[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = top[n][x];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) t = fmaxf(t, __shfl_xor_sync(kFullMask, t, d));
          al[x] = 1.f;
          if (t > limit[n][x]) {
            al[x] = ex2((m[n][x] - t) * fac[n][x]);  // (0 from -inf)
            m[n][x] = t;
            limit[n][x] = rise_limit(t, fac[n][x]);
            l[n][x] *= al[x];
          }
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          o[n][j][0] *= al[0];
          o[n][j][1] *= al[1];
          o[n][j][2] *= al[0];
          o[n][j][3] *= al[1];
        }
      }
    }
    // the weights: 2^((s - m) fac + kBias) (s fac - m fac would be off by 2^-24 of
    // m fac, which from 2^27 on is more than fp16 holds)
    uint32_t pb[2][NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0], m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(fmaf(s[h][n][2 * t] - m0, fac[n][0], kBias));
          const float p1 = ex2(fmaf(s[h][n][2 * t + 1] - m1, fac[n][1], kBias));
          l[n][0] += p0;
          l[n][1] += p1;
          pb[h][n][t] = transpose8x8(pack_f16(p0, p1));
        }
    }
    // ---- O^T += V^T P^T: the lane's keys c, c + 4 (k = 2c, 2c + 1) of each eight
    const uint8_t* vt = tile + T::kV;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t vw[2][2][DH / 64], vs[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t b[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int key = at + 16 * h + 8 * t + c + 4 * x;
          if constexpr (DH == 128) {
            const uint2 y = *reinterpret_cast<const uint2*>(vt + key * 64 + rr * 8);
            vw[t][x][0] = y.x;
            vw[t][x][1] = y.y;
            b[x] = vt[T::kCodes + key * 8 + rr];
          } else {
            vw[t][x][0] = *reinterpret_cast<const uint32_t*>(vt + key * 32 + rr * 4);
            b[x] = vt[T::kCodes + key * 4 + (rr >> 1)];
          }
        }
        vs[t] = e4m3x2_to_f16x2(b[0] | (b[1] << 8));
        if constexpr (!kAll) vs[t] = finite_scales(vs[t]);
      }
#pragma unroll
      for (int w = 0; w < DH / 64; ++w) {
        uint32_t ev[2][4], od[2][4];  // (first key's, second key's) codes of the even, odd dims
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t x = vw[t][0][w], y = vw[t][1][w];
          e2m1x8_to_f16(bit_select(0x0F0F0F0Fu, x, y << 4), ev[t]);
          e2m1x8_to_f16(bit_select(0x0F0F0F0Fu, x >> 4, y), od[t]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a[4] = {h2mul(ev[0][k], vs[0]), h2mul(od[0][k], vs[0]), h2mul(ev[1][k], vs[1]),
                                 h2mul(od[1][k], vs[1])};
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma_f16(o[n][4 * w + k], a, pb[h][n][0], pb[h][n][1]);
        }
      }
    }
  };

  auto landed = [&](uint64_t* bar, uint32_t par) {
    if (p.wait_limit >= kWaitLimitCycles) return mbar_wait(bar, par, p.err);
    const long long t0 = clock64();
    while (!poll<true>(smem_u32(bar), par))
      if (clock64() - t0 > p.wait_limit) {
        atomicOr(p.err, DT_ERR_TIMEOUT);
        return false;
      }
    return true;
  };
  int done = 0;
  for (int i = 0; i < mine; ++i) {
    const int st = i % kStages;
    if (!__all_sync(kFullMask, landed(&sm.full[warp][st], static_cast<uint32_t>((i / kStages) & 1)))) break;
    done = i + 1;
    const uint8_t* tile = sm.stage[warp][st];
    const int key0 = first_key(i);
    const uint64_t valid = sm.valid[warp][st];
    if (valid == ~0ull && key0 + kTileKeys <= sp.Lp) {
#pragma unroll 1
      for (int at = 0; at < kTileKeys; at += kStep) step(IntC<1>{}, tile, at, key0 + at, ~0u);
    } else {
#pragma unroll 1
      for (int at = 0; at < kTileKeys; at += kStep)
        if (static_cast<uint32_t>(valid >> at)) step(IntC<0>{}, tile, at, key0 + at, static_cast<uint32_t>(valid >> at));
    }
    // the stage is free: the tile after the next goes there, and its
    // successor's page is looked up
    __syncwarp();
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    issue(i + kStages, next_page);
    next_page = page_of(i + kStages + 1);
  }
  // (a wait that ran out: every copy must have landed before the block may end)
  for (int i = done; i < min(mine, done + kStages); ++i)
    mbar_wait(&sm.full[warp][i % kStages], static_cast<uint32_t>((i / kStages) & 1), p.err);
  __syncthreads();
  // ---- the warp's rows into shared memory
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[n][x] += __shfl_xor_sync(kFullMask, l[n][x], d);
      const int row = 8 * n + 2 * c + x;
      if (rr == 0) sm.ml[warp][row] = make_float2(m[n][x] * fac[n][x], l[n][x]);
      float* dst = &sm.red[warp][row][rr * (DH / 8)];
#pragma unroll
      for (int j = 0; j < kSteps; j += 2)
        *reinterpret_cast<float4*>(dst + 2 * j) =
            make_float4(o[n][j][x], o[n][j][x + 2], o[n][j + 1][x], o[n][j + 1][x + 2]);
    }
  if (p.cluster) cluster_sync();  // (every CTA's stages are free: the rows may be sent)
  else __syncthreads();
  // ---- the four warps' shares of each row, joined in warp order
  for (int row = warp; row < min(live, kRows); row += kWarps) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.ml[w][row].x);
    float f[kWarps], L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = sm.ml[w][row].x == -INFINITY ? 0.f : ex2(sm.ml[w][row].x - M);
      L += sm.ml[w][row].y * f[w];
    }
    constexpr int kE = DH / 32;  // dims per lane
    float v[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      v[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v[e] += sm.red[w][row][lane * kE + e] * f[w];
    }
    if (p.cluster) {
      // row i is the (i / n)-th that CTA i % n joins
      const int owner = row % p.n_split, at = split * ((kRows + p.n_split - 1) / p.n_split) + row / p.n_split;
      float* dst = at_rank(&sm.recv[at][0], owner);
#pragma unroll
      for (int e = 0; e < kE; ++e) dst[lane * kE + e] = v[e];
      if (lane == 0) *at_rank(&sm.recv_ml[at], owner) = make_float2(M, L);
    } else if (p.n_split > 1) {
      float* dst = cache_part_row(p, r, hk, 0, split, row);
#pragma unroll
      for (int e = 0; e < kE; e += 2)
        *reinterpret_cast<float2*>(dst + kPartHead + lane * kE + e) = make_float2(v[e], v[e + 1]);
      if (lane == 0) *reinterpret_cast<float2*>(dst) = make_float2(M, L);
    } else {
      const float inv = L > 0.f ? p.c.v_scale / L : 0.f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q0 + row) + lane * kE);
#pragma unroll
      for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
    }
  }
  if (!p.cluster) return;
  cluster_sync();
  // ---- the rows this CTA joins, in split order
  const int each = (kRows + p.n_split - 1) / p.n_split;
  for (int row = split + warp * p.n_split; row < min(live, kRows); row += kWarps * p.n_split) {
    const int at = row / p.n_split;
    float M = -INFINITY, L = 0.f;
    for (int k = 0; k < p.n_split; ++k) M = fmaxf(M, sm.recv_ml[k * each + at].x);
    constexpr int kE = DH / 32;
    float v[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = 0.f;
    for (int k = 0; k < p.n_split; ++k) {
      const float2 ml = sm.recv_ml[k * each + at];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] += sm.recv[k * each + at][lane * kE + e] * f;
    }
    const float inv = L > 0.f ? p.c.v_scale / L : 0.f;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q0 + row) + lane * kE);
#pragma unroll
    for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
  }
}

template <int DH, int NQ>
__global__ void __launch_bounds__(kThreads, 3) k_cache_attention(const CacheAttnParams p) {
  if (!p.tail) {
    pdl_wait();
    // (not ahead of a join: its blocks would take the place of these)
    if (p.cluster || p.n_split == 1) pdl_trigger();
  }
  attend_rows<DH, NQ>(p);
  // The rows left over by the tensor-core kernel: launched while that one
  // runs, whose outputs these are not; one CTA sees it complete, so that what
  // follows this launch follows both.
  if (p.tail && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) pdl_wait();
}

template <int DH, int NQ>
cudaError_t launch_rows(const CacheAttnParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(k_cache_attention<DH, NQ>, &done);
  if (e != cudaSuccess) return e;
  const dim3 grid(p.n_split, p.c.Hkv, p.R);
  if (p.cluster)
    return launch_kernel_cluster(k_cache_attention<DH, NQ>, grid, dim3(kThreads), sizeof(AttnSmem<DH, NQ>), st,
                                 true, p.n_split, p);
  return launch_kernel(k_cache_attention<DH, NQ>, grid, dim3(kThreads), sizeof(AttnSmem<DH, NQ>), st, true, p);
}

// The shares of each row over the key splits, joined in a fixed order: M =
// max m_s, O = sum O_s 2^(m_s - M) / sum l_s 2^(m_s - M).  W warps per row
// take every W-th split and meet in shared memory; grid (rows / (8 / W), Hkv,
// R).
template <int DH, int W>
__global__ void __launch_bounds__(256) k_cache_attention_join(const CacheAttnParams p) {
  constexpr int kE = DH / 32, kPerBlock = 8 / W;
  __shared__ float s_v[W > 1 ? 8 : 1][DH];
  __shared__ float2 s_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp % W;
  const int q = blockIdx.x * kPerBlock + warp / W, hk = blockIdx.y, r = blockIdx.z;
  pdl_wait();
  Span sp;
  bool on = request_span(p, r, &sp);
  int q0 = 0;  // the launch's first row
  if (on) {
    const int all = (sp.n + 1) * p.g, tail = p.tile_rows == kTreeRowsCta || p.tail ? tail_rows(all) : 0;
    q0 = p.tail ? all - tail : 0;
    on = q < (p.tail ? tail : all - tail);
  }
  if (W == 1 && !on) return;
  float M = -INFINITY, L = 0.f, v[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) v[e] = 0.f;
  if (on) {
    const int mt = q / p.tile_rows;
    const int ns = (row_tile_keys(p, sp, mt) + p.split_tiles - 1) / p.split_tiles;  // splits that had keys
    const size_t step = static_cast<size_t>(p.tile_rows) * (DH + kPartHead);
    const float* src = cache_part_row(p, r, hk, mt, 0, q - mt * p.tile_rows);
    for (int s = w + lane * W; s < ns; s += 32 * W) M = fmaxf(M, src[s * step]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, x));
#pragma unroll 4
    for (int s = w; s < ns; s += W) {
      const float2 ml = *reinterpret_cast<const float2*>(src + s * step);
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < kE; e += 2) {
        const float2 x = *reinterpret_cast<const float2*>(src + s * step + kPartHead + lane * kE + e);
        v[e] += x.x * f;
        v[e + 1] += x.y * f;
      }
    }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < kE; ++e) s_v[warp][lane * kE + e] = v[e];
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (w != 0 || !on) return;
    float T = M;
#pragma unroll
    for (int k = 1; k < W; ++k) T = fmaxf(T, s_ml[warp + k].x);
    L = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) v[e] = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 ml = s_ml[warp + k];
      const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - T);
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < kE; ++e) v[e] += s_v[warp + k][lane * kE + e] * f;
    }
  }
  const float inv = L > 0.f ? p.c.v_scale / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q0 + q) + lane * kE);
#pragma unroll
  for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
}

template <int DH>
cudaError_t launch_join(const CacheAttnParams& p, cudaStream_t st) {
  // eight warps per row where a row has many shares and few rows would leave
  // the GPU to a handful of blocks
  if (p.n_split > 8 && static_cast<long long>(p.R) * p.c.Hkv * p.rows < 152 * 16)
    return launch_kernel(k_cache_attention_join<DH, 8>, dim3(p.rows, p.c.Hkv, p.R), dim3(256), 0, st, true, p);
  return launch_kernel(k_cache_attention_join<DH, 1>, dim3((p.rows + 7) / 8, p.c.Hkv, p.R), dim3(256), 0, st, true, p);
}

// Zeros in the rows that a call leaves as they were: those behind a request's
// tree, all of a skipped one.  Grid (R).  (Where it is asked for, a launch of
// its own, 0.6 to 3 us: in the attention kernels its code made 32 trees 5% slower.)
__global__ void __launch_bounds__(256) k_cache_zero_rest(const CacheAttnParams p) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  Span sp;
  const int first = request_span(p, r, &sp) ? sp.n + 1 : 0;
  const size_t per = static_cast<size_t>(p.Hq) * p.c.dh / 8;  // 16-byte units of a node
  uint4* o = reinterpret_cast<uint4*>(p.O) + static_cast<size_t>(r) * (p.B + 1) * per;
  for (size_t i = first * per + threadIdx.x; i < (p.B + 1) * per; i += 256) o[i] = make_uint4(0, 0, 0, 0);
}

// How a call is cut: up to kTreeRows rows per key/value head by the kernel
// above, in tiles of 64 keys, four warps a tile each; more by the tensor-core
// kernel in tiles of 256 rows and 128 keys.  The keys are split until the GPU
// is full: here once over (three CTAs per SM), a tile per warp at least, and
// with several requests at the latest every 2048 keys, so that sequences of
// different lengths share the SMs evenly (8 key/value heads, times against
// every 4096: 32 requests of up to 8000 keys 52 us and 67, 48 of 6000 54 and
// 69, 16 of 16001 53 and 75, but 64 of 16001 141 and 138, 128 of 2500 64 and
// 59; a single one of 131072: one wave 36 us, in 2048 keys, a wave and an
// eighth, 46); there one wave of one CTA per SM.  Up to eight splits are a
// thread-block cluster each and join in shared memory, without a second kernel
// and a workspace, where the whole grid is resident at once.  Beyond that whole
// clusters wait for room: with up to two waves of clusters 16 requests of 4100
// keys took 32 us (21 by way of the workspace), 32 of 1000 19 (13), 8 of 16001
// 43 (31); with more waves a third to a half more.
constexpr int kTreeRows = 16;
constexpr int kSplitTiles = 32;  // 2048 keys

struct Plan {
  int rows, tile_rows, tile_keys, m_tiles, n_split, split_tiles, cluster;
  size_t work;
};

Plan plan_rows(bool tree, long long rows, int R, int max_len, int Hkv, int dh, int most_splits, int sms) {
  Plan pl;
  pl.rows = static_cast<int>(rows);
  pl.tile_rows = tree ? kTreeRowsCta : rows > 8 ? 16 : 8;
  pl.tile_keys = tree ? 128 : kTileKeys;
  // (a tree's rows behind its last whole tile of 128 are planned by themselves)
  const int odd = static_cast<int>(rows % kTreeTile);
  const long long mine = tree && rows > kTreeTile && odd <= kTreeTail ? rows - odd : rows;
  pl.m_tiles = static_cast<int>((mine + pl.tile_rows - 1) / pl.tile_rows);
  const int tiles = max_len < 1 ? 1 : (max_len - 1) / pl.tile_keys + 1;
  const long long ctas = static_cast<long long>(R) * Hkv * pl.m_tiles;
  long long n = tree ? sms / ctas : (sms * 3 + ctas - 1) / ctas;
  if (!tree && R > 1 && n < (tiles + kSplitTiles - 1) / kSplitTiles) n = (tiles + kSplitTiles - 1) / kSplitTiles;
  const long long most = tree ? (tiles + 3) / 4 : (tiles + kWarps - 1) / kWarps;
  n = n < most ? n : most;
  n = n < most_splits ? n : most_splits;
  n = n < 1 ? 1 : n;
  pl.split_tiles = static_cast<int>((tiles + n - 1) / n);
  if (!tree) pl.split_tiles = (pl.split_tiles + kWarps - 1) / kWarps * kWarps;
  pl.n_split = (tiles + pl.split_tiles - 1) / pl.split_tiles;
  pl.cluster = !tree && pl.n_split > 1 && pl.n_split <= kMaxCluster &&
               (ctas * pl.n_split <= sms * 3 || most_splits == kMaxCluster);
  pl.work = pl.n_split > 1 && !pl.cluster
                ? static_cast<size_t>(ctas) * pl.n_split * pl.tile_rows * (dh + kPartHead) * sizeof(float)
                : 0;
  return pl;
}

// The launches of a call: [0] all rows, or those of whole tiles; [1] (tree
// only) the rows behind them, where a request may have some.
int plan_of(int R, int B, int max_len, int Hq, int Hkv, int dh, Plan (&pl)[2]) {
  const long long rows = static_cast<long long>(B + 1) * (Hq / Hkv);
  const bool tree = rows > kTreeRows, left = tree && rows > kTreeTile;
  int sms = 152;
  if (left) {
    // the rows left over: up to a cluster's splits (they run beside the others
    // and need no launch more), three CTAs to an SM, which the splits of the
    // others leave free (40 SMs at most: half of them cost one tree of 129 rows
    // 42 us, 32 with these)
    pl[1] = plan_rows(false, kTreeTail, R, max_len, Hkv, dh, kMaxCluster, sms);
    const long long theirs = (static_cast<long long>(R) * Hkv * pl[1].n_split + 2) / 3;
    sms -= static_cast<int>(theirs < 40 ? theirs : 40);
  }
  pl[0] = plan_rows(tree, rows, R, max_len, Hkv, dh, 1 << 30, sms);
  return left ? 2 : 1;
}

}  // namespace
}  // namespace dt

extern "C" size_t dartree_cache_attention_workspace(int32_t R, int32_t B, int32_t max_len, int32_t Hq,
                                                    int32_t Hkv, int32_t dh) {
  if (R < 1 || B < 0 || B > DARTREE_MAX_B || max_len < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 ||
      (dh != 64 && dh != 128))
    return 0;
  dt::Plan pl[2];
  dt::plan_of(R, B, max_len, Hq, Hkv, dh, pl);
  return pl[0].work;
}

extern "C" dartree_status dartree_cache_attention_ex(const dartree_cache* cache, int32_t layer, const void* Q,
                                                     int64_t q_token_stride, const uint32_t* mask,
                                                     const int32_t* n_nodes, const int32_t* table,
                                                     int32_t max_pages, const int32_t* lens, int32_t R,
                                                     int32_t B, int32_t max_len, int32_t Hq, float scale,
                                                     int32_t zero_rest, void* O, void* work, size_t work_bytes,
                                                     int32_t* err, void* stream) {
  using namespace dt;
  CacheAttnParams p{};
  if (const char* why = cache_view(cache, &p.c)) return cache_fail(DARTREE_ERR_INVALID_ARG, why);
  if (!Q || !table || !lens || !O || (B > 0 && !mask))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (layer < 0 || layer >= cache->layers) return cache_fail(DARTREE_ERR_INVALID_ARG, "no such layer");
  if (R < 1 || B < 0 || B > DARTREE_MAX_B || max_pages < 1 || max_len < 0 || Hq < 1 || Hq % p.c.Hkv != 0 ||
      !(scale > 0.f) || !(scale <= 3.0e38f))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "bad R, B, max_pages, max_len, Hq or scale");
  const int dh = p.c.dh;
  if (q_token_stride % 8 != 0 || q_token_stride < static_cast<int64_t>(Hq) * dh)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "q_token_stride must be a multiple of 8, at least Hq * dh");
  if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(O) | reinterpret_cast<uintptr_t>(work)) & 15)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "Q, O and work must be 16-byte aligned");
  Plan pl[2];
  const int launches = plan_of(R, B, max_len, Hq, p.c.Hkv, dh, pl);
  if (pl[0].work > 0 && (!work || work_bytes < pl[0].work))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "work is smaller than dartree_cache_attention_workspace()");
  p.g = Hq / p.c.Hkv;
  if (R > 65535 || static_cast<long long>(p.c.Hkv) * pl[0].m_tiles > 65535 || max_len > (1 << 30))
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "too many requests, heads or keys");
  p.c.pool += static_cast<size_t>(layer) * p.c.layer_bytes;
  p.Q = static_cast<const uint16_t*>(Q);
  p.q_stride = q_token_stride;
  p.mask = mask;
  p.n_nodes = n_nodes;
  p.table = table;
  p.lens = lens;
  p.max_pages = max_pages;
  p.R = R;
  p.B = B;
  p.max_len = max_len;
  p.Hq = Hq;
  p.words = (B + 31) / 32;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.O = static_cast<uint16_t*>(O);
  p.err = err;
  p.wait_limit = kWaitLimitCycles;
  // test knob (as for contexts): shorten the pipeline waits to provoke TIMEOUT
  if (const char* v = getenv("DARTREE_WAIT_LIMIT_CYCLES"))
    if (const long long c = atoll(v); c > 0) p.wait_limit = c;
  if (!(p.scale_log2 * p.c.k_scale <= 3.0e38f)) return cache_fail(DARTREE_ERR_INVALID_ARG, "scale times k_scale is too large");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!p.err) e = cudaGetSymbolAddress(reinterpret_cast<void**>(&p.err), g_cache_err);
  if (e != cudaSuccess) return cache_launched(e);
  if (zero_rest) e = launch_kernel(k_cache_zero_rest, dim3(R), dim3(256), 0, st, true, p);
  // (without n_nodes it is known here whether rows are left over)
  const int odd = pl[0].rows % kTreeTile;
  const int run = launches > 1 && !n_nodes && (odd == 0 || odd > kTreeTail) ? 1 : launches;
  CacheAttnParams first = p;
  for (int k = 0; k < run && e == cudaSuccess; ++k) {
    p.rows = pl[k].rows;
    p.tile_rows = pl[k].tile_rows;
    p.tile_keys = pl[k].tile_keys;
    p.m_tiles = pl[k].m_tiles;
    p.n_split = pl[k].n_split;
    p.split_tiles = pl[k].split_tiles;
    p.cluster = pl[k].cluster;
    p.tail = k;
    p.part = static_cast<float*>(work);
    if (k == 0) first = p;
    if (p.tile_rows == kTreeRowsCta) e = launch_cache_tree(p, st);
    else if (p.tile_rows == 8) e = dh == 128 ? launch_rows<128, 1>(p, st) : launch_rows<64, 1>(p, st);
    else e = dh == 128 ? launch_rows<128, 2>(p, st) : launch_rows<64, 2>(p, st);
  }
  // (the rows left over have joined in their cluster)
  if (e == cudaSuccess && first.n_split > 1 && !first.cluster)
    e = dh == 128 ? launch_join<128>(first, st) : launch_join<64>(first, st);
  return cache_launched(e);
}

extern "C" dartree_status dartree_cache_attention(const dartree_cache* cache, int32_t layer, const void* Q,
                                                  int64_t q_token_stride, const uint32_t* mask,
                                                  const int32_t* n_nodes, const int32_t* table,
                                                  int32_t max_pages, const int32_t* lens, int32_t R,
                                                  int32_t B, int32_t max_len, int32_t Hq, float scale,
                                                  void* O, void* work, size_t work_bytes, int32_t* err,
                                                  void* stream) {
  return dartree_cache_attention_ex(cache, layer, Q, q_token_stride, mask, n_nodes, table, max_pages, lens, R, B,
                                    max_len, Hq, scale, 0, O, work, work_bytes, err, stream);
}
