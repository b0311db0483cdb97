// Attention of single tokens and draft trees over the paged 4-bit cache
// (dartree_cache_attention).
//
// Rows (queries) of a key/value head: q = node * g + query head within the
// group, g = Hq / Hkv.  A CTA takes 16 rows of one request and one key/value
// head and a share of its keys (the keys are split over CTAs until the GPU
// is full; a second kernel joins the shares).  Four consumer warps take 16
// of a 64-key tile's keys each, with a softmax state and an output of their
// own until the end; a producer warp brings the tiles' codes and scales into
// shared memory with bulk copies, kStages tiles ahead.
//
// Both products are mma m16n8k16 in fp16 with fp32 sums: S = Q K^T (16 rows
// x 8 keys x 16 dims), O += P V (16 rows x 8 dims x 16 keys).  A code times
// its scale has 6 significant bits and lies between 2^-10 and 2688: exact in
// fp16.  The queries are scaled per row by a power of two to at most 1
// before they become fp16, so all that rounds is fp32 sums, P (2^-11, with
// its reference maximum at 2^6 so that weights down to 2^-20 of the largest
// keep all their bits) and the output.
//
// The k index of a product may run over the dims (or keys) in any order, and
// so may the n index: the orders are chosen so that a lane's codes lie
// together.  In S, lane (r = lane / 4, c = lane % 4) holds the dims
// [c dh/4, (c + 1) dh/4) of its key: one 16-byte (dh = 128) load.  In O, the
// n index r of n-tile j is dim r dh/8 + j: a lane holds dh/8 dims of four
// keys, and an output lane the dims [c dh/4, (c + 1) dh/4) of its rows.
#include "cache_attn.cuh"

namespace dt {
namespace {

constexpr int kTileKeys = 64;
constexpr int kStages = 4;
constexpr int kWarps = 4;                      // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRows = 16;                      // query rows per CTA

__device__ int g_cache_err;  // error word when the caller passes none

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes of one tile in shared memory: key codes, key scales, value codes,
// value scales of 64 tokens (a 64-token page's chunk, byte for byte).
template <int DH>
struct Tile {
  static constexpr int kCodes = kTileKeys * DH / 2, kScales = kTileKeys * DH / 16;
  static constexpr int kV = kCodes + kScales;
  static constexpr int kBytes = 2 * kV;
};

template <int DH>
struct __align__(128) AttnSmem {
  uint8_t stage[kStages][Tile<DH>::kBytes];
  uint64_t full[kStages], empty[kStages];
  uint64_t valid[kStages];       // bit k: key k of the tile is there
  float red[kWarps][kRows][DH + 4];
  float2 ml[kWarps][kRows];
  int abort_flag;
};

// The producer warp: tile f's pages into its stage.  A tile is pieces of
// min(page, 64) tokens; each piece is four copies (one when a page is a tile).
template <int DH>
__device__ __forceinline__ void produce(const CacheAttnParams& p, AttnSmem<DH>& sm, int r, int hk,
                                        const Span& sp, int t_beg, int nt) {
  using T = Tile<DH>;
  const int lane = threadIdx.x & 31;
  const int P = 1 << p.c.log_page;
  const int piece = P < kTileKeys ? P : kTileKeys;
  const int pieces = kTileKeys / piece;              // 4, 2, 1, 1
  const int segs = P == kTileKeys ? 1 : 4;           // copies per piece
  const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
  int issued = 0;
  bool flagged = false;
  for (int f = 0; f < nt; ++f) {
    const int st = f % kStages;
    if (f >= kStages) {
      int ok = 1;
      if (lane == 0)
        ok = mbar_wait(&sm.empty[st], static_cast<uint32_t>((f / kStages) & 1) ^ 1u, p.err) ? 1 : 0;
      if (!__shfl_sync(kFullMask, ok, 0)) {
        if (lane == 0) *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
        break;
      }
    }
    const int key0 = (t_beg + f) * kTileKeys;
    // lane (pc, seg): one copy
    const int pc = lane / segs, seg = lane % segs;
    const bool mine = lane < pieces * segs && key0 + pc * piece < sp.L;
    int page = -1;
    if (mine) {
      const int slot = (key0 + pc * piece) >> p.c.log_page;
      if (slot < p.max_pages) page = row[slot];
      if (page >= p.c.pages) page = -1;
    }
    const bool there = mine && page >= 0;
    if (mine && !there && !flagged) {
      flagged = true;
      atomicOr(p.err, DT_ERR_BAD_INDEX);
    }
    const unsigned got = __ballot_sync(kFullMask, there);
    const uint32_t piece_bytes = static_cast<uint32_t>(piece * DH / 8 * 9);
    if (lane == 0) {
      uint64_t v = 0;
      for (int k = 0; k < pieces; ++k)
        if ((got >> (k * segs)) & 1u) {
          const uint64_t m = piece == 64 ? ~0ull : ((1ull << piece) - 1) << (k * piece);
          v |= m;
        }
      const int left = sp.L - key0;
      if (left < kTileKeys) v &= (1ull << left) - 1;
      sm.valid[st] = v;
      mbar_arrive_expect_tx(&sm.full[st], __popc(got) / segs * piece_bytes);
    }
    __syncwarp();
    if (there) {
      const int tok0 = (key0 + pc * piece) & (P - 1);  // first token of the piece in its page
      const uint8_t* chunk = p.c.pool + static_cast<size_t>(page) * p.c.page_bytes +
                             static_cast<size_t>(hk) * p.c.chunk;
      uint8_t* dst = sm.stage[st];
      if (segs == 1) {
        bulk_load(dst, chunk, piece_bytes, &sm.full[st]);
      } else {
        const bool codes = (seg & 1) == 0;
        const int unit = codes ? DH / 2 : DH / 16;       // bytes of a token
        const int from = (seg >> 1) * (p.c.chunk >> 1) + (codes ? 0 : P * DH / 2) + tok0 * unit;
        const int to = (seg >> 1) * T::kV + (codes ? 0 : T::kCodes) + pc * piece * unit;
        bulk_load(dst + to, chunk + from, static_cast<uint32_t>(piece * unit), &sm.full[st]);
      }
    }
    issued = f + 1;
  }
  // every copy must have landed before the block may end
  if (lane == 0)
    for (int f = issued > kStages ? issued - kStages : 0; f < issued; ++f)
      mbar_wait(&sm.full[f % kStages], static_cast<uint32_t>((f / kStages) & 1), p.err);
}

template <int DH>
__global__ void __launch_bounds__(kThreads) k_cache_attention(const CacheAttnParams p) {
  constexpr int kSteps = DH / 16;   // k-steps of S
  constexpr int kNT = DH / 8;       // n-tiles of O
  using T = Tile<DH>;
  extern __shared__ __align__(128) uint8_t raw[];
  AttnSmem<DH>& sm = *reinterpret_cast<AttnSmem<DH>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, hk = blockIdx.y / p.m_tiles, mt = blockIdx.y % p.m_tiles, r = blockIdx.z;
  Span sp;
  if (!request_span(p, r, &sp)) return;
  const int q0 = mt * kRows;
  const int live = min((sp.n + 1) * p.g - q0, kRows);  // rows of this tile
  if (live <= 0) return;
  const int t_all = row_tile_keys(p, sp, mt);
  const int t_beg = split * p.split_tiles;
  const int nt = min(t_all, t_beg + p.split_tiles) - t_beg;
  if (nt <= 0 && !(split == 0 && p.n_split == 1)) return;  // (one split: rows without keys are written as 0)

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], kWarps);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
    if (split == 0 && hk == 0 && mt == 0 &&
        static_cast<long long>(p.lens[r]) + sp.n > p.max_len)
      atomicOr(p.err, DT_ERR_BAD_INDEX);
  }
  __syncthreads();

  if (warp == kWarps) {
    produce<DH>(p, sm, r, hk, sp, t_beg, nt);
  } else {
    const int rr = lane >> 2, c = lane & 3;
    // ---- queries: rows q0 + rr and q0 + rr + 8, dims [c DH/4, (c+1) DH/4)
    uint32_t qa[kSteps][4];
    float fac[2];
    int node[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = q0 + rr + 8 * h;
      const bool on = rr + 8 * h < live;
      node[h] = on ? q / p.g : 0;
      uint32_t w[DH / 8];  // DH/4 bf16
      const uint4* src = reinterpret_cast<const uint4*>(
          p.Q + (static_cast<size_t>(r) * (p.B + 1) + node[h]) * p.q_stride +
          static_cast<size_t>(hk * p.g + (on ? q % p.g : 0)) * DH + c * (DH / 4));
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
      // 2^-e with 2^e <= top < 2^(e+1) (e within what the factors can be)
      int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      e = top > 0.f ? max(-100, min(e, 100)) : 0;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      fac[h] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t x = w[2 * s], y = w[2 * s + 1];  // dims 4s, 4s+1 | 4s+2, 4s+3 of the lane's
        qa[s][h] = pack_f16(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xFFFF0000u) * down);
        qa[s][2 + h] = pack_f16(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xFFFF0000u) * down);
      }
    }
    float o[kNT][4];
#pragma unroll
    for (int j = 0; j < kNT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int k0 = warp * 16;  // the warp's keys within a tile

    for (int f = 0; f < nt; ++f) {
      const int st = f % kStages;
      int ok = 1;
      if (lane == 0)
        ok = !*reinterpret_cast<volatile int*>(&sm.abort_flag) &&
             mbar_wait(&sm.full[st], static_cast<uint32_t>((f / kStages) & 1), p.err);
      if (!__shfl_sync(kFullMask, ok, 0)) {
        if (lane == 0) *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
        break;
      }
      // (every lane's own look at the barrier: the copies are visible to it)
      mbar_try_wait(smem_u32(&sm.full[st]), static_cast<uint32_t>((f / kStages) & 1));
      const uint8_t* tile = sm.stage[st];
      const int key0 = (t_beg + f) * kTileKeys + k0;
      const uint32_t valid = static_cast<uint32_t>(sm.valid[st] >> k0) & 0xFFFFu;
      const bool plain = valid == 0xFFFFu && key0 + 16 <= sp.Lp;  // all seen by every row
      // ---- S: two n-tiles of 8 keys; n index r is key (r / 2) + 4 (r % 2) + 8 t
      float s[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
        const int key = k0 + (rr >> 1) + 4 * (rr & 1) + 8 * t;
        uint32_t w[DH / 32];
        uint32_t sc[2];
        if constexpr (DH == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + key * 64 + c * 16);
          w[0] = x.x;
          w[1] = x.y;
          w[2] = x.z;
          w[3] = x.w;
          const uint32_t two = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t*>(tile + T::kCodes + key * 8 + c * 2));
          sc[0] = __byte_perm(two, two, 0x1010);
          sc[1] = __byte_perm(two, two, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(tile + key * 32 + c * 8);
          w[0] = x.x;
          w[1] = x.y;
          const uint32_t b = tile[T::kCodes + key * 4 + c];
          sc[0] = sc[1] = e4m3x2_to_f16x2(b | (b << 8));
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint32_t two = (w[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
          const uint32_t scl = sc[k >> 2];
          mma_f16(s[t], qa[k], h2mul(e2m1x2_to_f16x2(two & 0xFFu), scl),
                  h2mul(e2m1x2_to_f16x2(two >> 8), scl));
        }
      }
      // ---- scores in base 2; lane's keys: col 2c + i of n-tile t is key c + 4 i + 8 t
      if (plain) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[t][x] *= fac[x >> 1];
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int h = x >> 1, kk = c + 4 * (x & 1) + 8 * t, pos = key0 + kk;
            bool seen = (valid >> kk) & 1u;
            if (seen && pos >= sp.Lp) {
              const int j = pos - sp.Lp;
              seen = node[h] > 0 &&
                     ((__ldg(p.mask + (static_cast<size_t>(r) * p.B + node[h] - 1) * p.words + (j >> 5)) >>
                       (j & 31)) & 1u);
            }
            s[t][x] = seen ? s[t][x] * fac[h] : -INFINITY;
          }
      }
      const float t0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      const float t1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
      if (__any_sync(kFullMask, t0 > m[0] + kRaise || t1 > m[1] + kRaise)) {
        float top[2] = {t0, t1}, al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(kFullMask, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(kFullMask, top[h], 2));
          al[h] = 1.f;
          if (top[h] > m[h] + kRaise) {
            al[h] = ex2(m[h] - top[h]);  // (0 from -inf)
            m[h] = top[h];
            l[h] *= al[h];
          }
        }
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
          o[j][0] *= al[0];
          o[j][1] *= al[0];
          o[j][2] *= al[1];
          o[j][3] *= al[1];
        }
      }
      const float sub0 = m[0] == -INFINITY ? 0.f : m[0] - kBias, sub1 = m[1] == -INFINITY ? 0.f : m[1] - kBias;
      uint32_t pa[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = ex2(s[t][0] - sub0), p1 = ex2(s[t][1] - sub0);
        const float p2 = ex2(s[t][2] - sub1), p3 = ex2(s[t][3] - sub1);
        l[0] += p0 + p1;
        l[1] += p2 + p3;
        pa[2 * t] = pack_f16(p0, p1);
        pa[2 * t + 1] = pack_f16(p2, p3);
      }
      // ---- O += P V: lane's keys c, c+4 | c+8, c+12; dims [rr DH/8, (rr+1) DH/8)
      const uint8_t* vt = tile + T::kV;
      uint32_t vw[4][DH / 64], vs[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t b[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = c + 4 * i + 8 * t, key = k0 + kk;
          if constexpr (DH == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(vt + key * 64 + rr * 8);
            vw[2 * t + i][0] = x.x;
            vw[2 * t + i][1] = x.y;
            b[i] = vt[T::kCodes + key * 8 + rr];
          } else {
            vw[2 * t + i][0] = *reinterpret_cast<const uint32_t*>(vt + key * 32 + rr * 4);
            b[i] = vt[T::kCodes + key * 4 + (rr >> 1)];
          }
          // what lies behind the keys may be anything: a zero weight needs a finite value
          if (!plain && !((valid >> kk) & 1u)) b[i] = 0;
        }
        vs[t] = e4m3x2_to_f16x2(b[0] | (b[1] << 8));
      }
#pragma unroll
      for (int w = 0; w < DH / 64; ++w) {
        uint32_t ev[2], od[2];  // bytes: (first key's, second key's) codes of the even, odd dims
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t x = vw[2 * t][w], y = vw[2 * t + 1][w];
          ev[t] = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
          od[t] = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          mma_f16(o[8 * w + 2 * k], pa, h2mul(e2m1x2_to_f16x2((ev[0] >> (8 * k)) & 0xFFu), vs[0]),
                  h2mul(e2m1x2_to_f16x2((ev[1] >> (8 * k)) & 0xFFu), vs[1]));
          mma_f16(o[8 * w + 2 * k + 1], pa, h2mul(e2m1x2_to_f16x2((od[0] >> (8 * k)) & 0xFFu), vs[0]),
                  h2mul(e2m1x2_to_f16x2((od[1] >> (8 * k)) & 0xFFu), vs[1]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
    }
    // ---- the warp's rows into shared memory
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(kFullMask, l[h], 1);
      l[h] += __shfl_xor_sync(kFullMask, l[h], 2);
      if (c == 0) sm.ml[warp][rr + 8 * h] = make_float2(m[h], l[h]);
      float* dst = &sm.red[warp][rr + 8 * h][c * (DH / 4)];
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        dst[j] = o[j][2 * h];
        dst[kNT + j] = o[j][2 * h + 1];
      }
    }
  }
  __syncthreads();
  // ---- the four warps' shares of each row, joined in warp order
  const float out_scale = p.c.v_scale;
  for (int row = warp; row < live; row += kWarps + 1) {
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
    if (p.n_split > 1) {
      float* dst = cache_part_row(p, r, hk, mt, split, row);
#pragma unroll
      for (int e = 0; e < kE; e += 2)
        *reinterpret_cast<float2*>(dst + 2 + lane * kE + e) = make_float2(v[e], v[e + 1]);
      if (lane == 0) *reinterpret_cast<float2*>(dst) = make_float2(M, L);
    } else {
      const float inv = L > 0.f ? out_scale / L : 0.f;
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q0 + row) + lane * kE);
#pragma unroll
      for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
    }
  }
}

// The shares of each row over the key splits, joined in split order:
// M = max m_s, O = sum O_s 2^(m_s - M) / sum l_s 2^(m_s - M).  One warp per
// row; grid (rows / 8, Hkv, R).
template <int DH>
__global__ void __launch_bounds__(256) k_cache_attention_join(const CacheAttnParams p) {
  const int lane = threadIdx.x & 31;
  const int q = blockIdx.x * 8 + (threadIdx.x >> 5), hk = blockIdx.y, r = blockIdx.z;
  pdl_wait();
  Span sp;
  if (!request_span(p, r, &sp) || q >= (sp.n + 1) * p.g) return;
  const int mt = q / p.tile_rows;
  const int ns = (row_tile_keys(p, sp, mt) + p.split_tiles - 1) / p.split_tiles;  // splits that had keys
  constexpr int kE = DH / 32;
  const size_t step = static_cast<size_t>(p.tile_rows) * (DH + 2);
  const float* src = cache_part_row(p, r, hk, mt, 0, q - mt * p.tile_rows);
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, src[s * step]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, x));
  float L = 0.f, v[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) v[e] = 0.f;
  for (int s = 0; s < ns; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(src + s * step);
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    L += ml.y * f;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const float2 x = *reinterpret_cast<const float2*>(src + s * step + 2 + lane * kE + e);
      v[e] += x.x * f;
      v[e + 1] += x.y * f;
    }
  }
  const float inv = L > 0.f ? p.c.v_scale / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q) + lane * kE);
#pragma unroll
  for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
}

// How a call is cut: up to kTreeRows rows per key/value head by the kernel
// above, in tiles of 16 rows and 64 keys; more by the tensor-core kernel in
// tiles of 128 rows and 128 keys.  The keys are split until the GPU is full:
// here enough CTAs for about three waves of the three that an SM holds, two
// tiles each at least; there one wave of one CTA per SM.
constexpr int kTreeRows = 16;

struct Plan {
  int tile_rows, tile_keys, m_tiles, n_split, split_tiles;
  size_t work;
};

Plan plan_of(int R, int B, int max_len, int Hq, int Hkv, int dh) {
  Plan pl;
  const long long rows = static_cast<long long>(B + 1) * (Hq / Hkv);
  const bool tree = rows > kTreeRows;
  pl.tile_rows = tree ? 128 : kRows;
  pl.tile_keys = tree ? 128 : kTileKeys;
  pl.m_tiles = static_cast<int>((rows + pl.tile_rows - 1) / pl.tile_rows);
  const int tiles = max_len < 1 ? 1 : (max_len - 1) / pl.tile_keys + 1;
  const long long ctas = static_cast<long long>(R) * Hkv * pl.m_tiles;
  long long n = tree ? 152 / ctas : (152 * 6 + ctas - 1) / ctas;
  const long long most = (tiles + 1) / 2;
  n = n < most ? n : most;
  n = n < 1 ? 1 : n;
  pl.split_tiles = static_cast<int>((tiles + n - 1) / n);
  pl.n_split = (tiles + pl.split_tiles - 1) / pl.split_tiles;
  pl.work = pl.n_split > 1 ? static_cast<size_t>(ctas) * pl.n_split * pl.tile_rows * (dh + 2) * sizeof(float) : 0;
  return pl;
}

}  // namespace
}  // namespace dt

extern "C" size_t dartree_cache_attention_workspace(int32_t R, int32_t B, int32_t max_len, int32_t Hq,
                                                    int32_t Hkv, int32_t dh) {
  if (R < 1 || B < 0 || B > DARTREE_MAX_B || max_len < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 ||
      (dh != 64 && dh != 128))
    return 0;
  return dt::plan_of(R, B, max_len, Hq, Hkv, dh).work;
}

extern "C" dartree_status dartree_cache_attention(const dartree_cache* cache, int32_t layer, const void* Q,
                                                  int64_t q_token_stride, const uint32_t* mask,
                                                  const int32_t* n_nodes, const int32_t* table,
                                                  int32_t max_pages, const int32_t* lens, int32_t R,
                                                  int32_t B, int32_t max_len, int32_t Hq, float scale,
                                                  void* O, void* work, size_t work_bytes, int32_t* err,
                                                  void* stream) {
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
  const Plan pl = plan_of(R, B, max_len, Hq, p.c.Hkv, dh);
  if (pl.work > 0 && (!work || work_bytes < pl.work))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "work is smaller than dartree_cache_attention_workspace()");
  p.g = Hq / p.c.Hkv;
  if (R > 65535 || static_cast<long long>(p.c.Hkv) * pl.m_tiles > 65535 || max_len > (1 << 30))
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
  p.rows = (B + 1) * p.g;
  p.tile_rows = pl.tile_rows;
  p.tile_keys = pl.tile_keys;
  p.m_tiles = pl.m_tiles;
  p.n_split = pl.n_split;
  p.split_tiles = pl.split_tiles;
  p.scale_log2 = scale * 1.4426950408889634f * p.c.k_scale;
  p.O = static_cast<uint16_t*>(O);
  p.part = static_cast<float*>(work);
  p.err = err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(pl.n_split, p.c.Hkv * pl.m_tiles, R);
  cudaError_t e = cudaSuccess;
  if (!p.err) e = cudaGetSymbolAddress(reinterpret_cast<void**>(&p.err), g_cache_err);
  if (e != cudaSuccess) return cache_launched(e);
  if (pl.tile_rows == 128) {
    e = launch_cache_tree(p, st);
  } else if (dh == 128) {
    e = set_max_dynamic_smem(k_cache_attention<128>);
    if (e == cudaSuccess)
      e = launch_kernel(k_cache_attention<128>, grid, dim3(kThreads), sizeof(AttnSmem<128>), st, false, p);
  } else {
    e = set_max_dynamic_smem(k_cache_attention<64>);
    if (e == cudaSuccess)
      e = launch_kernel(k_cache_attention<64>, grid, dim3(kThreads), sizeof(AttnSmem<64>), st, false, p);
  }
  if (e == cudaSuccess && pl.n_split > 1) {
    const dim3 jgrid((p.rows + 7) / 8, p.c.Hkv, R);
    e = launch_kernel(dh == 128 ? k_cache_attention_join<128> : k_cache_attention_join<64>, jgrid, dim3(256), 0,
                      st, true, p);
  }
  return cache_launched(e);
}
