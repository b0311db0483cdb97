// Attention of draft trees over the paged 4-bit cache on the 5th-generation
// tensor cores (dartree_cache_attention with more than a few query rows per
// key/value head).
//
// A CTA owns 128 query rows (one TMEM lane each) of one request and one
// key/value head and a share of the key range, in tiles of 128 keys.  Warp
// roles (448 threads):
//   0-7   softmax: two warpgroups, a thread owns a row and half of each
//         tile's keys and of the head dimensions of O;
//   8-11  expand the tiles: codes and scales to fp16 keys and values (exact);
//   12    producer: bulk copies of the pages' codes and scales, kRaw tiles
//         ahead;
//   13    TMEM owner, issues the MMAs.
// S = Q K^T (M 128, N 128, fp16, fp32 sums) into double-buffered TMEM; P =
// 2^(s - m + kBias) in fp16 to TMEM; O += P V with P from TMEM.  Keys and
// values lie in shared memory in the same layout (a token's row of 64 head
// dimensions is a 128-byte swizzled line): for S it is a K-major operand, for
// O the same lines are MN-major (the transposed read is the tensor core's).
// The running maximum is a reference that rises only when a score passes it
// by kRaise, which rescales O in TMEM.
#include "cache_attn.cuh"

namespace dt {
namespace {

constexpr int kRowsQ = 128, kKeys = 128, kHalf = kKeys / 2;
constexpr int kSoftmaxWarps = 8, kExpandWarps = 4;
constexpr int kExpandWarp0 = 8, kProducerWarp = 12, kMmaWarp = 13;
constexpr int kTreeThreads = 14 * 32;
constexpr int kStages = 2, kRaw = 3;
constexpr int kValid = kRaw + 5;     // tiles from a raw tile's copy to the end of its softmax
constexpr uint32_t kTmemCols = 512;  // S0 [0,128) S1 [128,256) O [256,256+dh) P0 [384,448) P1 [448,512)
constexpr uint32_t kColO = 256, kColP = 384;

template <int DH>
struct TreeSmem {
  static constexpr int kTile = kKeys * DH * 2;           // fp16 keys or values of a tile
  static constexpr int kCodes = kKeys * DH / 2, kScales = kKeys * DH / 16;
  static constexpr int kV = kCodes + kScales, kRawBytes = 2 * kV;
  static constexpr int kQ = 0;
  static constexpr int kStage = kQ + kRowsQ * DH * 2;    // stage s: keys, values
  static constexpr int kRaw0 = kStage + kStages * 2 * kTile;
  static constexpr int kBars = kRaw0 + kRaw * kRawBytes;
  static constexpr int kTotal = kBars + 512;
  static constexpr int kOPitch = DH + 4;                 // floats per staged row of O
  static_assert(kRowsQ * kOPitch * 4 <= kStages * 2 * kTile + kRaw * kRawBytes, "O is staged over the tiles");
};

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t sw128(int r, int gr) {
  return static_cast<uint32_t>(r * 128 + ((gr ^ (r & 7)) << 4));
}

// Instruction descriptor: fp16 operands, fp32 sums, M = 128; b_mn: B is
// MN-major.
__device__ __forceinline__ constexpr uint32_t idesc_f16(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

// Descriptor of an MN-major operand in 128-byte swizzled lines: 64 elements
// of the MN extent per line, a line per k; 8 lines are an atom (the stride
// between atoms along k), the next 64 elements of the MN extent `lead` bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <int DH>
__global__ void __launch_bounds__(kTreeThreads, 1) k_cache_tree(const CacheAttnParams p) {
  using L = TreeSmem<DH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem + L::kQ;
  uint8_t* sStage = smem + L::kStage;
  uint8_t* sRaw = smem + L::kRaw0;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* k_full = raw_empty + kRaw;
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;
  uint64_t* s_empty = s_full + 2;
  uint64_t* p_full = s_empty + 2;
  uint64_t* p_empty = p_full + 2;
  uint64_t* o_done = p_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // bit k of a tile's 128: key k is there.  Tile f's copy starts after tile
  // f - 3 (kRaw) is expanded, its keys after the scores of f - 5 (kStages),
  // they after the softmax of f - 7 (two buffers) has begun: that of f - 8 is
  // done, so eight slots do.
  __shared__ uint32_t s_valid[kValid][4];
  __shared__ float s_fac[kRowsQ];
  __shared__ float2 s_ml[kRowsQ];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = blockIdx.z, hk = blockIdx.y;
  const int mt = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split;
  Span sp;
  if (!request_span(p, r, &sp)) return;
  const int q0 = mt * kRowsQ;
  const int live = min((sp.n + 1) * p.g - q0, kRowsQ);
  if (live <= 0) return;
  const int t_all = row_tile_keys(p, sp, mt);
  const int t_beg = split * p.split_tiles;
  const int nt = min(t_all, t_beg + p.split_tiles) - t_beg;
  if (nt <= 0 && !(split == 0 && p.n_split == 1)) return;

  if (warp == kMmaWarp) tmem_alloc<kTmemCols>(tmem_slot);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1);
      mbar_init(&raw_empty[s], kExpandWarps);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], kExpandWarps);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], kExpandWarps);
      mbar_init(&v_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&s_empty[b], kSoftmaxWarps);
      mbar_init(&p_full[b], kSoftmaxWarps);
      mbar_init(&p_empty[b], 1);
    }
    mbar_init(o_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (split == 0 && hk == 0 && mt == 0 && static_cast<long long>(p.lens[r]) + sp.n > p.max_len)
      atomicOr(p.err, DT_ERR_BAD_INDEX);
  }
  // the queries, as fp16 rows scaled by a power of two to at most 2 each
  if (threadIdx.x < kRowsQ) {
    const int row = threadIdx.x, q = q0 + row;
    const bool on = row < live;
    const int node = on ? q / p.g : 0;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.Q + (static_cast<size_t>(r) * (p.B + 1) + node) * p.q_stride +
        static_cast<size_t>(hk * p.g + (on ? q - node * p.g : 0)) * DH);
    uint4 w[DH / 8];
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < DH / 8; ++k) {
      w[k] = on ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[j] << 16)), fabsf(__uint_as_float(x[j] & 0xFFFF0000u))));
    }
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = top > 0.f ? max(-100, min(e, 100)) : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    s_fac[row] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int k = 0; k < DH / 8; ++k) {
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_f16(__uint_as_float(x[j] << 16) * down, __uint_as_float(x[j] & 0xFFFF0000u) * down);
      *reinterpret_cast<uint4*>(sQ + (k >> 3) * (kRowsQ * 128) + sw128(row, k & 7)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // a warp-uniform bounded wait (lane 0 polls); false: give up
  auto wait_w = [&](uint64_t* bar, uint32_t par) {
    int ok = 0;
    if (lane == 0) ok = !*abort_flag && mbar_wait(bar, par, p.err) ? 1 : 0;
    return __shfl_sync(kFullMask, ok, 0) != 0;
  };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------ producer
    const int P = 1 << p.c.log_page;
    const int pieces = kKeys / P;                  // 8, 4, 2, 1
    const int segs = pieces == 1 ? 1 : 4;          // copies per piece (a 128-token page's chunk is a raw tile)
    const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
    const int pc = lane / segs, seg = lane % segs;
    const uint32_t piece_bytes = static_cast<uint32_t>(P * DH / 8 * 9);
    int issued = 0;
    bool flagged = false;
    for (int f = 0; f < nt; ++f) {
      const int st = f % kRaw;
      if (f >= kRaw && !wait_w(&raw_empty[st], static_cast<uint32_t>((f / kRaw) & 1) ^ 1u)) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      const int key0 = (t_beg + f) * kKeys;
      const bool mine = lane < pieces * segs && key0 + pc * P < sp.L;
      int page = -1;
      if (mine) {
        const int slot = (key0 >> p.c.log_page) + pc;
        if (slot < p.max_pages) page = row[slot];
        if (page >= p.c.pages) page = -1;
      }
      const bool there = mine && page >= 0;
      if (mine && !there && !flagged) {
        flagged = true;
        atomicOr(p.err, DT_ERR_BAD_INDEX);
      }
      const unsigned got = __ballot_sync(kFullMask, there);
      if (lane < 4) {  // keys 32 lane .. 32 lane + 31
        uint32_t v = 0;
        for (int k = 0; k < pieces; ++k) {
          if (!((got >> (k * segs)) & 1u)) continue;
          const int a = max(k * P - 32 * lane, 0), b = min(min((k + 1) * P, sp.L - key0) - 32 * lane, 32);
          if (b > a) v |= (b == 32 ? 0xFFFFFFFFu : (1u << b) - 1u) & ~((1u << a) - 1u);
        }
        s_valid[f % kValid][lane] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&raw_full[st], __popc(got) / segs * piece_bytes);
      __syncwarp();
      if (there) {
        const uint8_t* chunk = p.c.pool + static_cast<size_t>(page) * p.c.page_bytes +
                               static_cast<size_t>(hk) * p.c.chunk;
        uint8_t* dst = sRaw + st * L::kRawBytes;
        if (segs == 1) {
          bulk_load(dst, chunk, piece_bytes, &raw_full[st]);
        } else {
          const bool codes = (seg & 1) == 0;
          const int unit = codes ? DH / 2 : DH / 16;
          bulk_load(dst + (seg >> 1) * L::kV + (codes ? 0 : L::kCodes) + pc * P * unit,
                    chunk + (seg >> 1) * (p.c.chunk >> 1) + (codes ? 0 : P * DH / 2),
                    static_cast<uint32_t>(P * unit), &raw_full[st]);
        }
      }
      issued = f + 1;
    }
    if (lane == 0)  // every copy must have landed before the block may end
      for (int f = issued > kRaw ? issued - kRaw : 0; f < issued; ++f)
        mbar_wait(&raw_full[f % kRaw], static_cast<uint32_t>((f / kRaw) & 1), p.err);
  } else if (warp >= kExpandWarp0 && warp < kProducerWarp) {
    // ------------------------------------------------- codes to fp16 tiles
    // Lane (key = lane / 4, c = lane % 4) of a warp's 8 keys takes the dims
    // [c DH/4, (c+1) DH/4): one load of codes, two (one) scales, DH/32 lines
    // of 16 bytes.  The lanes of c >= 2 write theirs in another order: the
    // eight lanes of a store's phase then lie in eight different 16-byte
    // columns.
    const int ew = warp - kExpandWarp0, kl = lane >> 2, c = lane & 3;
    bool go = true;
    for (int f = 0; f < nt && go; ++f) {
      const int st = f % kStages, rs = f % kRaw;
      const uint32_t ph = static_cast<uint32_t>((f / kStages) & 1);
      go = wait_w(&raw_full[rs], static_cast<uint32_t>((f / kRaw) & 1));
      if (!go) break;
      mbar_try_wait(smem_u32(&raw_full[rs]), static_cast<uint32_t>((f / kRaw) & 1));
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        if (f >= kStages && !wait_w(kv == 0 ? &k_empty[st] : &v_empty[st], ph ^ 1u)) {
          go = false;
          break;
        }
        const uint8_t* raw = sRaw + rs * L::kRawBytes + kv * L::kV;
        uint8_t* dst = sStage + st * 2 * L::kTile + kv * L::kTile;
#pragma unroll
        for (int it = 0; it < kKeys / (kExpandWarps * 8); ++it) {
          const int key = (it * kExpandWarps + ew) * 8 + kl;
          const bool there = (s_valid[f % kValid][key >> 5] >> (key & 31)) & 1u;
          uint32_t w[DH / 32], sc[2];
          if constexpr (DH == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(raw + key * 64 + c * 16);
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
            uint32_t two = *reinterpret_cast<const uint16_t*>(raw + L::kCodes + key * 8 + c * 2);
            two = e4m3x2_to_f16x2(there ? two : 0u);
            sc[0] = __byte_perm(two, two, 0x1010);
            sc[1] = __byte_perm(two, two, 0x3232);
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(raw + key * 32 + c * 8);
            w[0] = x.x;
            w[1] = x.y;
            const uint32_t b = there ? raw[L::kCodes + key * 4 + c] : 0u;
            sc[0] = sc[1] = e4m3x2_to_f16x2(b | (b << 8));
          }
          uint8_t* line = dst + (DH == 128 ? (c >> 1) * (kKeys * 128) : 0);
#pragma unroll
          for (int i = 0; i < DH / 32; ++i) {
            const int g = DH == 128 ? ((c & 1) << 2) : (c << 1);
            const int ii = DH == 128 ? i ^ (c & 2) : i;     // (which of the lane's lines)
            uint32_t word = w[i];
            uint32_t scl = sc[DH == 128 ? i >> 1 : 0];
            if (DH == 128 && (c & 2)) {                      // i ^ 2
              word = w[i ^ 2];
              scl = sc[(i ^ 2) >> 1];
            }
            uint32_t y[4];
            e2m1x8_to_f16(word, y);
            *reinterpret_cast<uint4*>(line + sw128(key, g + ii)) =
                make_uint4(h2mul(y[0], scl), h2mul(y[1], scl), h2mul(y[2], scl), h2mul(y[3], scl));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(kv == 0 ? &k_full[st] : &v_full[st]);
          if (kv == 1) mbar_arrive(&raw_empty[rs]);
        }
      }
    }
    if (!go && lane == 0) *abort_flag = 1;
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16(kKeys, false), idesc_o = idesc_f16(DH, true);
      const uint32_t q_addr = smem_u32(sQ);
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t par) {
        if (ok && !*abort_flag && mbar_wait(bar, par, p.err)) return true;
        ok = false;
        *abort_flag = 1;
        return false;
      };
      auto issue_s = [&](int j) {
        const int b = j & 1, st = j % kStages;
        if (!wait(&s_empty[b], (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u)) return;
        if (!wait(&k_full[st], static_cast<uint32_t>((j / kStages) & 1))) return;
        tc_fence_after();
        const uint32_t k_addr = smem_u32(sStage + st * 2 * L::kTile);
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = (kk & 3) * 32u;
          tc_mma_bf16(tmem_base + static_cast<uint32_t>(b * kKeys),
                      smem_desc_sw128(q_addr + (kk >> 2) * (kRowsQ * 128) + off),
                      smem_desc_sw128(k_addr + (kk >> 2) * (kKeys * 128) + off), idesc_s, kk != 0 ? 1u : 0u);
        }
        tc_commit(&s_full[b]);
        tc_commit(&k_empty[st]);
      };
      auto issue_o = [&](int j) {
        const int st = j % kStages, pb = j & 1;
        if (!wait(&p_full[pb], static_cast<uint32_t>(j >> 1) & 1u)) return;
        if (!wait(&v_full[st], static_cast<uint32_t>((j / kStages) & 1))) return;
        tc_fence_after();
        const uint32_t v_addr = smem_u32(sStage + st * 2 * L::kTile + L::kTile);
        const uint32_t pa = tmem_base + kColP + static_cast<uint32_t>(pb * (kKeys / 2));
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)  // 16 keys: two atoms of 8 lines
          tc_mma_bf16_ta(tmem_base + kColO, pa + static_cast<uint32_t>(kk * 8),
                         smem_desc_mn(v_addr + kk * 2048, kKeys * 128), idesc_o, (j != 0 || kk != 0) ? 1u : 0u);
        tc_commit(&p_empty[pb]);
        tc_commit(&v_empty[st]);
      };
      for (int j = 0; j < nt && ok; ++j) {
        issue_s(j);
        if (ok && j > 0) issue_o(j - 1);
      }
      if (ok && nt > 0) issue_o(nt - 1);
      tc_commit(o_done);
      mbar_wait(o_done, 0, p.err);
    }
  } else {
    // ------------------------------------------------------------- softmax
    __shared__ float red[2][kRowsQ];
    __shared__ float red2[2][2][kRowsQ];
    __shared__ int stop_slot[2][kSoftmaxWarps];
    const int wg = warp >> 2, wq = warp & 3;
    const int row = wq * 32 + lane, q = q0 + row;
    const int node = row < live ? q / p.g : 0;
    const uint32_t* mrow =
        node >= 1 ? p.mask + (static_cast<size_t>(r) * p.B + node - 1) * p.words : nullptr;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const int col0 = wg * kHalf;
    const float fac = s_fac[row];
    const bool idle = wq * 32 >= live;  // none of the warp's rows exists
    constexpr int kOH = DH / 2;
    float m = -INFINITY, l = 0.f;
    bool go = true;
    for (int j = 0; j < nt; ++j) {
      const int key0 = (t_beg + j) * kKeys + col0;
      // the mask words of this group's half of the tile (three from the one
      // that holds its first node)
      uint32_t mw[3] = {0u, 0u, 0u};
      if (mrow && key0 + kHalf > sp.Lp) {
        const int wb = (key0 > sp.Lp ? key0 - sp.Lp : 0) >> 5;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (wb + k < p.words) mw[k] = __ldg(mrow + wb + k);
      }
      const bool okw = go && wait_w(&s_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u);
      float s[kHalf];
      float mh = -INFINITY;
      if (okw) {
        tc_fence_after();
        const uint32_t taddr = tmem_base + lane_base + static_cast<uint32_t>((j & 1) * kKeys + col0);
        if (!idle) {
#pragma unroll
          for (int c = 0; c < kHalf; c += 16) {
            float x[16];
            tmem_ld16(taddr + c, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[c + i] = x[i];
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[j & 1]);
        if (!idle) {
          const uint32_t va = s_valid[j % kValid][2 * wg], vb = s_valid[j % kValid][2 * wg + 1];
          if (key0 + kHalf <= sp.Lp && (va & vb) == 0xFFFFFFFFu) {
#pragma unroll
            for (int c = 0; c < kHalf; ++c) s[c] *= fac;
          } else {
            const int np = sp.Lp > key0 ? sp.Lp - key0 : 0;  // prefix keys of the window
            const int tf = key0 > sp.Lp ? key0 - sp.Lp : 0;  // its first node
            const uint32_t lo = __funnelshift_r(mw[0], mw[1], tf & 31);
            const uint32_t hi = __funnelshift_r(mw[1], mw[2], tf & 31);
            uint64_t vis = (static_cast<uint64_t>(hi) << 32) | lo;
            vis = np >= 64 ? ~0ull : (vis << np) | ((1ull << np) - 1);
            const uint32_t v0 = static_cast<uint32_t>(vis) & va, v1 = static_cast<uint32_t>(vis >> 32) & vb;
#pragma unroll
            for (int c = 0; c < kHalf; ++c) {
              const bool seen = (((c < 32 ? v0 : v1) >> (c & 31)) & 1u) != 0u;
              s[c] = seen ? s[c] * fac : -INFINITY;
            }
          }
#pragma unroll
          for (int c = 0; c < kHalf; ++c) mh = fmaxf(mh, s[c]);
        }
      }
      red2[j & 1][wg][row] = mh;
      if (lane == 0) stop_slot[j & 1][warp] = okw ? 0 : 1;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      int stop = 0;
#pragma unroll
      for (int w = 0; w < kSoftmaxWarps; ++w) stop |= stop_slot[j & 1][w];
      if (stop) {  // the same for all 256 threads
        go = false;
        *abort_flag = 1;
        break;
      }
      const float mx = fmaxf(red2[j & 1][0][row], red2[j & 1][1][row]);
      const bool raise = mx > m + kRaise;  // the same in both groups
      bool failed = false;
      if (__any_sync(kFullMask, raise)) {
        const float m_new = raise ? mx : m;
        const float alpha = raise ? ex2(m - m_new) : 1.f;
        l *= alpha;
        m = m_new;
        if (j > 0) {
          failed = !wait_w(&p_empty[(j - 1) & 1], static_cast<uint32_t>((j - 1) >> 1) & 1u);
          if (!failed) {
            tc_fence_after();
            const uint32_t oaddr = tmem_base + lane_base + kColO + wg * kOH;
#pragma unroll
            for (int c = 0; c < kOH; c += 16) {
              float x[16];
              tmem_ld16(oaddr + c, x);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] *= alpha;
              tmem_st16(oaddr + c, x);
            }
            tmem_wait_st();
          }
        }
      }
      const float sub = m == -INFINITY ? 0.f : m - kBias;
      uint32_t pk[kHalf / 2];
      if (!idle) {
#pragma unroll
        for (int c = 0; c < kHalf; c += 2) {
          const float a = ex2(s[c] - sub), b = ex2(s[c + 1] - sub);
          l += a + b;
          pk[c / 2] = pack_f16(a, b);
        }
      }
      if (!failed && j > 1) failed = !wait_w(&p_empty[j & 1], (static_cast<uint32_t>(j >> 1) & 1u) ^ 1u);
      if (failed) {
        go = false;
        *abort_flag = 1;
        continue;
      }
      if (!idle) {
        tmem_st32(tmem_base + lane_base + kColP + static_cast<uint32_t>((j & 1) * (kKeys / 2) + wg * 32), pk);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[j & 1]);
    }
    red[wg][row] = l;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    l = red[0][row] + red[1][row];
    float* sO = reinterpret_cast<float*>(sStage);
    const bool have = go && nt > 0 && wait_w(o_done, 0);
    if (have) tc_fence_after();
    if (!idle) {
      float* dst = sO + row * L::kOPitch + wg * kOH;
#pragma unroll
      for (int c = 0; c < kOH; c += 16) {
        float x[16];
        if (have) {
          tmem_ld16(tmem_base + lane_base + kColO + wg * kOH + c, x);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(dst + c + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
      }
      if (wg == 0) s_ml[row] = make_float2(m, have ? l : 0.f);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    constexpr int kE = DH / 32;
    for (int rr = warp; rr < live; rr += kSoftmaxWarps) {
      const float2 ml = s_ml[rr];
      const float* v = sO + rr * L::kOPitch + lane * kE;
      if (p.n_split > 1) {
        float* dst = cache_part_row(p, r, hk, mt, split, rr);
#pragma unroll
        for (int e = 0; e < kE; e += 2)
          *reinterpret_cast<float2*>(dst + 2 + lane * kE + e) = make_float2(v[e], v[e + 1]);
        if (lane == 0) *reinterpret_cast<float2*>(dst) = ml;
      } else {
        const float inv = ml.y > 0.f ? p.c.v_scale / ml.y : 0.f;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.O + cache_out_row(p, r, hk, q0 + rr) + lane * kE);
#pragma unroll
        for (int e = 0; e < kE; e += 2) dst[e / 2] = pack_bf16(v[e] * inv, v[e + 1] * inv);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem_base);
  }
}

}  // namespace

cudaError_t launch_cache_tree(const CacheAttnParams& p, cudaStream_t st) {
  const dim3 grid(p.m_tiles * p.n_split, p.c.Hkv, p.R);
  static std::atomic<uint64_t> done128{0}, done64{0};
  cudaError_t e = p.c.dh == 128 ? opt_in_smem(k_cache_tree<128>, &done128) : opt_in_smem(k_cache_tree<64>, &done64);
  if (e != cudaSuccess) return e;
  return launch_kernel(p.c.dh == 128 ? k_cache_tree<128> : k_cache_tree<64>, grid, dim3(kTreeThreads),
                       (p.c.dh == 128 ? TreeSmem<128>::kTotal : TreeSmem<64>::kTotal) + 1024, st, false, p);
}

}  // namespace dt
