// Attention of draft trees over the paged 4-bit cache on the 5th-generation
// tensor cores (dartree_cache_attention with more than 16 query rows per
// key/value head).
//
// A CTA owns up to 256 query rows of one request and one key/value head, as
// two tiles of 128 (a TMEM lane each), up to 8 more ("tail": a tree of 2^k
// nodes and its root are a few rows more than whole tiles), and a share of
// the key range in tiles of 128 keys.  Warp roles (512 threads):
//   0-3, 4-7  softmax of the two row tiles: a thread owns a row;
//   8-11      expand: codes and scales from memory to fp16 keys and values in
//             shared memory (exact), a tile ahead in registers;
//   12-13     the tail rows, by mma.sync on the same fp16 tiles, half of a
//             tile's keys each;
//   14, 15    issue the MMAs of one row tile each (14 owns the TMEM): what
//             waits on the issue all wait for, and two warps issue twice as fast.
// In steps of 64 keys: S = Q K^T (M 128, N 64, fp16, fp32 sums) into TMEM,
// double-buffered per row tile, P = 2^(s - m + kBias) in fp16 over the S
// columns it came from, O += P V with P from TMEM; S runs a step ahead of P.
// Keys and values lie in shared memory in the same layout (a token's
// row of 64 head dimensions is a 128-byte swizzled line): for S it is a
// K-major operand, for O the same lines are MN-major (the transposed read is
// the tensor core's).
// The running maximum is a reference that rises only when a score passes it
// by kRaise, which rescales O in TMEM.
// Requests go to the SMs longest first (the CTA's request is the z-th
// longest), so that the last ones to start are the short ones.
#include <type_traits>

#include "cache_attn.cuh"

namespace dt {
namespace {

constexpr int kMRows = 128, kKeys = 128, kStepKeys = 64;
constexpr int kExpandWarp0 = 8, kExpandWarps = 4, kTailWarp0 = 12, kMmaWarp0 = 14;
constexpr int kTreeThreads = 16 * 32;
constexpr int kStages = 2;
// (a tile's keys are expanded after all scores of the tile two before are
// issued, and they after the weights of the tile three before are there)
constexpr int kValid = 4;
constexpr int kTail = kTreeTail;
constexpr int kTreeSorted = 256;  // requests that are taken longest first (each CTA ranks them: R^2 / 512 steps)
constexpr uint32_t kTmemCols = 512;  // S of row tile i, buffer b: 128 i + 64 b; O of row tile i: 256 + 128 i; P over S
constexpr uint32_t kColO = 256;

template <int DH>
struct TreeSmem {
  static constexpr int kTile = kKeys * DH * 2;           // fp16 keys or values of a tile
  static constexpr int kQTile = kMRows * DH * 2;
  static constexpr int kStage = 2 * kQTile;              // stage s: keys, values
  static constexpr int kBars = kStage + kStages * 2 * kTile;
  static constexpr int kTotal = kBars + 256;
};

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of a converged warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

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

// 32 consecutive columns of the thread's lane (no wait: tmem_wait_ld).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
}

// Pairs of fp32 in one operand (two lanes of the fp32 pipe per instruction).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Codes and scales are read once: past L1.
__device__ __forceinline__ uint4 ld_once16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_once8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Which of the 32 keys from position pos on a row sees: the prefix, and the
// nodes of its mask row (null: none), before the keys' own bits.
__device__ __forceinline__ uint32_t row_sees(int pos, int Lp, const uint32_t* mrow, int words) {
  if (pos + 32 <= Lp) return ~0u;
  const int np = pos < Lp ? Lp - pos : 0, tf = pos > Lp ? pos - Lp : 0;
  uint32_t w0 = 0, w1 = 0;
  if (mrow) {
    const int wb = tf >> 5;
    if (wb < words) w0 = __ldg(mrow + wb);
    if (wb + 1 < words) w1 = __ldg(mrow + wb + 1);
  }
  const uint32_t nodes = __funnelshift_r(w0, w1, tf & 31);
  return (nodes << np) | ((1u << np) - 1u);
}

// A query row: its factor to base 2 and its power of two (bf16 words w).
__device__ __forceinline__ float row_exponent(float top, float scale_log2, float* down) {
  int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  e = top > 0.f ? max(-100, min(e, 100)) : 0;
  *down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  return scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

template <int DH>
__global__ void __launch_bounds__(kTreeThreads, 1) k_cache_tree(const CacheAttnParams p) {
  using L = TreeSmem<DH>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sStage = smem + L::kStage;
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + L::kBars);
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;  // [row tile][buffer]
  uint64_t* p_full = s_full + 4;         // [row tile][buffer]
  uint64_t* o_full = p_full + 4;         // [row tile][buffer]: P V of a step has landed
  uint64_t* mma_done = o_full + 4;       // [row tile]: everything issued has
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ __align__(16) uint8_t s_valid[kValid][kKeys / 8];  // bit k of a tile: key k is there
  __shared__ float s_tail[kTail][DH + 2];                       // the second tail warp's rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  const int mt = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split;
  __shared__ int s_r;
  if (p.R > 1 && p.R <= kTreeSorted) {  // the z-th longest request
    for (int a = threadIdx.x; a < p.R; a += kTreeThreads) {
      const int len = p.lens[a];
      int before = 0;
      for (int b = 0; b < p.R; ++b) {
        const int other = __ldg(p.lens + b);
        before += other > len || (other == len && b < a);
      }
      if (before == static_cast<int>(blockIdx.z)) s_r = a;
    }
    __syncthreads();
  }
  const int r = p.R > 1 && p.R <= kTreeSorted ? s_r : blockIdx.z;
  Span sp;
  if (!request_span(p, r, &sp)) return;
  const int q0 = mt * kTreeRowsCta;
  int live = (sp.n + 1) * p.g - q0;              // rows of this CTA: 256, and the tail in the last
  if (live > kTreeRowsCta + kTail) live = kTreeRowsCta;
  if (live <= 0 || (mt > 0 && live <= kTail)) return;  // (the tile before has them as its tail)
  const int t_all = row_tile_keys(p, sp, mt);
  const int t_beg = split * p.split_tiles;
  const int nt = min(t_all, t_beg + p.split_tiles) - t_beg;
  if (nt <= 0 && !(split == 0 && p.n_split == 1)) return;
  // steps of 64 keys (the last tile may need one only)
  const int steps = nt > 0 ? min(2 * nt, (sp.L - t_beg * kKeys + kStepKeys - 1) / kStepKeys) : 0;
  const int odd = live % kMRows;
  const int tail = live > kMRows && odd <= kTail ? odd : 0;
  const int rows = live - tail;                  // by the tensor cores' two tiles
  const int two = rows > kMRows ? 2 : 1;

  if (warp == kMmaWarp0) tmem_alloc<kTmemCols>(tmem_slot);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], kExpandWarps);
      mbar_init(&k_empty[s], two + (tail ? 2 : 0));
      mbar_init(&v_full[s], kExpandWarps);
      mbar_init(&v_empty[s], two + (tail ? 2 : 0));
    }
    for (int i = 0; i < 2; ++i) {
      const int n = min(rows - i * kMRows, kMRows);  // one arrival per warp with rows
      for (int b = 0; b < 2; ++b) {
        mbar_init(&s_full[2 * i + b], 1);
        mbar_init(&p_full[2 * i + b], n > 0 ? (n + 31) / 32 : 1);
        mbar_init(&o_full[2 * i + b], 1);
      }
      mbar_init(&mma_done[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    if (split == 0 && hk == 0 && mt == 0 && static_cast<long long>(p.lens[r]) + sp.n > p.max_len)
      atomicOr(p.err, DT_ERR_BAD_INDEX);
  }
  // the queries, as fp16 rows scaled by a power of two to at most 2 each
  float fac = 1.f;
  if (threadIdx.x < 2 * kMRows && threadIdx.x < two * kMRows) {
    const int row = threadIdx.x, q = q0 + row;
    const bool on = row < rows;
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
    float down;
    fac = row_exponent(top, p.scale_log2, &down);
    uint8_t* dst = smem + (row >> 7) * L::kQTile;
#pragma unroll
    for (int k = 0; k < DH / 8; ++k) {
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = pack_f16(__uint_as_float(x[j] << 16) * down, __uint_as_float(x[j] & 0xFFFF0000u) * down);
      *reinterpret_cast<uint4*>(dst + (k >> 3) * (kMRows * 128) + sw128(row & 127, k & 7)) =
          make_uint4(y[0], y[1], y[2], y[3]);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // a bounded wait of the whole warp; false: give up (another warp has, or
  // the time is over)
  auto wait_w = [&](uint64_t* bar, uint32_t par) {
    const uint32_t addr = smem_u32(bar);
    bool ok = mbar_try_wait(addr, par);
    if (!ok) {
      const long long t0 = clock64();
      while (!(ok = mbar_try_wait(addr, par)) && !*abort_flag)
        if (clock64() - t0 > kWaitLimitCycles) {
          atomicOr(p.err, DT_ERR_TIMEOUT);
          break;
        }
    }
    return __all_sync(kFullMask, ok) != 0;
  };

  if (warp >= kExpandWarp0 && warp < kTailWarp0) {
    // ------------------------------------------------- codes to fp16 tiles
    // Lane (key = lane / 4, c = lane % 4) of a warp's 8 keys takes the dims
    // [c DH/4, (c+1) DH/4): one load of codes, two (one) scales, DH/32 lines
    // of 16 bytes.  The lanes of c >= 2 write theirs in another order: the
    // eight lanes of a store's phase then lie in eight different 16-byte
    // columns.  A tile's codes are loaded while the one before is expanded,
    // its pages' numbers a tile earlier still.
    constexpr int kIt = kKeys / (kExpandWarps * 8);
    const int ew = warp - kExpandWarp0, kl = lane >> 2, c = lane & 3;
    const int P = 1 << p.c.log_page;
    const int32_t* trow = p.table + static_cast<size_t>(r) * p.max_pages;
    const uint8_t* head = p.c.pool + static_cast<size_t>(hk) * p.c.chunk;
    const int half = p.c.chunk >> 1;
    using Codes = typename std::conditional<DH == 128, uint4, uint2>::type;
    Codes code[2][kIt];
    uint32_t scl[2][kIt];
    int page[kIt];
    bool flagged = false;
    auto key_of = [&](int f, int it) { return (t_beg + f) * kKeys + (it * kExpandWarps + ew) * 8 + kl; };
    auto look_up = [&](int f) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int key = key_of(f, it), slot = key >> p.c.log_page;
        page[it] = -1;
        if (f < nt && key < sp.L) {
          if (slot < p.max_pages) page[it] = trow[slot];
          if (page[it] < 0 || page[it] >= p.c.pages) {
            page[it] = -1;
            if (!flagged) atomicOr(p.err, DT_ERR_BAD_INDEX);
            flagged = true;
          }
        }
      }
    };
    auto fetch = [&](int f, int kv) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        scl[kv][it] = 0;
        code[kv][it] = Codes{};
        if (page[it] >= 0) {
          const int t = key_of(f, it) & (P - 1);
          const uint8_t* chunk = head + static_cast<size_t>(page[it]) * p.c.page_bytes + kv * half;
          if constexpr (DH == 128) {
            code[kv][it] = ld_once16(chunk + t * 64 + c * 16);
            scl[kv][it] = *reinterpret_cast<const uint16_t*>(chunk + P * 64 + t * 8 + c * 2);
          } else {
            code[kv][it] = ld_once8(chunk + t * 32 + c * 8);
            scl[kv][it] = chunk[P * 32 + t * 4 + c];
          }
        }
      }
    };
    uint8_t there[2];  // bits of the warp's groups of 8 keys: this tile's (lane it), the next one's
    auto note = [&](int slot) {
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        uint32_t x = __ballot_sync(kFullMask, page[it] >= 0) & 0x11111111u;  // (lane 4 k: key k)
        x = (x | x >> 3) & 0x03030303u;
        x = (x | x >> 6) & 0x000F000Fu;
        x = (x | x >> 12) & 0xFFu;
        if (lane == it) there[slot] = static_cast<uint8_t>(x);
      }
    };
    look_up(0);
    fetch(0, 0);
    fetch(0, 1);
    note(0);
    look_up(1);
    bool go = true;
    for (int f = 0; f < nt && go; ++f) {
      const int st = f % kStages;
      const uint32_t ph = static_cast<uint32_t>((f / kStages) & 1);
      note(1);  // (of tile f + 1)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (f >= kStages && !wait_w(kv == 0 ? &k_empty[st] : &v_empty[st], ph ^ 1u)) {
          go = false;
          break;
        }
        if (kv == 0 && lane < kIt) s_valid[f % kValid][lane * kExpandWarps + ew] = there[0];
        uint8_t* dst = sStage + st * 2 * L::kTile + kv * L::kTile;
#pragma unroll
        for (int it = 0; it < kIt; ++it) {
          const int key = (it * kExpandWarps + ew) * 8 + kl;
          uint32_t w[DH / 32], sc[2];
          const uint32_t* cw = reinterpret_cast<const uint32_t*>(&code[kv][it]);
#pragma unroll
          for (int i = 0; i < DH / 32; ++i) w[i] = cw[i];
          if constexpr (DH == 128) {
            const uint32_t s2 = e4m3x2_to_f16x2(scl[kv][it]);
            sc[0] = __byte_perm(s2, s2, 0x1010);
            sc[1] = __byte_perm(s2, s2, 0x3232);
            if (c & 2) {  // the lines in the order 2, 3, 0, 1
              uint32_t x = w[0];
              w[0] = w[2];
              w[2] = x;
              x = w[1];
              w[1] = w[3];
              w[3] = x;
              x = sc[0];
              sc[0] = sc[1];
              sc[1] = x;
            }
          } else {
            sc[0] = sc[1] = e4m3x2_to_f16x2(scl[kv][it] | (scl[kv][it] << 8));
          }
          uint8_t* line = dst + (DH == 128 ? (c >> 1) * (kKeys * 128) : 0);
#pragma unroll
          for (int i = 0; i < DH / 32; ++i) {
            const int gr = DH == 128 ? ((c & 1) << 2) + (i ^ (c & 2)) : (c << 1) + i;
            uint32_t y[4];
            e2m1x8_to_f16(w[i], y);
            const uint32_t s2 = sc[DH == 128 ? i >> 1 : 0];
            *reinterpret_cast<uint4*>(line + sw128(key, gr)) =
                make_uint4(h2mul(y[0], s2), h2mul(y[1], s2), h2mul(y[2], s2), h2mul(y[3], s2));
          }
        }
        fetch(f + 1, kv);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(kv == 0 ? &k_full[st] : &v_full[st]);
      }
      there[0] = there[1];
      look_up(f + 2);
    }
    if (!go && lane == 0) *abort_flag = 1;
  } else if (warp >= kMmaWarp0 && warp - kMmaWarp0 < two) {
    // --------------------------------------------------------- MMA issuers
    constexpr uint32_t idesc_s = idesc_f16(kStepKeys, false), idesc_o = idesc_f16(DH, true);
    const int i = warp - kMmaWarp0;
    const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + i * L::kQTile));
    const uint64_t k_desc = smem_desc_sw128(smem_u32(sStage));
    const uint64_t v_desc = smem_desc_mn(smem_u32(sStage + L::kTile), kKeys * 128);
    const uint32_t s_col = tmem_base + static_cast<uint32_t>(i * kKeys);
    const uint32_t o_col = tmem_base + kColO + static_cast<uint32_t>(i * 128);
    const bool elected = elect_one();
    bool go = true;
    for (int u = -2; u < steps; ++u) {  // (a step's scores two steps ahead of its products)
      if (u >= 0) {  // O += P V of step u
        const int f = u >> 1, st = f % kStages, b = u & 1;
        if (!(go = wait_w(&p_full[2 * i + b], static_cast<uint32_t>(f) & 1u))) break;
        if (b == 0 && !(go = wait_w(&v_full[st], static_cast<uint32_t>((f / kStages) & 1)))) break;
        tc_fence_after();
        if (elected) {
          const uint64_t vd = v_desc + static_cast<uint64_t>(st * (2 * L::kTile >> 4) + b * (kStepKeys * 128 >> 4));
          const uint32_t pa = s_col + static_cast<uint32_t>(b * kStepKeys);
#pragma unroll
          for (int kk = 0; kk < kStepKeys / 16; ++kk)  // 16 keys: two atoms of 8 lines
            tc_mma_bf16_ta(o_col, pa + static_cast<uint32_t>(kk * 8), vd + static_cast<uint64_t>(kk * (2048 >> 4)),
                           idesc_o, (u != 0 || kk != 0) ? 1u : 0u);
          tc_commit(&o_full[2 * i + b]);
          if (b == 1 || u == steps - 1) tc_commit(&v_empty[st]);
        }
        __syncwarp();
      }
      if (u + 2 < steps) {  // S of step u + 2, over P(u), which the product just issued has read
        const int f = (u + 2) >> 1, st = f % kStages, b = u & 1;
        if (b == 0 && !(go = wait_w(&k_full[st], static_cast<uint32_t>((f / kStages) & 1)))) break;
        tc_fence_after();
        if (elected) {
          // (descriptors count in 16 bytes: 16 dims are 2, the next 64 dims a
          // tile's lines, 64 keys half of them)
          const uint64_t kd = k_desc + static_cast<uint64_t>(st * (2 * L::kTile >> 4) + b * (kStepKeys * 128 >> 4));
          const uint32_t col = s_col + static_cast<uint32_t>(b * kStepKeys);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            constexpr uint64_t kAtom = kKeys * 128 >> 4;
            const uint64_t off = (kk & 3) * 2 + (kk >> 2) * kAtom;
            tc_mma_bf16(col, q_desc + off, kd + off, idesc_s, kk != 0 ? 1u : 0u);
          }
          tc_commit(&s_full[2 * i + b]);
          if (b == 1 || u + 2 == steps - 1) tc_commit(&k_empty[st]);
        }
        __syncwarp();
      }
    }
    if (!go && lane == 0) *abort_flag = 1;
    if (elected) {  // what was issued has landed before the block may end
      tc_commit(&mma_done[i]);
      mbar_wait(&mma_done[i], 0, p.err);
    }
    __syncwarp();
  } else if (warp < kExpandWarp0 && warp * 32 < rows) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2, row = threadIdx.x, q = q0 + row;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(i * kKeys);
    const uint32_t o_addr = tmem_base + lane_base + kColO + static_cast<uint32_t>(i * 128);
    const int node = row < rows ? q / p.g : 0;
    const uint32_t* mrow = node >= 1 ? p.mask + (static_cast<size_t>(r) * p.B + node - 1) * p.words : nullptr;
    float m = -INFINITY, l = 0.f;
    float limit = -INFINITY;  // the unscaled score above which the reference rises
    bool go = true;
    for (int u = 0; u < steps; ++u) {
      const int f = u >> 1, b = u & 1, key0 = t_beg * kKeys + u * kStepKeys;
      if (!(go = wait_w(&s_full[2 * i + b], static_cast<uint32_t>(f) & 1u))) break;
      tc_fence_after();
      uint32_t x[kStepKeys];
      tmem_ld64(s_addr + b * kStepKeys, x);
      const uint2 there = *reinterpret_cast<const uint2*>(&s_valid[f % kValid][b * (kStepKeys / 8)]);
      tmem_wait_ld();
      if (key0 + kStepKeys > sp.Lp || (there.x & there.y) != ~0u) {  // -inf where not seen
        const uint32_t lo = row_sees(key0, sp.Lp, mrow, p.words) & there.x;
        const uint32_t hi = row_sees(key0 + 32, sp.Lp, mrow, p.words) & there.y;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if (!((lo >> k) & 1u)) x[k] = 0xFF800000u;
          if (!((hi >> k) & 1u)) x[32 + k] = 0xFF800000u;
        }
      }
      float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int k = 0; k < kStepKeys; k += 2)
        t[(k >> 1) & 3] = fmaxf(t[(k >> 1) & 3], fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 1])));
      const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
      if (__any_sync(kFullMask, top > limit)) {
        float alpha = 1.f;
        if (top > limit) {
          const float y = top * fac;
          alpha = ex2(m - y);  // (0 from -inf)
          m = y;
          limit = __fdividef(y + kRaise, fac);
          l *= alpha;
        }
        if (u > 0) {
          // O holds the products of the steps before, once the last has landed
          // (the scores of this step came after the one of u - 2, and the
          // barrier of u - 1 is that of u - 3: its parity is certain)
          if (!(go = wait_w(&o_full[2 * i + (b ^ 1)], static_cast<uint32_t>((u - 1) >> 1) & 1u))) break;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < DH / 16; ++ch) {
            float y[16];
            tmem_ld16(o_addr + ch * 16, y);
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] *= alpha;
            tmem_st16(o_addr + ch * 16, y);
          }
        }
      }
      // the weights, over the columns their scores came from
      const float sub = m == -INFINITY ? 0.f : kBias - m;
      const uint64_t fac2 = pack2(fac, fac), sub2 = pack2(sub, sub);
      uint64_t sum[2] = {0ull, 0ull};
      uint32_t pk[kStepKeys / 2];
#pragma unroll
      for (int k = 0; k < kStepKeys; k += 2) {
        float a, c;
        unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), fac2, sub2), a, c);
        a = ex2(a);
        c = ex2(c);
        sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, c));
        pk[k / 2] = pack_f16(a, c);
      }
      tmem_st32(s_addr + b * kStepKeys, pk);
      float a, c;
      unpack2(add2(sum[0], sum[1]), a, c);
      l += a + c;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * i + b]);
    }
    if (!go && lane == 0) *abort_flag = 1;
    const bool have = go && steps > 0 && wait_w(&mma_done[i], 0);
    if (have) tc_fence_after();
    else l = 0.f;
    const bool on = row < rows;
    const float inv = l > 0.f ? p.c.v_scale / l : 0.f;
    float* part = p.n_split > 1 && on ? cache_part_row(p, r, hk, mt, split, row) : nullptr;
    uint4* out = p.n_split > 1 || !on ? nullptr : reinterpret_cast<uint4*>(p.O + cache_out_row(p, r, hk, q));
    if (part) *reinterpret_cast<float2*>(part) = make_float2(m, l);
#pragma unroll
    for (int ch = 0; ch < DH / 32; ++ch) {
      uint32_t x[32];
      if (have) {
        tmem_ld32(o_addr + ch * 32, x);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = 0u;
      }
      if (part) {
#pragma unroll
        for (int k = 0; k < 32; k += 2)
          *reinterpret_cast<float2*>(part + 2 + ch * 32 + k) =
              make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
      }
      if (out) {
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          uint32_t y[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            y[u] = pack_bf16(__uint_as_float(x[k + 2 * u]) * inv, __uint_as_float(x[k + 2 * u + 1]) * inv);
          out[ch * 4 + k / 8] = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
    }
  } else if ((warp == kTailWarp0 || warp == kTailWarp0 + 1) && tail > 0) {
    // ------------------------------------------------------------ tail rows
    // S^T = K Q^T and O^T += V^T P^T by mma m16n8k16 with the tiles' keys as
    // the 16-row operand (as the kernel of few rows does from the codes).  The
    // loops run over independent sums inside.
    const int rr = lane >> 2, c = lane & 3, tw = warp - kTailWarp0;
    constexpr int kSteps = DH / 16, kGroups = kKeys / 32;  // 16-key groups of this warp
    uint32_t qb[kSteps][2];
    float tf[2];
    int nd[2];
    {
      const bool on = rr < tail;
      const int q = q0 + rows + (on ? rr : 0), n = q / p.g;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.Q + (static_cast<size_t>(r) * (p.B + 1) + n) * p.q_stride +
          static_cast<size_t>(hk * p.g + (q - n * p.g)) * DH);
      float top = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          qb[s][h] = on ? __ldg(src + 8 * s + 4 * h + c) : 0u;  // dims 16 s + 8 h + 2 c, + 1
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(qb[s][h] << 16)), fabsf(__uint_as_float(qb[s][h] & 0xFFFF0000u))));
        }
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      float down;
      const float f = row_exponent(top, p.scale_log2, &down);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          qb[s][h] = pack_f16(__uint_as_float(qb[s][h] << 16) * down, __uint_as_float(qb[s][h] & 0xFFFF0000u) * down);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tf[x] = __shfl_sync(kFullMask, f, (2 * c + x) * 4);
        nd[x] = __shfl_sync(kFullMask, n, (2 * c + x) * 4);
      }
    }
    float o[kSteps][4];  // dims 16 s + rr, + 8 of rows 2 c, 2 c + 1
#pragma unroll
    for (int s = 0; s < kSteps; ++s) o[s][0] = o[s][1] = o[s][2] = o[s][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, limit[2] = {-INFINITY, -INFINITY};
    const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: row lr of matrix lm
    bool go = true;
    for (int j = 0; j < nt; ++j) {
      const int st = j % kStages, key0 = (t_beg + j) * kKeys + tw * (kKeys / 2);
      const uint32_t ph = static_cast<uint32_t>((j / kStages) & 1);
      if (!(go = wait_w(&k_full[st], ph))) break;
      const uint32_t k_addr = smem_u32(sStage + st * 2 * L::kTile), v_addr = k_addr + L::kTile;
      const uint2 there = *reinterpret_cast<const uint2*>(&s_valid[j % kValid][tw * (kKeys / 16)]);
      const bool plain = key0 + kKeys / 2 <= sp.Lp && (there.x & there.y) == ~0u;
      float s[kGroups][4];
#pragma unroll
      for (int g = 0; g < kGroups; ++g) s[g][0] = s[g][1] = s[g][2] = s[g][3] = 0.f;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int gr = 2 * k + (lm >> 1);  // matrices: keys 0-7 | 8-15, dims 0-7; the same, dims 8-15
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          uint32_t a[4];
          const int key = tw * (kKeys / 2) + 16 * g + lr + 8 * (lm & 1);
          ldmatrix_x4(k_addr + (gr >> 3) * (kKeys * 128) + sw128(key, gr & 7), a);
          mma_f16(s[g], a, qb[k][0], qb[k][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[st]);
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!plain) {
            const int kk = 16 * g + 8 * (x >> 1) + rr, pos = key0 + kk;
            bool seen = ((g < 2 ? there.x : there.y) >> (kk & 31)) & 1u;
            if (seen && pos >= sp.Lp) {
              const int t = pos - sp.Lp, n = nd[x & 1];
              seen = n > 0 &&
                     ((__ldg(p.mask + (static_cast<size_t>(r) * p.B + n - 1) * p.words + (t >> 5)) >> (t & 31)) & 1u);
            }
            if (!seen) s[g][x] = -INFINITY;
          }
          top[x & 1] = fmaxf(top[x & 1], s[g][x]);
        }
      if (__any_sync(kFullMask, top[0] > limit[0] || top[1] > limit[1])) {
        float al[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = top[x];
#pragma unroll
          for (int d = 4; d < 32; d *= 2) t = fmaxf(t, __shfl_xor_sync(kFullMask, t, d));
          al[x] = 1.f;
          if (t > limit[x]) {
            t *= tf[x];
            al[x] = ex2(m[x] - t);
            m[x] = t;
            limit[x] = __fdividef(t + kRaise, tf[x]);
            l[x] *= al[x];
          }
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          o[k][0] *= al[0];
          o[k][1] *= al[1];
          o[k][2] *= al[0];
          o[k][3] *= al[1];
        }
      }
      const float sub0 = m[0] == -INFINITY ? 0.f : kBias - m[0], sub1 = m[1] == -INFINITY ? 0.f : kBias - m[1];
      uint32_t pb[kGroups][2];
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float p0 = ex2(fmaf(s[g][2 * t], tf[0], sub0)), p1 = ex2(fmaf(s[g][2 * t + 1], tf[1], sub1));
          l[0] += p0;
          l[1] += p1;
          pb[g][t] = transpose8x8(pack_f16(p0, p1));
        }
      if (!(go = wait_w(&v_full[st], ph))) break;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int key = tw * (kKeys / 2) + 16 * g + lr + 8 * (lm >> 1);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          const int gr = 2 * k + (lm & 1);  // matrices: dims 0-7 | 8-15, keys 0-7; the same, keys 8-15
          ldmatrix_x4_trans(v_addr + (gr >> 3) * (kKeys * 128) + sw128(key, gr & 7), a);
          mma_f16(o[k], a, pb[g][0], pb[g][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_empty[st]);
    }
    if (!go && lane == 0) *abort_flag = 1;
    // the second warp's rows to the first, which joins them
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[x] += __shfl_xor_sync(kFullMask, l[x], d);
      if (tw == 1) {
        float* dst = s_tail[2 * c + x];
        if (rr == 0) {
          dst[DH] = m[x];
          dst[DH + 1] = l[x];
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          dst[16 * k + rr] = o[k][x];
          dst[16 * k + 8 + rr] = o[k][2 + x];
        }
      }
    }
    asm volatile("bar.sync 1, 64;" ::: "memory");
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int row = 2 * c + x;
      if (tw == 1 || row >= tail) continue;
      const float* other = s_tail[row];
      const float M = fmaxf(m[x], other[DH]);
      const float f0 = m[x] == -INFINITY ? 0.f : ex2(m[x] - M), f1 = other[DH] == -INFINITY ? 0.f : ex2(other[DH] - M);
      const float Lr = l[x] * f0 + other[DH + 1] * f1;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        o[k][x] = o[k][x] * f0 + other[16 * k + rr] * f1;
        o[k][2 + x] = o[k][2 + x] * f0 + other[16 * k + 8 + rr] * f1;
      }
      if (p.n_split > 1) {
        float* dst = cache_part_row(p, r, hk, mt, split, rows + row);
        if (rr == 0) *reinterpret_cast<float2*>(dst) = make_float2(M, Lr);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          dst[2 + 16 * k + rr] = o[k][x];
          dst[2 + 16 * k + 8 + rr] = o[k][2 + x];
        }
      } else {
        const float inv = Lr > 0.f ? p.c.v_scale / Lr : 0.f;
        uint16_t* dst = p.O + cache_out_row(p, r, hk, q0 + rows + row);
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          dst[16 * k + rr] = float_to_bf16_bits(o[k][x] * inv);
          dst[16 * k + 8 + rr] = float_to_bf16_bits(o[k][2 + x] * inv);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp0) {
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
