// Attention of draft trees over the paged 4-bit cache on the 5th-generation
// tensor cores (dartree_cache_attention with more than 16 query rows per
// key/value head).
//
// A CTA owns up to 256 query rows of one request and one key/value head, as
// two tiles of 128 (a TMEM lane each), and a share of the key range in tiles
// of 128 keys.  Warp roles (832 threads):
//   0-7, 8-15  softmax of the two row tiles: two threads share a row, each
//              has half of a step's keys and of the head dimensions of O;
//   16-23      expand: codes and scales from memory to fp16 keys (16-19) and
//              values (20-23) in shared memory (exact), a tile ahead in
//              registers;
//   24, 25     issue the MMAs of one row tile each (24 owns the TMEM): what
//              waits on the issue all wait for, and two warps issue twice as
//              fast.
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
//
// Bound by the latency of a step's chain (scores, maximum, weights, product)
// at two row tiles per SM: 32 trees of 65 rows over up to 2500 tokens, 32 heads
// over 8 of 128: 73 us (76 in a graph), 730 TFLOP/s, the tensor pipe active 37% of the time,
// issue 0.62 (the exponentials and the conversions of the codes alone would
// take 29 us); one of 129 rows over 4099 tokens: 28 us.  Steps for the 32 (the
// one): one row tile 181 us (41); two, and codes expanded from registers 121
// (53); scores a step of 64 keys ahead and two issuers 85 (47); leftover rows in
// a launch beside 89 (43); two threads per row 83 (35); queries loaded by the
// softmax warps beside the first codes, output addresses out of the loop 77
// (31).  A polynomial for part of the exponentials and row tiles that take
// turns were slower (no figures kept).
#include <type_traits>

#include "cache_attn.cuh"

namespace dt {
namespace {

constexpr int kMRows = 128, kKeys = 128, kStepKeys = 64;
constexpr int kExpandWarp0 = 16, kExpandWarps = 8, kMmaWarp0 = 24;
constexpr int kLoadWarps = 8;  // that load a row tile's queries: its softmax warps
constexpr int kTreeThreads = 26 * 32;
constexpr int kStages = 2;
// (a tile's keys are expanded after all scores of the tile two before are
// issued, and they after the weights of the tile three before are there)
constexpr int kValid = 4;
constexpr int kTreeSorted = 256;  // requests that are taken longest first (each CTA ranks them: R^2 / 832 steps)
// A weight is 2^(s fac - m + kBias) with m = ref fac rounded, off by 2^-24 of
// itself.  Where it would pass kFar, whose unit is 1/2, the row goes on with the
// factor that puts it there: the weights of scores within 2^-18 of the largest
// then differ by less than they should, those of all others are 0 either way (a
// score's own sum in fp32 is off by as much).  Without it a weight passes fp16's
// range from 2^27 on; taking the distance s - ref first costs 4% of the time.
constexpr float kFar = 4194304.f;
constexpr uint32_t kTmemCols = 512;  // S of row tile i, buffer b: 128 i + 64 b; O of row tile i: 256 + 128 i; P over S
constexpr uint32_t kColO = 256;

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

// 32 consecutive columns of the thread's lane (one statement with its wait: no
// use of a value can come before it).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// A barrier of 64 threads that gives the OR of their predicates.
__device__ __forceinline__ bool barrier_or(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\t"
      "barrier.cta.red.or.aligned.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
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

// SHORT: with a limit of the waits (the form that a wait that runs out is tested with).
template <int DH, bool SHORT>
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
  uint64_t* q_full = mma_done + 2;       // [row tile]: the queries are there
  constexpr int kBarriers = 4 * kStages + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ float s_fac[2 * kMRows], s_top[2][2 * kMRows];  // of the rows: factor; by half: maximum, sum
  __shared__ float s_ref[2][2 * kMRows];                     // by half: the reference as a score
  __shared__ __align__(16) uint8_t s_valid[kValid][kKeys / 8];  // bit k of a tile: key k is there

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.y;
  const int mt = blockIdx.x / p.n_split, split = blockIdx.x % p.n_split;
  pdl_wait();
  pdl_trigger();  // (the launch of the rows left over may fill the SMs that come free)
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
  // rows of this CTA, without the few behind the request's last whole tile
  const int all = (sp.n + 1) * p.g;
  const int rows = min(all - tail_rows(all) - q0, kTreeRowsCta);
  if (rows <= 0) return;
  const int t_all = row_tile_keys(p, sp, mt);
  const int t_beg = split * p.split_tiles;
  const int nt = min(t_all, t_beg + p.split_tiles) - t_beg;
  if (nt <= 0 && !(split == 0 && p.n_split == 1)) return;
  // steps of 64 keys (the last tile may need one only)
  const int steps = nt > 0 ? min(2 * nt, (sp.L - t_beg * kKeys + kStepKeys - 1) / kStepKeys) : 0;
  const int two = rows > kMRows ? 2 : 1;

  if (warp == kMmaWarp0) tmem_alloc<kTmemCols>(tmem_slot);
  if (warp == 0) {
    static_assert(kStages == 2 && kBarriers <= 32, "a lane per barrier");
    if (lane < kBarriers) {
      int count = 1;                                      // s_full, o_full, mma_done
      if (lane < 8) count = lane & 2 ? two : kExpandWarps / 2;  // k_full, k_empty, v_full, v_empty
      if (lane >= 12 && lane < 16) {                      // p_full: one arrival per warp with rows
        const int n = min(rows - ((lane - 12) >> 1) * kMRows, kMRows);
        if (n > 0) count = 2 * ((n + 31) / 32);
      }
      if (lane >= 22) count = kLoadWarps;                 // q_full
      mbar_init(&k_full[lane], count);
      fence_mbar_init();
    }
    if (lane == 0) *abort_flag = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // a bounded wait of the whole warp; false: give up (another warp has, or
  // the time is over)
  auto wait_w = [&](uint64_t* bar, uint32_t par) {
    const uint32_t addr = smem_u32(bar);
    bool ok = poll<SHORT>(addr, par);
    if (!ok) {
      const long long t0 = clock64(), limit = SHORT ? p.wait_limit : kWaitLimitCycles;
      while (!(ok = poll<SHORT>(addr, par)) && !*abort_flag)
        if (clock64() - t0 > limit) {
          atomicOr(p.err, DT_ERR_TIMEOUT);
          break;
        }
    }
    return __all_sync(kFullMask, ok) != 0;
  };

  if (warp < two * kLoadWarps) {
    // the queries, as fp16 rows scaled by a power of two to at most 2 each: a
    // warp takes 16 rows, DH / 8 lanes a row, all loads before their use (a
    // thread per row: 9400 cycles)
    constexpr int kRowLanes = DH / 8, kRowsIt = 32 / kRowLanes, kIts = kMRows / kLoadWarps / kRowsIt;
    const int k = lane % kRowLanes, first = warp * (kMRows / kLoadWarps) + lane / kRowLanes;
    uint4 w[kIts];
#pragma unroll
    for (int j = 0; j < kIts; ++j) {
      const int row = first + j * kRowsIt, q = q0 + row, node = row < rows ? q / p.g : 0;
      w[j] = make_uint4(0, 0, 0, 0);
      if (row < rows)
        w[j] = __ldg(reinterpret_cast<const uint4*>(
                         p.Q + (static_cast<size_t>(r) * (p.B + 1) + node) * p.q_stride +
                         static_cast<size_t>(hk * p.g + (q - node * p.g)) * DH) + k);
    }
    uint8_t* dst = smem + (warp / kLoadWarps) * L::kQTile + (k >> 3) * (kMRows * 128);
#pragma unroll
    for (int j = 0; j < kIts; ++j) {
      const int row = first + j * kRowsIt;
      const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[e] << 16)), fabsf(__uint_as_float(x[e] & 0xFFFF0000u))));
#pragma unroll
      for (int o = 1; o < kRowLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
      float down;
      const float fac = row_exponent(p, top, &down);
      if (k == 0) s_fac[row] = fac;
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = pack_f16(__uint_as_float(x[e] << 16) * down, __uint_as_float(x[e] & 0xFFFF0000u) * down);
      *reinterpret_cast<uint4*>(dst + sw128(row & 127, k & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&q_full[warp / kLoadWarps]);
  }

  if (warp >= kExpandWarp0 && warp < kMmaWarp0) {
    // ------------------------------------------------- codes to fp16 tiles
    // Four warps take the keys, four the values; a warp's it-th group is 8
    // tokens (of one page).  Lane (r = lane / 4, c = lane % 4) takes the dims
    // [c DH/4, (c+1) DH/4) of one of the 8: one load of codes, two (one)
    // scales, DH/32 lines of 16 bytes.  The lanes of c >= 2 take token r ^ 2
    // instead of r: the eight lanes of a store's phase then lie in eight
    // different 16-byte columns.  A group's codes are loaded when the same
    // group of the tile before has been expanded, the pages' numbers (lane
    // `it` has group it's) a tile earlier still.
    constexpr int kSub = kExpandWarps / 2, kIt = kKeys / (8 * kSub);
    const int ew = warp - kExpandWarp0, kv = ew / kSub, sub = ew % kSub;
    const int c = lane & 3, kl = (lane >> 2) ^ (c & 2);
    const int P = 1 << p.c.log_page;
    const int32_t* trow = p.table + static_cast<size_t>(r) * p.max_pages;
    const uint8_t* head = p.c.pool + static_cast<size_t>(hk) * p.c.chunk + kv * (p.c.chunk >> 1) + c * (DH / 8);
    const uint8_t* head_sc = head - c * (DH / 8) + P * (DH / 2) + c * (DH / 64);
    using Codes = typename std::conditional<DH == 128, uint4, uint2>::type;
    Codes code[kIt];
    uint32_t scl[kIt];
    auto group = [&](int f, int it) { return (t_beg + f) * kKeys + (it * kSub + sub) * 8; };  // its first token
    // lane it's page of tile f (not looked at before the next tile)
    auto look_up = [&](int f) {
      const int slot = group(f, lane) >> p.c.log_page;
      return lane < kIt && f < nt && slot < p.max_pages ? trow[slot] : -1;
    };
    // the page, or -1; the bits of the group's tokens that are there
    auto check = [&](int f, int raw, uint32_t* bits) {
      const int left = sp.L - group(f, lane);
      *bits = 0;
      if (lane >= kIt || f >= nt || left <= 0) return -1;
      if (raw < 0 || raw >= p.c.pages) {
        atomicOr(p.err, DT_ERR_BAD_INDEX);
        return -1;
      }
      *bits = left >= 8 ? 0xFFu : (1u << left) - 1u;
      return raw;
    };
    auto load = [&](int f, int page_of_lane, int it) {
      const int page = __shfl_sync(kFullMask, page_of_lane, it);
      scl[it] = 0;
      code[it] = Codes{};
      const int key = group(f, it) + kl;
      if (page >= 0 && key < sp.L) {
        const size_t at = static_cast<size_t>(page) * p.c.page_bytes;
        const int t = key & (P - 1);
        if constexpr (DH == 128) {
          code[it] = ld_once16(head + at + t * 64);
          scl[it] = *reinterpret_cast<const uint16_t*>(head_sc + at + t * 8);
        } else {
          code[it] = ld_once8(head + at + t * 32);
          scl[it] = head_sc[at + t * 4];
        }
      }
    };
    uint32_t bits, next_bits;
    int page = check(0, look_up(0), &bits);
#pragma unroll
    for (int it = 0; it < kIt; ++it) load(0, page, it);
    int raw = look_up(1);
    uint64_t* full = kv ? v_full : k_full;
    uint64_t* empty = kv ? v_empty : k_empty;
    bool go = true;
#pragma unroll 1
    for (int f = 0; f < nt; ++f) {
      const int st = f % kStages;
      if (f >= kStages && !(go = wait_w(&empty[st], static_cast<uint32_t>((f / kStages) & 1) ^ 1u))) break;
      if (kv == 0 && lane < kIt) s_valid[f % kValid][lane * kSub + sub] = static_cast<uint8_t>(bits);
      page = check(f + 1, raw, &next_bits);
      bits = next_bits;
      raw = look_up(f + 2);
      uint8_t* dst = sStage + (st * 2 + kv) * L::kTile + (DH == 128 ? (c >> 1) * (kKeys * 128) : 0);
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int key = (it * kSub + sub) * 8 + kl;
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&code[it]);
        uint32_t sc[2];
        if constexpr (DH == 128) {
          const uint32_t s2 = finite_scales(e4m3x2_to_f16x2(scl[it]));
          sc[0] = __byte_perm(s2, s2, 0x1010);
          sc[1] = __byte_perm(s2, s2, 0x3232);
        } else {
          sc[0] = sc[1] = finite_scales(e4m3x2_to_f16x2(scl[it] | (scl[it] << 8)));
        }
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          const int gr = DH == 128 ? ((c & 1) << 2) + i : (c << 1) + i;
          uint32_t y[4];
          e2m1x8_to_f16(w[i], y);
          const uint32_t s2 = sc[DH == 128 ? i >> 1 : 0];
          *reinterpret_cast<uint4*>(dst + sw128(key, gr)) =
              make_uint4(h2mul(y[0], s2), h2mul(y[1], s2), h2mul(y[2], s2), h2mul(y[3], s2));
        }
        load(f + 1, page, it);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
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
    bool go = wait_w(&q_full[i], 0);
    for (int u = -1; go && u < steps; ++u) {
      if (u + 1 < steps) {  // S of step u + 1, over P(u - 1) once its product has landed
        const int f = (u + 1) >> 1, st = f % kStages, b = (u + 1) & 1;
        if (u >= 1 && !(go = wait_w(&o_full[2 * i + b], static_cast<uint32_t>((u - 1) >> 1) & 1u))) break;
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
          if (b == 1 || u + 1 == steps - 1) tc_commit(&k_empty[st]);
        }
        __syncwarp();
      }
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
    }
    if (!go && lane == 0) *abort_flag = 1;
    if (elected) {  // what was issued has landed before the block may end
      tc_commit(&mma_done[i]);
      mbar_wait(&mma_done[i], 0, p.err);
    }
    __syncwarp();
  } else if (warp < kExpandWarp0 && (warp >> 3) * kMRows + (warp & 3) * 32 < rows) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int row = i * kMRows + quarter * 32 + lane, q = q0 + row;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem_base + lane_base + static_cast<uint32_t>(i * kKeys);
    const uint32_t o_addr = tmem_base + lane_base + kColO + static_cast<uint32_t>(i * 128 + half * (DH / 2));
    const int pair = 1 + i * 4 + quarter;  // the barrier of the two warps that share rows
    const int node = row < rows ? q / p.g : 0;
    const uint32_t* mrow = node >= 1 ? p.mask + (static_cast<size_t>(r) * p.B + node - 1) * p.words : nullptr;
    bool go = wait_w(&q_full[i], 0);  // (the same in both warps after every barrier)
    float fac = s_fac[row];
    float m = -INFINITY, l = 0.f;  // the row's reference (the same in both threads), this half's sum
    float& ref = s_ref[half][row]; // the reference as a score
    float limit = -INFINITY;       // the score above which the reference rises
    ref = -INFINITY;
    for (int u = 0; u < steps; ++u) {
      const int f = u >> 1, b = u & 1, key0 = t_beg * kKeys + u * kStepKeys + half * (kStepKeys / 2);
      go = go && wait_w(&s_full[2 * i + b], static_cast<uint32_t>(f) & 1u);
      tc_fence_after();
      const uint32_t there = *reinterpret_cast<const uint32_t*>(&s_valid[f % kValid][(2 * b + half) * 4]);
      uint32_t see = ~0u;
      if (key0 + 32 > sp.Lp || there != ~0u) see = row_sees(key0, sp.Lp, mrow, p.words) & there;
      // the weights with the reference as it is; where a score passes the
      // limit the reference rises and they are computed once more
      uint32_t pk[16];
      float add = 0.f;
      for (int round = 0;; ++round) {
        float top = -INFINITY;
        if (go) {
          uint32_t x[32];
          tmem_ld32(s_addr + b * kStepKeys + half * 32, x);
          if (__any_sync(kFullMask, see != ~0u)) {  // -inf where not seen
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((see >> k) & 1u)) x[k] = 0xFF800000u;
          }
          const float sub = m == -INFINITY ? 0.f : kBias - m;
          const uint64_t fac2 = pack2(fac, fac), sub2 = pack2(sub, sub);
          uint64_t sum[2] = {0ull, 0ull};
          float t[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float a = __uint_as_float(x[k]), c = __uint_as_float(x[k + 1]);
            t[(k >> 1) & 1] = fmaxf(t[(k >> 1) & 1], fmaxf(a, c));
            unpack2(fma2(pack2(a, c), fac2, sub2), a, c);
            a = ex2(a);
            c = ex2(c);
            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, c));
            pk[k / 2] = pack_f16(a, c);
          }
          float a, c;
          unpack2(add2(sum[0], sum[1]), a, c);
          add = a + c;
          top = fmaxf(t[0], t[1]);
        }
        // (every way on from here: both halves' scores are read, their columns
        // may be written)
        if (round > 0) {
          barrier_or(pair, false);
          break;
        }
        if (!barrier_or(pair, !go || top > limit)) break;
        s_top[half][row] = top;
        if (barrier_or(pair, !go)) {
          go = false;
          break;
        }
        top = fmaxf(s_top[0][row], s_top[1][row]);
        float alpha = 1.f;
        if (top > limit) {
          const float full = s_fac[row], y = top * full;
          alpha = ex2((ref - top) * full);  // (0 from -inf)
          ref = top;
          fac = fabsf(y) > kFar ? full * __fdividef(kFar, fabsf(y)) : full;
          m = top * fac;
          limit = rise_limit(top, fac);
          l *= alpha;
        }
        bool landed = true;
        if (u > 0) {
          // O holds the products of the steps before, once the last has landed
          // (the scores of this step came after the one of u - 2, and the
          // barrier of u - 1 is that of u - 3: its parity is certain)
          landed = wait_w(&o_full[2 * i + (b ^ 1)], static_cast<uint32_t>((u - 1) >> 1) & 1u);
          tc_fence_after();
          if (landed) {
#pragma unroll 1
            for (int ch = 0; ch < DH / 32; ++ch) {
              float y[16];
              tmem_ld16(o_addr + ch * 16, y);
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] *= alpha;
              tmem_st16(o_addr + ch * 16, y);
            }
          }
        }
        if (barrier_or(pair, !landed)) {  // (also: s_top may be written again)
          go = false;
          break;
        }
      }
      if (!go) break;
      l += add;
      tmem_st16(s_addr + b * kStepKeys + half * 16, reinterpret_cast<const float(&)[16]>(pk));
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[2 * i + b]);
    }
    if (!go) {  // (a rescaled output's stores end before the TMEM goes)
      if (lane == 0) *abort_flag = 1;
      tmem_wait_st();
    }
    s_top[half][row] = l;
    barrier_or(pair, false);
    l = s_top[0][row] + s_top[1][row];
    const bool have = go && steps > 0 && wait_w(&mma_done[i], 0);
    if (have) tc_fence_after();
    if (!have || m == -INFINITY) l = 0.f;
    const float inv = l > 0.f ? p.c.v_scale / l : 0.f;
    if (half == 0 && p.n_split > 1 && row < rows)
      *reinterpret_cast<float2*>(cache_part_row(p, r, hk, mt, split, row)) = make_float2(have ? ref * s_fac[row] : -INFINITY, l);
    // O by way of the row tile's queries' place in shared memory (the scores
    // are done), an eighth of the dims at a time, so that a warp's accesses are
    // whole pieces of rows: kC dims of a row by kC / 4 lanes
    constexpr int kC = DH / 8, kPitch = kC + 4, kLanes = kC / 4;
    float* stage = reinterpret_cast<float*>(smem + i * L::kQTile) + (warp & 7) * 32 * kPitch;
    static_assert(8 * 32 * kPitch * 4 <= L::kQTile, "the staged rows fit");
    const float mul = p.n_split > 1 ? 1.f : inv;
    // the lane's pieces of rows k = lane / kLanes, + 32 / kLanes, ..: where they
    // go, a chunk's step on (looked up once: in the loop 3000 cycles)
    uint8_t* to[kLanes];
#pragma unroll
    for (int j = 0; j < kLanes; ++j) {
      const int rr = i * kMRows + quarter * 32 + lane / kLanes + j * (32 / kLanes);
      const int d = half * (DH / 2) + (lane % kLanes) * 4;
      to[j] = nullptr;
      if (rr < rows)
        to[j] = p.n_split > 1 ? reinterpret_cast<uint8_t*>(cache_part_row(p, r, hk, mt, split, rr) + kPartHead + d)
                              : reinterpret_cast<uint8_t*>(p.O + cache_out_row(p, r, hk, q0 + rr) + d);
    }
#pragma unroll 1
    for (int ch = 0; ch < 4; ++ch) {
      float x[kC];
      if (have) {
        if constexpr (kC == 16) tmem_ld16(o_addr + ch * kC, x);
        else tmem_ld8(o_addr + ch * kC, x);
      } else {
#pragma unroll
        for (int k = 0; k < kC; ++k) x[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kC; k += 4)
        *reinterpret_cast<float4*>(stage + lane * kPitch + k) =
            make_float4(x[k] * mul, x[k + 1] * mul, x[k + 2] * mul, x[k + 3] * mul);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < kLanes; ++j) {
        const float4 v = *reinterpret_cast<const float4*>(stage + (lane / kLanes + j * (32 / kLanes)) * kPitch +
                                                          (lane % kLanes) * 4);
        if (!to[j]) continue;
        if (p.n_split > 1) {
          *reinterpret_cast<float4*>(to[j]) = v;
          to[j] += kC * 4;
        } else {
          *reinterpret_cast<uint2*>(to[j]) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
          to[j] += kC * 2;
        }
      }
      __syncwarp();
    }
  }
  if (threadIdx.x == kMmaWarp0 * 32 && split == 0 && hk == 0 && mt == 0 &&
      static_cast<long long>(p.lens[r]) + sp.n > p.max_len)
    atomicOr(p.err, DT_ERR_BAD_INDEX);
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp0) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem_base);
  }
}

template <int DH, bool SHORT>
cudaError_t launch_tree(const CacheAttnParams& p, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = opt_in_smem(k_cache_tree<DH, SHORT>, &done);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_cache_tree<DH, SHORT>, dim3(p.m_tiles * p.n_split, p.c.Hkv, p.R), dim3(kTreeThreads),
                       TreeSmem<DH>::kTotal + 1024, st, true, p);
}

}  // namespace

cudaError_t launch_cache_tree(const CacheAttnParams& p, cudaStream_t st) {
  if (p.wait_limit < kWaitLimitCycles) return p.c.dh == 128 ? launch_tree<128, true>(p, st) : launch_tree<64, true>(p, st);
  return p.c.dh == 128 ? launch_tree<128, false>(p, st) : launch_tree<64, false>(p, st);
}

}  // namespace dt
