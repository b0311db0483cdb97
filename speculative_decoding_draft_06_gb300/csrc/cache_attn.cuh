// What the attention kernels over the 4-bit cache share: their parameters, a
// request's keys, and the rows' way out (directly, or as shares of several
// key splits in the workspace, which a join kernel brings together).
#pragma once
#include "cache.cuh"
#include "ptx.cuh"

namespace dt {

constexpr float kBias = 6.f;   // the reference maximum's weight is 2^kBias
constexpr float kRaise = 8.f;  // the reference rises when a score passes it by this

// Rows of a CTA of the tensor-core kernel: two tiles of 128.  Up to kTreeTail
// rows that a request has behind its last whole tile of 128 (a tree of 2^k
// nodes and its root: the root's) are the few-rows kernel's, in a launch of
// their own.
constexpr int kTreeRowsCta = 256, kTreeTile = 128, kTreeTail = 8;

struct CacheAttnParams {
  CacheView c;              // the layer
  const uint16_t* Q;
  long long q_stride;       // elements between rows (nodes)
  const uint32_t* mask;     // [R][B][words]
  const int32_t *n_nodes, *table, *lens;
  int max_pages, R, B, max_len, Hq, g, words, rows;
  int tile_rows, tile_keys;  // of the kernel: 8 or 16 x 64, 256 x 128
  int m_tiles;               // row tiles
  int n_split, split_tiles;  // key tiles per split
  int cluster;               // the splits are one cluster and join there
  int tail;                  // the few-rows kernel works on the rows behind the whole tiles
  float scale_log2;          // scale * log2(e)
  uint16_t* O;               // [R][B+1][Hq][dh]
  float* part;               // [R][Hkv][m_tiles][n_split][tile_rows][dh + kPartHead] (n_split > 1)
  int* err;
  long long wait_limit;      // cycles that a pipeline wait may take
};

// A request's keys: its prefix and nodes, cut at max_len.
struct Span {
  int Lp, n, L;  // prefix, nodes, keys
};

__device__ __forceinline__ bool request_span(const CacheAttnParams& p, int r, Span* s) {
  const int len = p.lens[r];
  int n = p.n_nodes ? min(p.n_nodes[r], p.B) : p.B;
  if (len < 0 || n < 0) return false;
  s->Lp = min(len, p.max_len);
  s->n = n;
  s->L = static_cast<int>(min(static_cast<long long>(len) + n, static_cast<long long>(p.max_len)));
  return true;
}


// The rows behind a request's whole tiles of 128 that are the few-rows
// kernel's (of `rows` in all).
__device__ __forceinline__ int tail_rows(int rows) {
  const int odd = rows % kTreeTile;
  return rows > kTreeTile && odd <= kTreeTail ? odd : 0;
}

// Key tiles that the rows of row tile mt can see: the prefix
// and the nodes up to the tile's last row's.
__device__ __forceinline__ int row_tile_keys(const CacheAttnParams& p, const Span& s, int mt) {
  const int last = p.tail ? s.n : min(s.n, (mt * p.tile_rows + p.tile_rows - 1) / p.g);
  const int keys = min(s.L, s.Lp + last);
  return (keys + p.tile_keys - 1) / p.tile_keys;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Whether a phase is complete.  try_wait waits itself for longer than any wait
// of these kernels lasts, so a short limit needs the poll that does not.
template <bool SHORT>
__device__ __forceinline__ bool poll(uint32_t addr, uint32_t parity) {
  if constexpr (!SHORT) return mbar_try_wait(addr, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(addr), "r"(parity)
      : "memory");
  return ok != 0;
}

// Scales as the products with weights take them: what nothing has written may
// be e4m3's NaN, which a weight of zero does not cancel.  (max takes the other
// operand of a NaN; scales are not negative.)
__device__ __forceinline__ uint32_t finite_scales(uint32_t s2) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(s2), "r"(0u));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}


// D (16x8, fp32) += A (16x16) B (16x8), fp16.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A 16x8 block of fp16 pairs, rows to columns: lane (r, c)'s pair (row r,
// columns 2c, 2c + 1) of an 8x8 matrix becomes (column r, rows 2c, 2c + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A query row becomes fp16 as multiples of 2^e, its largest magnitude (`top`)
// in [1, 2) of them, or below 4 and above 2^-8 at the ends of bf16's range.
// *down: 2^-e.  Returns the factor of its scores to base 2, 2^e scale log2(e)
// k_scale, held between 2^-126 (0 would make NaN of the keys that are not seen)
// and 2^100 (a score is below 2^21, so no product overflows): scores, whose
// unit is 2^-34 or more, weigh the same beyond either end.
__device__ __forceinline__ float row_exponent(const CacheAttnParams& p, float top, float* down) {
  const int e = top > 0.f ? max(-126, min(static_cast<int>(__float_as_uint(top) >> 23) - 127, 126)) : 0;
  *down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float f = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.c.k_scale;
  return fmaxf(fminf(f, 0x1p100f), 0x1p-126f);
}

// The score above which a reference m rises: kRaise behind it in the exponent
// (rounded down: no weight passes 2^(kBias + kRaise) and fp16's range).
__device__ __forceinline__ float rise_limit(float m, float fac) { return __fadd_rd(m, __fdividef(kRaise, fac)); }

// Row q of a key/value head in the output (node q / g, query head hk g + q % g).
__device__ __forceinline__ size_t cache_out_row(const CacheAttnParams& p, int r, int hk, int q) {
  const int nd = q / p.g;
  return ((static_cast<size_t>(r) * (p.B + 1) + nd) * p.Hq + hk * p.g + (q - nd * p.g)) * p.c.dh;
}

// Row `row` of row tile mt and one split in the workspace: (m, l), and behind
// kPartHead the dh unnormalised outputs (rows of 16-byte pieces).
constexpr int kPartHead = 4;
__device__ __forceinline__ float* cache_part_row(const CacheAttnParams& p, int r, int hk, int mt, int split, int row) {
  const size_t tile = ((static_cast<size_t>(r) * p.c.Hkv + hk) * p.m_tiles + mt) * p.n_split + split;
  return p.part + (tile * p.tile_rows + row) * (p.c.dh + kPartHead);
}

// The tensor-core kernel of many rows (cache_tree.cu).
cudaError_t launch_cache_tree(const CacheAttnParams& p, cudaStream_t st);

}  // namespace dt
