// The paged 4-bit key/value cache as the kernels see it: addresses of tokens
// and the conversions of the format (e2m1 codes, e4m3 scales of 16
// dimensions; the layout is described with dartree_cache).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <string>

#include "../../include/dartree.h"
#include "common.cuh"
#include "kernels.h"

namespace dt {

struct CacheView {
  uint8_t* pool;        // the layer's pages (page operations: all layers')
  int pages, log_page;  // page_tokens = 1 << log_page
  int Hkv, dh;
  int chunk;            // bytes of a page's one head: page_tokens * dh * 9 / 8
  size_t page_bytes;    // Hkv * chunk
  size_t layer_bytes;   // pages * page_bytes
  int layers;
  float k_scale, v_scale;
};

inline int cache_log_page(int page_tokens) {
  return page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : page_tokens == 128 ? 7 : -1;
}

// Whether x is a power of two in [2^-64, 2^64].
inline bool cache_pow2(float x) {
  uint32_t b;
  __builtin_memcpy(&b, &x, 4);
  const int e = static_cast<int>(b >> 23) - 127;
  return (b & 0x807FFFFFu) == 0 && e >= -64 && e <= 64;
}

// Checks the descriptor and fills the view; nullptr, or why it is bad.
inline const char* cache_view(const dartree_cache* c, CacheView* v) {
  if (!c || !c->pool) return "null cache or pool";
  if (c->layers < 1 || c->pages < 1 || c->Hkv < 1 || c->Hkv > 65535) return "bad cache layers, pages or Hkv";
  const int lp = cache_log_page(c->page_tokens);
  if (lp < 0) return "page_tokens must be 16, 32, 64 or 128";
  if (c->dh != 64 && c->dh != 128) return "the cache's head dimension must be 64 or 128";
  if (reinterpret_cast<uintptr_t>(c->pool) & 15) return "the pool must be 16-byte aligned";
  if (!cache_pow2(c->k_scale) || !cache_pow2(c->v_scale))
    return "k_scale and v_scale must be powers of two from 2^-64 to 2^64";
  v->pool = static_cast<uint8_t*>(c->pool);
  v->pages = c->pages;
  v->log_page = lp;
  v->Hkv = c->Hkv;
  v->dh = c->dh;
  v->chunk = (c->page_tokens * c->dh / 8) * 9;
  v->page_bytes = static_cast<size_t>(c->Hkv) * v->chunk;
  v->layer_bytes = v->page_bytes * static_cast<size_t>(c->pages);
  v->layers = c->layers;
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  return nullptr;
}

inline dartree_status cache_fail(dartree_status s, const char* why) {
  try {
    set_context_free_error(why);
  } catch (...) {  // (no memory for the text: the status stands)
  }
  return s;
}

// (The cache's and the sampler's kernels are launched while the kernel before
// them still runs and wait for it before all else, which hides the launches:
// 32 forks 29 -> 25 us, a prompt in and out 63 -> 59, a tree 33 -> 31, 17 rows
// sampled 25 -> 22.)
inline dartree_status cache_launched(cudaError_t e) {
  return e == cudaSuccess ? DARTREE_OK : cache_fail(DARTREE_ERR_CUDA, cudaGetErrorString(e));
}

// Opts a kernel into its dynamic shared memory, once per device (the calls
// cost as much as a launch).
template <typename Kern>
inline cudaError_t opt_in_smem(Kern* k, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = set_max_dynamic_smem(k);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

// The eight e2m1 codes of a word -> four fp16 pairs, byte by byte (low nibble
// in the low half), exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two e4m3 bytes (low 16 bits) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

// fp32 pair -> two e2m1 codes in a byte (lo in the low nibble), to nearest
// even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t d;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(d)
      : "f"(lo), "f"(hi));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same object in CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T* at_rank(T* p, int rank) {
  uint64_t out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(reinterpret_cast<uint64_t>(p)), "r"(rank));
  return reinterpret_cast<T*>(out);
}

}  // namespace dt
