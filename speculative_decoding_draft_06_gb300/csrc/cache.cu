// The paged 4-bit key/value cache: writing and reading tokens, and the page
// operations (reserve, fork, commit, release, copy).
#include <cuda_bf16.h>

#include "cache_pages.cuh"

namespace dt {
namespace {

// ------------------------------------------------------- append and read
// Tokens lens[r] + offset + i, i < min(n, count[r]), of the requests r.
// A warp takes the tokens of one head that make 32 blocks of 16 dimensions
// (dh = 128: 4 tokens, dh = 64: 8), keys and values; a lane takes one block:
// 32 bytes of bf16 on one side, 8 bytes of codes and 1 of scale on the
// other.  Consecutive warps take consecutive heads, so that the bf16 rows
// are touched in their order and the codes of a warp's tokens are one
// contiguous piece.
// Bound by memory and, in append, by issue as well (0.83 instructions a cycle
// and scheduler): 2 x 16000 tokens of 8 heads of 128 take 59 us in and out (the
// look at a page's holders 1 of them), 336 MB, 86% of a copy's rate (9 us more with loads behind the page lookup and
// plain stores; several heads per warp, one lookup for all, 4 to 8 more: fewer
// loads in flight).  A step's 8 x 129 tokens: 5.7 us in and out.
struct TokenParams {
  CacheView c;
  const uint16_t *K, *V;   // append: input rows
  uint16_t *Ko, *Vo;       // read: output rows
  long long req_stride, token_stride;
  const int32_t *table, *lens, *count;
  const int32_t* refs;     // append: the pages' holders (or null)
  int max_pages, offset, R, n, groups;  // groups: ceil(n / tokens per warp)
  int zero_rest;           // read: tokens that no row has are written as 0
  int* err;
};

struct TokenSlot {
  int r, h, i, blk;
  bool live;
  const uint8_t* base;  // the token's page's chunk of head h (live and *paged)
  int t;                // token within the page
  bool paged;
  int page;
};

// Data that is read once (issued here, whatever the compiler would move).
__device__ __forceinline__ uint4 load_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <int DH>
__device__ __forceinline__ TokenSlot token_of(const TokenParams& p) {
  constexpr int kBlk = DH / 16, kTok = 32 / kBlk;
  TokenSlot s;
  const int lane = threadIdx.x & 31;
  const unsigned w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const unsigned rest = w / static_cast<unsigned>(p.c.Hkv);
  s.h = static_cast<int>(w - rest * p.c.Hkv);
  s.r = static_cast<int>(rest / static_cast<unsigned>(p.groups));
  s.i = static_cast<int>(rest - static_cast<unsigned>(s.r) * p.groups) * kTok + lane / kBlk;
  s.blk = lane % kBlk;
  s.live = s.paged = false;
  s.base = nullptr;
  s.t = 0;
  return s;
}

// The token's page and place in it, if it has them (r < R).
__device__ __forceinline__ void find_slot(const TokenParams& p, TokenSlot& s) {
  const int len = p.lens[s.r];
  const int n = p.count ? min(p.n, p.count[s.r]) : p.n;
  s.live = len >= 0 && s.i < n;
  if (!s.live) return;
  const long long pos = static_cast<long long>(len) + p.offset + s.i;
  const long long slot = pos >> p.c.log_page;
  if (pos >= 0 && slot < p.max_pages) {
    const int page = p.table[static_cast<size_t>(s.r) * p.max_pages + slot];
    if (page >= 0 && page < p.c.pages) {
      s.paged = true;
      s.page = page;
      s.base = p.c.pool + static_cast<size_t>(page) * p.c.page_bytes + static_cast<size_t>(s.h) * p.c.chunk;
      s.t = static_cast<int>(pos & ((1 << p.c.log_page) - 1));
    }
  }
  if (!s.paged && s.blk == 0 && s.h == 0 && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
}

// One block of 16 bf16 -> 8 bytes of codes and the scale byte.
// x / s is a product with the rounded reciprocal, rounded once more to fp16:
// a bf16 x and a tie t of two codes times an e4m3 scale differ by at least
// 2^-8 of x or not at all, so the product's error (2^-23) never crosses a
// tie, and the fp16 rounding (2^-12) puts a quotient that is a tie back on it.
__device__ __forceinline__ uint2 quantise16(const uint4 (&in)[2], float inv_scale, uint32_t* scale) {
  uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w, in[1].x, in[1].y, in[1].z, in[1].w};
  __nv_bfloat162 top = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[k]);
    w[k] &= __heq2_mask(x, x);  // NaN -> 0
    top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])));
  }
  const float amax = fmaxf(__low2float(top), __high2float(top)) * inv_scale;
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(__fdiv_rn(amax, 6.f)));
  *scale = two & 0xFFu;
  const uint32_t sh = e4m3x2_to_f16x2(two);
  const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sh)));
  const float r = s > 0.f ? __frcp_rn(s) * inv_scale : 0.f;
  uint32_t q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // (a huge quotient becomes inf in fp16 and saturates)
    const float lo = __uint_as_float(w[k] << 16) * r, hi = __uint_as_float(w[k] & 0xFFFF0000u) * r;
    const float2 f = __half22float2(__floats2half2_rn(lo, hi));
    q[k] = f32x2_to_e2m1x2(f.x, f.y);
  }
  return make_uint2(q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                    q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24));
}

template <int DH>
__global__ void __launch_bounds__(256) k_cache_append(const TokenParams p) {
  pdl_wait();
  pdl_trigger();
  TokenSlot s = token_of<DH>(p);
  if (s.r >= p.R || s.i >= p.n) return;
  const size_t at = static_cast<size_t>(s.r) * p.req_stride + static_cast<size_t>(s.i) * p.token_stride +
                    s.h * DH + s.blk * 16;
  const uint4* k = reinterpret_cast<const uint4*>(p.K + at);
  const uint4* v = reinterpret_cast<const uint4*>(p.V + at);
  // (on their way while the page is looked up)
  const uint4 kin[2] = {load_once(k), load_once(k + 1)};
  const uint4 vin[2] = {load_once(v), load_once(v + 1)};
  find_slot(p, s);
  if (!s.live || !s.paged) return;
  const int holders = p.refs ? p.refs[s.page] : 1;  // (on its way during the arithmetic)
  uint8_t* base = const_cast<uint8_t*>(s.base);
  const int codes = (DH / 2) << p.c.log_page;  // bytes of a chunk's key codes
  const int half = p.c.chunk >> 1;
  uint32_t sk, sv;
  const uint2 ck = quantise16(kin, 1.f / p.c.k_scale, &sk);
  const uint2 cv = quantise16(vin, 1.f / p.c.v_scale, &sv);
  if (holders > 1) {  // other rows read it
    if (s.blk == 0 && s.h == 0 && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
    return;
  }
  *reinterpret_cast<uint2*>(base + s.t * (DH / 2) + s.blk * 8) = ck;
  base[codes + s.t * (DH / 16) + s.blk] = static_cast<uint8_t>(sk);
  *reinterpret_cast<uint2*>(base + half + s.t * (DH / 2) + s.blk * 8) = cv;
  base[half + codes + s.t * (DH / 16) + s.blk] = static_cast<uint8_t>(sv);
}

// The same for packed tokens with slots of their own: token i goes to token
// slot[i] % page_tokens of page slot[i] / page_tokens (negative: nowhere).
// Bound as the above by memory: 24000 packed tokens of 8 heads of 128 written and read back 54 us.
template <int DH>
__global__ void __launch_bounds__(256) k_cache_append_slots(const TokenParams p) {
  pdl_wait();
  pdl_trigger();
  const TokenSlot s = token_of<DH>(p);
  if (s.r >= 1 || s.i >= p.n) return;
  const size_t at = static_cast<size_t>(s.i) * p.token_stride + s.h * DH + s.blk * 16;
  const uint4* k = reinterpret_cast<const uint4*>(p.K + at);
  const uint4* v = reinterpret_cast<const uint4*>(p.V + at);
  const uint4 kin[2] = {load_once(k), load_once(k + 1)};
  const uint4 vin[2] = {load_once(v), load_once(v + 1)};
  const int slot = __ldg(p.table + s.i);
  if (slot < 0) return;
  const int page = slot >> p.c.log_page, t = slot & ((1 << p.c.log_page) - 1);
  const bool there = page < p.c.pages;
  const int holders = p.refs && there ? p.refs[page] : 1;
  uint32_t sk, sv;
  const uint2 ck = quantise16(kin, 1.f / p.c.k_scale, &sk);
  const uint2 cv = quantise16(vin, 1.f / p.c.v_scale, &sv);
  if (!there || holders > 1) {  // (other rows read it)
    if (s.blk == 0 && s.h == 0 && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
    return;
  }
  uint8_t* base = p.c.pool + static_cast<size_t>(page) * p.c.page_bytes + static_cast<size_t>(s.h) * p.c.chunk;
  const int codes = (DH / 2) << p.c.log_page, half = p.c.chunk >> 1;
  *reinterpret_cast<uint2*>(base + t * (DH / 2) + s.blk * 8) = ck;
  base[codes + t * (DH / 16) + s.blk] = static_cast<uint8_t>(sk);
  *reinterpret_cast<uint2*>(base + half + t * (DH / 2) + s.blk * 8) = cv;
  base[half + codes + t * (DH / 16) + s.blk] = static_cast<uint8_t>(sv);
}

// 8 bytes of codes and a scale byte -> 16 bf16 (exact).
__device__ __forceinline__ void values16(uint2 codes, uint32_t scale, float mul, uint4 (&out)[2]) {
  const uint32_t s2 = e4m3x2_to_f16x2(scale | (scale << 8));
  uint32_t o[8], lo[4], hi[4];
  e2m1x8_to_f16(codes.x, lo);
  e2m1x8_to_f16(codes.y, hi);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t x = h2mul(k < 4 ? lo[k] : hi[k - 4], s2);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * mul, f.y * mul);
    o[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  out[0] = make_uint4(o[0], o[1], o[2], o[3]);
  out[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int DH>
__global__ void __launch_bounds__(256) k_cache_read(const TokenParams p) {
  pdl_wait();
  pdl_trigger();
  TokenSlot s = token_of<DH>(p);
  if (s.r >= p.R) return;
  find_slot(p, s);
  if (!s.live && !(p.zero_rest && s.i < p.n)) return;
  const size_t at = ((static_cast<size_t>(s.r) * p.n + s.i) * p.c.Hkv + s.h) * DH + s.blk * 16;
  uint4* k = reinterpret_cast<uint4*>(p.Ko + at);
  uint4* v = reinterpret_cast<uint4*>(p.Vo + at);
  uint4 ko[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  uint4 vo[2] = {ko[0], ko[0]};
  if (s.paged) {
    const int codes = (DH / 2) << p.c.log_page, half = p.c.chunk >> 1;
    const uint2 ck = *reinterpret_cast<const uint2*>(s.base + s.t * (DH / 2) + s.blk * 8);
    const uint32_t sk = s.base[codes + s.t * (DH / 16) + s.blk];
    const uint2 cv = *reinterpret_cast<const uint2*>(s.base + half + s.t * (DH / 2) + s.blk * 8);
    const uint32_t sv = s.base[half + codes + s.t * (DH / 16) + s.blk];
    values16(ck, sk, p.c.k_scale, ko);
    values16(cv, sv, p.c.v_scale, vo);
  }
  __stcs(k, ko[0]);
  __stcs(k + 1, ko[1]);
  __stcs(v, vo[0]);
  __stcs(v + 1, vo[1]);
}

// --------------------------------------------------------- page operations
constexpr int kMaxForks = 1024;

// Calls give(rank, page) for the first `need` free pages (refs == 0) in
// ascending order of their numbers; returns how many there were (at most
// need).  Stops at the 4096 pages that complete them.
template <typename Give>
__device__ __forceinline__ int find_free(const int32_t* refs, int pages, int need, int* sh, Give give) {
  int found = 0;
  for (long long b = 0; b < pages && found < need; b += 4 * kPlanThreads) {
    const long long at = b + 4 * threadIdx.x;
    unsigned free4 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k < pages && refs[at + k] == 0) free4 |= 1u << k;
    int total;
    int rank = found + block_exclusive(__popc(free4), sh, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((free4 >> k) & 1u) {
        if (rank < need) give(rank, static_cast<int>(at) + k);
        ++rank;
      }
    found += total;
  }
  return found < need ? found : need;
}

// Number of leading entries >= 0 of a page-table row, by a warp: 32 probes
// cut the range by 32 each time.
__device__ __forceinline__ int held_pages(const int32_t* row, int max_pages) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = max_pages;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const long long at = lo + static_cast<long long>(lane) * step;
    const bool end = at >= hi || row[at] < 0;
    const unsigned b = __ballot_sync(kFullMask, end);
    if (b == 0) {
      lo = lo + 31 * step + 1;
      continue;
    }
    const int f = __ffs(b) - 1;
    if (f == 0) return lo;
    const long long nhi = lo + static_cast<long long>(f) * step;
    lo = lo + (f - 1) * step + 1;
    if (nhi < hi) hi = static_cast<int>(nhi);
  }
  return lo;
}

struct ReserveParams {
  int32_t* refs;
  int32_t* table;
  const int32_t *lens, *want;
  int32_t* ok;
  int pages, log_page, max_pages, R, pending;
};

// One block: what each row lacks, the rows' first ranks among the free
// pages (prefix sums), then the free pages go to the row their rank falls in.
// Latency: 4.5 us alone with cold caches; the search is one block's and starts at
// page 0: behind 100000 pages in use 27 us, behind 500000 120.
__global__ void __launch_bounds__(kPlanThreads) k_cache_reserve(const ReserveParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_first[kMaxReserveRows + 1], s_held[kMaxReserveRows];
  __shared__ int sh[33];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int r = warp; r < p.R; r += kPlanThreads / 32) {
    const long long len = p.lens[r], want = p.want[r];
    const long long need = (len + want + (1 << p.log_page) - 1) >> p.log_page;
    int held = -1, lack = 0;  // held = -1: refused
    if (len >= 0 && want >= 0 && need <= p.max_pages) {
      held = held_pages(p.table + static_cast<size_t>(r) * p.max_pages, p.max_pages);
      lack = need > held ? static_cast<int>(need) - held : 0;
      // tokens would go into a page that another row reads
      bool shared = false;
      if (want > 0 || p.pending > 0)
        for (long long at = (max(len - p.pending, 0ll) >> p.log_page) + lane; at < need && at < held; at += 32) {
          const int page = p.table[static_cast<size_t>(r) * p.max_pages + at];
          shared |= page < p.pages && p.refs[page] > 1;
        }
      if (__any_sync(kFullMask, shared)) {
        held = -1;
        lack = 0;
      }
    }
    if (lane == 0) {
      s_held[r] = held;
      s_first[r] = lack;
    }
  }
  __syncthreads();
  int total = 0;
  {
    int v[4], sum = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 4 * tid + k;
      v[k] = r < p.R ? s_first[r] : 0;
      sum += v[k];
    }
    int at = block_exclusive(sum, sh, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 4 * tid + k;
      if (r < p.R) s_first[r] = at;
      at += v[k];
    }
    if (tid == 0) s_first[p.R] = total;
  }
  __syncthreads();
  const int found = find_free(p.refs, p.pages, total, sh, [&](int rank, int page) {
    int lo = 0, hi = p.R;  // the last row whose first rank is <= rank
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= rank) lo = mid;
      else hi = mid;
    }
    p.table[static_cast<size_t>(lo) * p.max_pages + s_held[lo] + rank - s_first[lo]] = page;
    p.refs[page] = 1;
  });
  __syncthreads();
  for (int r = tid; r < p.R; r += kPlanThreads) {
    const int lack = s_first[r + 1] - s_first[r];
    const bool ok = s_held[r] >= 0 && (lack == 0 || s_first[r + 1] <= found);
    p.ok[r] = ok ? 1 : 0;
    if (!ok && s_held[r] >= 0 && s_first[r] < found)  // the row the pages ran out in
      for (int k = 0; k < found - s_first[r]; ++k) {
        int32_t* e = p.table + static_cast<size_t>(r) * p.max_pages + s_held[r] + k;
        p.refs[*e] = 0;
        *e = -1;
      }
  }
}

struct ForkParams {
  int32_t* refs;
  int32_t *table, *lens;
  const int32_t *src, *dst;
  int32_t* ok;
  int pages, log_page, max_pages, R, n, pending;
  // the copy
  uint8_t* pool;
  size_t page_bytes, layer_bytes;
};

// Tokens of a row of len that are written: behind them `pending` are only
// counted, and their places are still to be written.
__device__ __forceinline__ int written(int len, int pending) { return max(len - pending, 0); }

// Pages of written tokens only are shared; those behind are the copy's own:
// the one in which the written tokens end (copied below) and, with more
// pending tokens, fresh ones.
__global__ void __launch_bounds__(kPlanThreads) k_cache_fork(const ForkParams p) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_src[kMaxForks], s_dst[kMaxForks], s_len[kMaxForks], s_first[kMaxForks + 1];
  __shared__ int sh[33];
  const int i = threadIdx.x;
  const int P = 1 << p.log_page;
  if (i < p.n) {
    s_src[i] = p.src[i];
    s_dst[i] = p.dst[i];
  }
  __syncthreads();
  bool valid = false;
  int len = -1, own = 0;  // own: pages that are not shared
  if (i < p.n) {
    const int s = s_src[i], d = s_dst[i];
    valid = s >= 0 && s < p.R && d >= 0 && d < p.R;
    for (int j = 0; j < p.n; ++j)
      if (s_src[j] == d || (j < i && s_dst[j] == d)) valid = false;
    if (valid) {
      len = p.lens[s];
      const int done = len < 0 ? 0 : written(len, p.pending);
      const int need = len < 0 ? 0 : static_cast<int>((static_cast<long long>(len) + P - 1) >> p.log_page);
      const int there = static_cast<int>((static_cast<long long>(done) + P - 1) >> p.log_page);
      valid = len >= 0 && need <= p.max_pages && p.table[static_cast<size_t>(d) * p.max_pages] < 0;
      if (valid && there > 0) {
        const int last = p.table[static_cast<size_t>(s) * p.max_pages + there - 1];
        valid = last >= 0 && last < p.pages;
      }
      if (valid) own = need - (done >> p.log_page);
    }
  }
  int total;
  const int first = block_exclusive(own, sh, &total);
  if (i < p.n) {
    s_len[i] = len;
    s_first[i] = first;
  }
  if (i == 0) s_first[p.n] = total;
  __syncthreads();
  // (the last row whose first rank is <= rank: refused ones have no ranks)
  const int found = find_free(p.refs, p.pages, total, sh, [&](int rank, int page) {
    int lo = 0, hi = p.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] <= rank) lo = mid;
      else hi = mid;
    }
    p.table[static_cast<size_t>(s_dst[lo]) * p.max_pages + (written(s_len[lo], p.pending) >> p.log_page) + rank -
            s_first[lo]] = page;
    p.refs[page] = 1;
  });
  __syncthreads();
  if (i < p.n) {
    const bool ok = valid && (own == 0 || first + own <= found);
    p.ok[i] = ok ? 1 : 0;
    if (!ok) {
      for (int k = 0; k < min(own, found - first); ++k) {  // the row the pages ran out in
        int32_t* e = p.table + static_cast<size_t>(s_dst[i]) * p.max_pages + (written(len, p.pending) >> p.log_page) + k;
        p.refs[*e] = 0;
        *e = -1;
      }
      s_len[i] = -1;
    }
  }
  __syncthreads();
  const int warp = i >> 5, lane = i & 31;
  for (int f = warp; f < p.n; f += kPlanThreads / 32) {
    if (s_len[f] < 0) continue;
    const int whole = written(s_len[f], p.pending) >> p.log_page;
    const int32_t* from = p.table + static_cast<size_t>(s_src[f]) * p.max_pages;
    int32_t* to = p.table + static_cast<size_t>(s_dst[f]) * p.max_pages;
    for (int j = lane; j < whole; j += 32) {
      const int page = from[j];
      to[j] = page;
      if (page >= 0 && page < p.pages) atomicAdd(&p.refs[page], 1);
    }
    if (lane == 0) p.lens[s_dst[f]] = s_len[f];
  }
}

// 16-byte units from src to dst by the block: unit (begin + k) for k < n,
// eight loads in flight per thread.
__device__ __forceinline__ void copy_units(const uint4* __restrict__ src, uint4* __restrict__ dst, int begin,
                                           int end) {
  constexpr int kU = 8;
  for (int b = begin; b < end; b += kU * blockDim.x) {
    uint4 v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = b + u * blockDim.x + threadIdx.x;
      if (at < end) v[u] = __ldcs(src + at);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = b + u * blockDim.x + threadIdx.x;
      if (at < end) __stcs(dst + at, v[u]);
    }
  }
}

// Block x of a page's pieces: [begin, end) in 16-byte units.
__device__ __forceinline__ void piece(size_t page_bytes, int* begin, int* end) {
  const long long units = static_cast<long long>(page_bytes >> 4);
  *begin = static_cast<int>(units * blockIdx.x / gridDim.x);
  *end = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
}

// The partly filled page of each fork, grid (pieces, layers, forks).  Bound by
// memory: 32 forks, 32 layers, pages of 64 tokens of 8 heads of 128: 151 MB
// with the release and the plan in front of it in 24 us, 6.3 TB/s (a graph's).
__global__ void __launch_bounds__(256) k_cache_fork_copy(const ForkParams p) {
  const int i = blockIdx.z;
  pdl_wait();
  if (!p.ok[i]) return;
  const int s = p.src[i], d = p.dst[i], done = written(p.lens[d], p.pending);
  if ((done & ((1 << p.log_page) - 1)) == 0) return;
  const int from = p.table[static_cast<size_t>(s) * p.max_pages + (done >> p.log_page)];
  const int to = p.table[static_cast<size_t>(d) * p.max_pages + (done >> p.log_page)];
  uint8_t* layer = p.pool + static_cast<size_t>(blockIdx.y) * p.layer_bytes;
  int b, e;
  piece(p.page_bytes, &b, &e);
  copy_units(reinterpret_cast<const uint4*>(layer + static_cast<size_t>(from) * p.page_bytes),
             reinterpret_cast<uint4*>(layer + static_cast<size_t>(to) * p.page_bytes), b, e);
}

struct CopyParams {
  uint8_t* pool;
  size_t page_bytes, layer_bytes;
  const int32_t *src, *dst;
  int n, pages;
  int* err;
};

// Grid (pieces, layers, pairs).  Every block looks for its own destination
// among the sources and the earlier destinations: such a pair is skipped, so
// that the result does not depend on the blocks' order.  Memory's while the pairs
// are few: pages of 64 tokens of 8 heads of 128 in 8 layers, 1024 pairs 177 us (6.8
// TB/s), 4096 801 us (6.0); the looks grow with their square.
__global__ void __launch_bounds__(256) k_cache_copy(const CopyParams p) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.z;
  const int s = p.src[i], d = p.dst[i];
  bool bad = s < 0 || s >= p.pages || d < 0 || d >= p.pages;
  for (int j = threadIdx.x; j < p.n; j += blockDim.x) bad |= p.src[j] == d || (j < i && p.dst[j] == d);
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
    return;
  }
  uint8_t* layer = p.pool + static_cast<size_t>(blockIdx.y) * p.layer_bytes;
  int b, e;
  piece(p.page_bytes, &b, &e);
  copy_units(reinterpret_cast<const uint4*>(layer + static_cast<size_t>(s) * p.page_bytes),
             reinterpret_cast<uint4*>(layer + static_cast<size_t>(d) * p.page_bytes), b, e);
}

struct ReleaseParams {
  int32_t* refs;
  int32_t *table, *lens;
  const int32_t *rows, *keep;
  int pages, log_page, max_pages, R;
  int* err;
};

// A block per listed row.  An entry is taken by an exchange with -1, so a
// row listed twice lets each page go once.
__global__ void __launch_bounds__(128) k_cache_release(const ReleaseParams p) {
  pdl_wait();
  pdl_trigger();
  const int r = p.rows[blockIdx.x], keep = p.keep[blockIdx.x];
  if (r < 0 || r >= p.R || keep < 0) {
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
    return;
  }
  const int first = static_cast<int>((static_cast<long long>(keep) + (1 << p.log_page) - 1) >> p.log_page);
  int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
  for (long long j = static_cast<long long>(first) + threadIdx.x; j < p.max_pages; j += blockDim.x) {
    if (row[j] == -1) continue;
    const int page = atomicExch(&row[j], -1);
    if (page == -1) continue;
    bool bad = page < 0 || page >= p.pages;
    if (!bad && atomicSub(&p.refs[page], 1) <= 0) {  // (held by nobody: the count stays)
      atomicAdd(&p.refs[page], 1);
      bad = true;
    }
    if (bad && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
  }
  if (threadIdx.x == 0) atomicMin(&p.lens[r], keep);
}

struct CommitParams {
  uint8_t* pool;
  size_t page_bytes, layer_bytes;
  const int32_t* table;
  int32_t* lens;
  const int32_t *nodes, *len;
  int pages, log_page, max_pages, layers, Hkv, chunk, R, max_len, extra;
  int* err;
};

// Accepted tokens of row r that can move: -1 for a row to leave as it is.
// Every thread of the block calls it (*bad: why, to be flagged).
__device__ __forceinline__ int commit_count(const CommitParams& p, int r, int* bad) {
  *bad = 0;
  const int len = p.lens[r];
  if (len < 0) return -1;
  const int m = max(0, min(p.len[r], p.max_len));
  const int32_t* nodes = p.nodes + static_cast<size_t>(r) * p.max_len;
  const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
  bool b = static_cast<long long>(len) + m + p.extra > INT32_MAX;  // (lengths and positions are 32 bits)
  for (int k = threadIdx.x; k < m; k += blockDim.x) {
    const int node = nodes[k];
    b |= node < 0 || (k > 0 && node <= nodes[k - 1]) || static_cast<long long>(len) + node > INT32_MAX;
    if (b) break;
    const long long from = (static_cast<long long>(len) + node) >> p.log_page;
    const long long to = (static_cast<long long>(len) + k) >> p.log_page;
    b |= from >= p.max_pages || to >= p.max_pages;
    if (b) break;
    const int f = row[from], t = row[to];
    b |= f < 0 || f >= p.pages || t < 0 || t >= p.pages;
  }
  *bad = __syncthreads_or(b);
  return *bad ? -1 : m;
}

// A cluster per row, its CTAs share the layers.  A token of one head is 18
// units of dh / 16 bytes (8 + 1 of keys, 8 + 1 of values).  Ranks rise, so
// token k's source is at or behind position k: a chunk of tokens is read whole
// before it is written, and no later chunk reads what an earlier one wrote.
// The row's length changes once every CTA of its cluster has read it.
// Latency of a read behind a lookup behind a read: release, reserve and commit
// of a path of 8 tokens in 32 layers take 10.8 us, of 32 paths 16.2.
template <typename U>
__global__ void __launch_bounds__(256) k_cache_commit(const CommitParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int kU = 8;
  unsigned cl, rank;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int r = blockIdx.x / cl;
  int bad;
  const int m = commit_count(p, r, &bad);
  const int len = p.lens[r], P = 1 << p.log_page;
  const int32_t* nodes = p.nodes + static_cast<size_t>(r) * p.max_len;
  const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
  // the CTA's layers, one after the other, m tokens of `per` units in each (all
  // in 32 bits; a layer at a time, in 64: 3 us more)
  const unsigned per = static_cast<unsigned>(p.Hkv) * 18u, units = m > 0 ? static_cast<unsigned>(m) * per : 0u;
  const unsigned total = units * ((p.layers - rank + cl - 1) / cl);
  cluster_arrive();
  // (a chunk is whole units, not whole tokens: a unit of token k is only
  // overwritten by the same unit of a token before k)
  for (unsigned b = 0; b < total; b += kU * 256) {
    U v[kU];
    U* to[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const unsigned at = b + u * 256 + threadIdx.x;
      to[u] = nullptr;
      if (at < total) {
        const unsigned y = at / units, in = at - y * units, k = in / per, rest = in - k * per;
        const unsigned h = rest / 18u, e = rest - h * 18u, w = e < 9u ? e : e - 9u;
        uint8_t* head = p.pool + static_cast<size_t>(rank + y * cl) * p.layer_bytes + static_cast<size_t>(h) * p.chunk +
                        (e < 9u ? 0 : p.chunk >> 1);
        auto address = [&](int pos) {
          const int t = pos & (P - 1);
          return reinterpret_cast<U*>(head + static_cast<size_t>(row[pos >> p.log_page]) * p.page_bytes +
                                      (w < 8u ? t * 8 + static_cast<int>(w) : P * 8 + t) * static_cast<int>(sizeof(U)));
        };
        v[u] = *address(len + nodes[k]);
        to[u] = address(len + static_cast<int>(k));
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (to[u]) *to[u] = v[u];
  }
  cluster_wait();
  if (rank == 0 && threadIdx.x == 0) {
    if (m >= 0) p.lens[r] = len + m + p.extra;
    if (bad && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
  }
}

// Blocks per page copy: about 32 KB each, a thread's eight 16-byte loads once,
// so that a page of a layer is spread over SMs.
int copy_pieces(size_t page_bytes) {
  const size_t k = (page_bytes + 32767) / 32768;
  return static_cast<int>(k < 1 ? 1 : k > 1024 ? 1024 : k);
}

dartree_status token_params(const dartree_cache* cache, int32_t layer, const void* K, const void* V,
                            const int32_t* table, int32_t max_pages, const int32_t* lens, int32_t offset,
                            const int32_t* count, int32_t R, int32_t n, int32_t* err, TokenParams* p,
                            unsigned* blocks) {
  if (const char* why = cache_view(cache, &p->c)) return cache_fail(DARTREE_ERR_INVALID_ARG, why);
  if (!K || !V || !table || !lens) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (layer < 0 || layer >= cache->layers) return cache_fail(DARTREE_ERR_INVALID_ARG, "no such layer");
  if (R < 1 || n < 1 || max_pages < 1) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad R, n or max_pages");
  if ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & 15)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "K and V must be 16-byte aligned");
  p->c.pool += static_cast<size_t>(layer) * p->c.layer_bytes;
  p->table = table;
  p->lens = lens;
  p->count = count;
  p->max_pages = max_pages;
  p->offset = offset;
  p->R = R;
  p->n = n;
  const int tok = 512 / p->c.dh;  // tokens per warp
  p->groups = (n - 1) / tok + 1;
  p->err = err;
  const long long warps = static_cast<long long>(R) * p->groups * p->c.Hkv;
  if (warps > 0x7FFFFFF0ll) return cache_fail(DARTREE_ERR_UNSUPPORTED, "too many tokens in one call");
  *blocks = static_cast<unsigned>((warps + 7) / 8);
  return DARTREE_OK;
}

// Shared checks of the page operations.
dartree_status page_check(const dartree_cache* cache, const void* table, const void* lens, int32_t max_pages,
                          int32_t R, bool refs, CacheView* v) {
  if (const char* why = cache_view(cache, v)) return cache_fail(DARTREE_ERR_INVALID_ARG, why);
  if (!table || !lens || (refs && !cache->refs))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (R < 1 || max_pages < 1) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad R or max_pages");
  return DARTREE_OK;
}

}  // namespace
}  // namespace dt

extern "C" size_t dartree_cache_page_bytes(int32_t page_tokens, int32_t Hkv, int32_t dh) {
  if (dt::cache_log_page(page_tokens) < 0 || Hkv < 1 || Hkv > 65535 || (dh != 64 && dh != 128)) return 0;
  return static_cast<size_t>(Hkv) * (page_tokens * dh / 8) * 9;
}

extern "C" dartree_status dartree_cache_append(const dartree_cache* cache, int32_t layer, const void* K,
                                               const void* V, int64_t req_stride, int64_t token_stride,
                                               const int32_t* table, int32_t max_pages, const int32_t* lens,
                                               int32_t offset, const int32_t* count, int32_t R, int32_t n,
                                               int32_t* err, void* stream) {
  using namespace dt;
  TokenParams p{};
  unsigned blocks = 0;
  const dartree_status s =
      token_params(cache, layer, K, V, table, max_pages, lens, offset, count, R, n, err, &p, &blocks);
  if (s != DARTREE_OK) return s;
  if (token_stride % 8 != 0 || req_stride % 8 != 0 || req_stride < 0 ||
      token_stride < static_cast<int64_t>(p.c.Hkv) * p.c.dh)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "strides must be multiples of 8 elements, tokens not overlapping");
  p.K = static_cast<const uint16_t*>(K);
  p.V = static_cast<const uint16_t*>(V);
  p.refs = cache->refs;
  p.req_stride = req_stride;
  p.token_stride = token_stride;
  return cache_launched(launch_kernel(p.c.dh == 128 ? k_cache_append<128> : k_cache_append<64>, dim3(blocks),
                                      dim3(256), 0, static_cast<cudaStream_t>(stream), true, p));
}

extern "C" dartree_status dartree_cache_append_slots(const dartree_cache* cache, int32_t layer, const void* K,
                                                     const void* V, int64_t token_stride, const int32_t* slot,
                                                     int32_t n, int32_t* err, void* stream) {
  using namespace dt;
  TokenParams p{};
  unsigned blocks = 0;
  const dartree_status s = token_params(cache, layer, K, V, slot, 1, slot, 0, nullptr, 1, n, err, &p, &blocks);
  if (s != DARTREE_OK) return s;
  if (token_stride % 8 != 0 || token_stride < static_cast<int64_t>(p.c.Hkv) * p.c.dh)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "strides must be multiples of 8 elements, tokens not overlapping");
  p.K = static_cast<const uint16_t*>(K);
  p.V = static_cast<const uint16_t*>(V);
  p.refs = cache->refs;
  p.token_stride = token_stride;
  return cache_launched(launch_kernel(p.c.dh == 128 ? k_cache_append_slots<128> : k_cache_append_slots<64>, dim3(blocks),
                                      dim3(256), 0, static_cast<cudaStream_t>(stream), true, p));
}

extern "C" dartree_status dartree_cache_read_ex(const dartree_cache* cache, int32_t layer, void* K, void* V,
                                                const int32_t* table, int32_t max_pages, const int32_t* lens,
                                                int32_t offset, const int32_t* count, int32_t R, int32_t n,
                                                int32_t zero_rest, int32_t* err, void* stream) {
  using namespace dt;
  TokenParams p{};
  unsigned blocks = 0;
  const dartree_status s =
      token_params(cache, layer, K, V, table, max_pages, lens, offset, count, R, n, err, &p, &blocks);
  if (s != DARTREE_OK) return s;
  p.Ko = static_cast<uint16_t*>(K);
  p.Vo = static_cast<uint16_t*>(V);
  p.zero_rest = zero_rest != 0;
  return cache_launched(launch_kernel(p.c.dh == 128 ? k_cache_read<128> : k_cache_read<64>, dim3(blocks),
                                      dim3(256), 0, static_cast<cudaStream_t>(stream), true, p));
}

extern "C" dartree_status dartree_cache_read(const dartree_cache* cache, int32_t layer, void* K, void* V,
                                             const int32_t* table, int32_t max_pages, const int32_t* lens,
                                             int32_t offset, const int32_t* count, int32_t R, int32_t n,
                                             int32_t* err, void* stream) {
  return dartree_cache_read_ex(cache, layer, K, V, table, max_pages, lens, offset, count, R, n, 0, err, stream);
}

extern "C" dartree_status dartree_cache_reserve_ex(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                                   const int32_t* lens, const int32_t* want, int32_t R,
                                                   int32_t pending, int32_t* ok, void* stream) {
  using namespace dt;
  CacheView v;
  const dartree_status s = page_check(cache, table, lens, max_pages, R, true, &v);
  if (s != DARTREE_OK) return s;
  if (!want || !ok) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (pending < 0) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad pending");
  if (R > kMaxReserveRows) return cache_fail(DARTREE_ERR_UNSUPPORTED, "reserve takes at most 4096 rows");
  if (static_cast<long long>(R) * max_pages > 0x7FFFFFFFll)  // (what the rows lack is summed in 32 bits)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "R * max_pages must be below 2^31");
  const ReserveParams p{cache->refs, table, lens, want, ok, v.pages, v.log_page, max_pages, R, pending};
  return cache_launched(launch_kernel(k_cache_reserve, dim3(1), dim3(kPlanThreads), 0,
                                      static_cast<cudaStream_t>(stream), true, p));
}

extern "C" dartree_status dartree_cache_reserve(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                                const int32_t* lens, const int32_t* want, int32_t R,
                                                int32_t* ok, void* stream) {
  return dartree_cache_reserve_ex(cache, table, max_pages, lens, want, R, 0, ok, stream);
}

extern "C" dartree_status dartree_cache_fork_ex(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                                int32_t* lens, int32_t R, const int32_t* src,
                                                const int32_t* dst, int32_t n, int32_t pending, int32_t* ok,
                                                void* stream) {
  using namespace dt;
  CacheView v;
  const dartree_status s = page_check(cache, table, lens, max_pages, R, true, &v);
  if (s != DARTREE_OK) return s;
  if (n < 0 || pending < 0) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad n or pending");
  if (n == 0) return DARTREE_OK;
  if (!src || !dst || !ok) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (n > kMaxForks || v.layers > 65535)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "fork takes at most 1024 rows and 65535 layers");
  if (pending > 0 && static_cast<long long>(n) * max_pages > 0x7FFFFFFFll)  // (the rows' pages are summed in 32 bits)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "n * max_pages must be below 2^31");
  const ForkParams p{cache->refs, table, lens, src,     dst,    ok,           v.pages,      v.log_page,
                     max_pages,   R,     n,    pending, v.pool, v.page_bytes, v.layer_bytes};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_kernel(k_cache_fork, dim3(1), dim3(kPlanThreads), 0, st, true, p);
  if (e == cudaSuccess)
    e = launch_kernel(k_cache_fork_copy, dim3(copy_pieces(v.page_bytes), v.layers, n), dim3(256), 0, st, true, p);
  return cache_launched(e);
}

extern "C" dartree_status dartree_cache_fork(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                             int32_t* lens, int32_t R, const int32_t* src,
                                             const int32_t* dst, int32_t n, int32_t* ok, void* stream) {
  return dartree_cache_fork_ex(cache, table, max_pages, lens, R, src, dst, n, 0, ok, stream);
}

extern "C" dartree_status dartree_cache_commit(const dartree_cache* cache, const int32_t* table,
                                               int32_t max_pages, int32_t* lens, const int32_t* nodes,
                                               const int32_t* len, int32_t R, int32_t max_len, int32_t extra,
                                               int32_t* err, void* stream) {
  using namespace dt;
  CacheView v;
  const dartree_status s = page_check(cache, table, lens, max_pages, R, false, &v);
  if (s != DARTREE_OK) return s;
  if (!nodes || !len) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (max_len < 1 || extra < 0) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad max_len or extra");
  if (R > (1 << 24)) return cache_fail(DARTREE_ERR_UNSUPPORTED, "commit takes at most 2^24 rows");
  if (static_cast<double>(max_len) * v.Hkv * 18 * ((v.layers + 7) / 8 + 1) > 2147483648.)  // (counted in 32 bits)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "max_len * Hkv * layers is too large");
  const CommitParams p{v.pool,     v.page_bytes, v.layer_bytes, table,   lens, nodes, len,     v.pages,
                       v.log_page, max_pages,    v.layers,      v.Hkv,   v.chunk, R,  max_len, extra, err};
  int cl = 1;  // CTAs per row: about one per layer, up to a cluster
  while (cl < 8 && cl < v.layers) cl *= 2;
  return cache_launched(launch_kernel_cluster(v.dh == 128 ? k_cache_commit<uint2> : k_cache_commit<uint32_t>,
                                              dim3(static_cast<unsigned>(R) * cl), dim3(256), 0,
                                              static_cast<cudaStream_t>(stream), true, cl, p));
}

extern "C" dartree_status dartree_cache_release(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                                int32_t* lens, int32_t R, const int32_t* rows,
                                                const int32_t* keep, int32_t n, int32_t* err, void* stream) {
  using namespace dt;
  CacheView v;
  const dartree_status s = page_check(cache, table, lens, max_pages, R, true, &v);
  if (s != DARTREE_OK) return s;
  if (n < 0) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad n");
  if (n == 0) return DARTREE_OK;
  if (!rows || !keep) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  const ReleaseParams p{cache->refs, table, lens, rows, keep, v.pages, v.log_page, max_pages, R, err};
  return cache_launched(launch_kernel(k_cache_release, dim3(n), dim3(128), 0, static_cast<cudaStream_t>(stream),
                                      true, p));
}

extern "C" dartree_status dartree_cache_copy_pages(const dartree_cache* cache, const int32_t* src,
                                                   const int32_t* dst, int32_t n, int32_t* err, void* stream) {
  using namespace dt;
  CacheView v;
  if (const char* why = cache_view(cache, &v)) return cache_fail(DARTREE_ERR_INVALID_ARG, why);
  if (n < 0) return cache_fail(DARTREE_ERR_INVALID_ARG, "bad n");
  if (n == 0) return DARTREE_OK;
  if (!src || !dst) return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (n > 65535 || v.layers > 65535)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "copy_pages takes at most 65535 pages and layers");
  const CopyParams p{v.pool, v.page_bytes, v.layer_bytes, src, dst, n, v.pages, err};
  return cache_launched(launch_kernel(k_cache_copy, dim3(copy_pieces(v.page_bytes), v.layers, n), dim3(256), 0,
                                      static_cast<cudaStream_t>(stream), true, p));
}
