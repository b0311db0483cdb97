// Page tables and slot maps from request lengths (dartree_cache_plan).
//
// One cluster plans: its CTAs share the rows, and the pages that are looked
// through for free ones.  The prefix sums over the rows (packed tokens, lacking
// pages) each CTA makes for itself from copies in its own shared memory, so that
// a page finds its row and a token its request without another exchange:
//   1. the rows' token ranges [f, e), and their packed starts;
//   2. the pages that the windows have left behind go (holders by atomics, so a
//      page that several rows hold is free when the last lets it go);
//   3. what each row lacks behind its held pages of the range, or why it gets
//      none, to every CTA;
//   4. rounds of kScan pages per CTA: free ones by rank, the lowest first, go to
//      the row their rank falls in;
//   5. ok, starts and, for few tokens, the maps (many: a launch of their own).
// Bound by latency: each step is a few dependent reads and a barrier of the
// cluster.  32 rows of 65 tokens at 9000 in pages of 16 behind a window: 14.3 us on
// the GPU with the release before it that makes the pages be taken again, 7.7 where
// all are held (a caller takes 20 to 25 us to launch it, five outputs' allocations
// among them); 1024 rows with prompts of 2000 tokens among them, maps of 265 thousand:
// 26.8 and 17.5 us, 8 of them the maps' launch.
#include "cache_pages.cuh"

namespace dt {
namespace {

constexpr int kMaxCl = 8;
constexpr int kScan = 4 * kPlanThreads;   // pages that a CTA looks at per round
constexpr int kOwnMaps = 8 * 4096;        // tokens that the planning cluster maps itself

struct PlanParams {
  int32_t* refs;
  int32_t* table;
  const int32_t *lens, *count;
  int32_t *ok, *start, *row, *pos, *slot;
  int pages, log_page, max_pages, R, offset, window, sinks, max_tokens;
  int own_maps;
  int* err;
};

struct PlanSmem {
  int f[kMaxReserveRows];          // first position (-1: refused)
  int start[kMaxReserveRows + 1];  // packed
  int lack[kMaxReserveRows];       // pages (-1: refused)
  int from[kMaxReserveRows];       // the first lacking slot
  int first[kMaxReserveRows + 1];  // rank of the first page
  long long sh64[33];
  int sh[33];
  int found[2][kMaxCl];
};

// The last of n ascending firsts that is <= x (the first is).
__device__ __forceinline__ int last_not_above(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Token t of the packed ones: its row, position and slot (-1 each behind the
// last).  ok_row(r): whether the row has its pages; first(r): its position 0.
template <typename Ok, typename First>
__device__ __forceinline__ void map_token(const PlanParams& p, const int* start, int t, Ok ok_row, First first) {
  int r = -1, pos = -1, slot = -1;
  if (t < start[p.R]) {
    r = last_not_above(start, p.R, t);
    pos = first(r) + t - start[r];
    if (ok_row(r)) {
      const int page = __ldcg(p.table + static_cast<size_t>(r) * p.max_pages + (pos >> p.log_page));
      if (page >= 0 && page < p.pages) slot = (page << p.log_page) + (pos & ((1 << p.log_page) - 1));
    }
  }
  p.row[t] = r;
  p.pos[t] = pos;
  p.slot[t] = slot;
}

__global__ void __launch_bounds__(kPlanThreads) k_cache_plan(const PlanParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  PlanSmem& sm = *reinterpret_cast<PlanSmem*>(raw);
  pdl_wait();
  unsigned cl_u, rank_u;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cl_u));
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank_u));
  const int cl = static_cast<int>(cl_u), rank = static_cast<int>(rank_u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gw = rank * (kPlanThreads / 32) + warp, warps = cl * (kPlanThreads / 32);
  constexpr int kPer = kMaxReserveRows / kPlanThreads;
  const int P = 1 << p.log_page;

  // ---- 1. ranges and packed starts (every CTA, all rows)
  {
    long long v[kPer], sum = 0;
    int f[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = kPer * tid + k;
      f[k] = -1;
      v[k] = 0;
      if (r < p.R) {
        const int len = p.lens[r], n = p.count[r];
        const long long at = static_cast<long long>(len) + p.offset;
        if (len >= 0 && n >= 0 && at >= 0 && at + n <= 0x7FFFFFFFll) {
          f[k] = static_cast<int>(at);
          v[k] = n;
        }
      }
      sum += v[k];
    }
    long long total, at = block_exclusive(sum, sm.sh64, &total);
    // rows that end behind the maps get nothing (nor any later one with tokens)
    int n[kPer], kept = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      at += v[k];
      if (v[k] > 0 && at > p.max_tokens) {
        f[k] = -1;
        v[k] = 0;
      }
      n[k] = static_cast<int>(v[k]);
      kept += n[k];
    }
    int all, before = block_exclusive(kept, sm.sh, &all);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = kPer * tid + k;
      if (r < p.R) {
        sm.f[r] = f[k];
        sm.start[r] = before;
      }
      before += n[k];
    }
    if (tid == 0) sm.start[p.R] = all;
  }
  __syncthreads();

  // ---- 2. pages behind the windows: those whose tokens t all have sinks <= t
  // <= f - window (several warps per row where there are few rows)
  if (p.window > 0) {
    const int per = max(1, warps / p.R);
    for (int i = gw; i < p.R * per; i += warps) {
      const int r = i % p.R, part = i / p.R, f = sm.f[r];
      if (f < 0) continue;
      const int beg = (p.sinks >> p.log_page) + ((p.sinks & (P - 1)) != 0);
      const int end = min(p.max_pages, f >= p.window ? (f - p.window + 1) >> p.log_page : 0);
      int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
      // (most are gone already: what takes the time is to look, all loads together)
      constexpr int kLooks = 8;
      for (int b = beg + part * 32 * kLooks; b < end; b += per * 32 * kLooks) {
        int page[kLooks];
        bool some = false;
#pragma unroll
        for (int k = 0; k < kLooks; ++k) {
          const int j = b + 32 * k + lane;
          page[k] = j < end ? row[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kLooks; ++k) some |= page[k] != -1;
        if (!some) continue;
#pragma unroll
        for (int k = 0; k < kLooks; ++k) {
          if (page[k] == -1) continue;
          row[b + 32 * k + lane] = -1;
          bool bad = page[k] < 0 || page[k] >= p.pages;
          if (!bad && atomicSub(&p.refs[page[k]], 1) <= 0) {  // (held by nobody: the count stays)
            atomicAdd(&p.refs[page[k]], 1);
            bad = true;
          }
          if (bad && p.err) atomicOr(p.err, DT_ERR_BAD_INDEX);
        }
      }
    }
  }
  cluster_sync();

  // ---- 3. what the rows lack
  for (int r = gw; r < p.R; r += warps) {
    const int f = sm.f[r], n = sm.start[r + 1] - sm.start[r];
    int lack = -1, from = 0;
    if (f >= 0) {
      const int beg = f >> p.log_page;
      const long long end = (static_cast<long long>(f) + n + P - 1) >> p.log_page;
      lack = 0;
      from = beg;
      if (n > 0) {
        // held pages first, then none: other orders, pages that another row
        // holds too and bad numbers are refused
        const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
        bool bad = end > p.max_pages;
        int held = 0;
        for (long long b = beg; !bad && b < end; b += 32) {
          const bool in = b + lane < end;
          const int page = in ? __ldcg(row + b + lane) : -1;
          const bool have = page >= 0;
          bad = __any_sync(kFullMask, have && (page >= p.pages || __ldcg(p.refs + page) > 1));
          const unsigned h = __ballot_sync(kFullMask, have);
          // (a held page behind one that is not)
          bad = bad || (h & (h + 1)) != 0 || (h != 0 && held < b - beg);
          held += __popc(h);
        }
        lack = bad ? -1 : static_cast<int>(end - beg) - held;
        from = beg + held;
      }
    }
    if (lane < cl) {
      PlanSmem* o = at_rank(&sm, lane);
      o->lack[r] = lack;
      o->from[r] = from;
    }
  }
  cluster_sync();
  int total = 0;
  {
    int v[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = kPer * tid + k;
      v[k] = r < p.R ? max(sm.lack[r], 0) : 0;
      sum += v[k];
    }
    int at = block_exclusive(sum, sm.sh, &total);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int r = kPer * tid + k;
      if (r < p.R) sm.first[r] = at;
      at += v[k];
    }
    if (tid == 0) sm.first[p.R] = total;
  }
  __syncthreads();

  // ---- 4. the free pages, lowest first
  int found = 0, round = 0;
  for (long long b = 0; b < p.pages && found < total; b += static_cast<long long>(cl) * kScan, ++round) {
    const long long at = b + static_cast<long long>(rank) * kScan + 4 * tid;
    unsigned free4 = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k < p.pages && __ldcg(p.refs + at + k) == 0) free4 |= 1u << k;
    int mine, rank_of = block_exclusive(__popc(free4), sm.sh, &mine);
    if (tid < cl) at_rank(&sm, tid)->found[round & 1][rank] = mine;
    cluster_sync();
    int before = found, all = 0;
    for (int q = 0; q < cl; ++q) {
      const int n = sm.found[round & 1][q];
      if (q < rank) before += n;
      all += n;
    }
    rank_of += before;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((free4 >> k) & 1u) {
        if (rank_of < total) {
          const int r = last_not_above(sm.first, p.R, rank_of);
          p.table[static_cast<size_t>(r) * p.max_pages + sm.from[r] + rank_of - sm.first[r]] = static_cast<int>(at) + k;
          p.refs[at + k] = 1;
        }
        ++rank_of;
      }
    found += all;
  }
  found = min(found, total);
  cluster_sync();

  // ---- 5. results
  auto has_pages = [&](int r) {
    return sm.lack[r] >= 0 && (sm.lack[r] == 0 || sm.first[r] + sm.lack[r] <= found);
  };
  for (int r = rank * kPlanThreads + tid; r < p.R; r += cl * kPlanThreads) {
    p.ok[r] = has_pages(r) ? 1 : 0;
    p.start[r] = sm.start[r];
    if (!has_pages(r) && sm.lack[r] > 0)  // the row the pages ran out in
      for (int k = 0; k < found - sm.first[r]; ++k) {
        int32_t* e = p.table + static_cast<size_t>(r) * p.max_pages + sm.from[r] + k;
        p.refs[__ldcg(e)] = 0;
        *e = -1;
      }
  }
  if (rank == 0 && tid == 0) p.start[p.R] = sm.start[p.R];
  if (p.own_maps)
    for (int t = rank * kPlanThreads + tid; t < p.max_tokens; t += cl * kPlanThreads)
      map_token(p, sm.start, t, has_pages, [&](int r) { return sm.f[r]; });
  cluster_sync();  // (no CTA leaves while another writes to its memory)
}

// The maps of many tokens: grid (tokens / 1024).
__global__ void __launch_bounds__(256) k_cache_maps(const PlanParams p) {
  __shared__ int s_start[kMaxReserveRows + 1];
  pdl_wait();
  pdl_trigger();
  for (int r = threadIdx.x; r <= p.R; r += 256) s_start[r] = p.start[r];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long t = static_cast<long long>(blockIdx.x) * 1024 + k * 256 + threadIdx.x;
    if (t < p.max_tokens)
      map_token(p, s_start, static_cast<int>(t), [&](int r) { return __ldcg(p.ok + r) != 0; },
                [&](int r) { return __ldg(p.lens + r) + p.offset; });
  }
}

}  // namespace
}  // namespace dt

extern "C" dartree_status dartree_cache_plan(const dartree_cache* cache, int32_t* table, int32_t max_pages,
                                             const int32_t* lens, const int32_t* count, int32_t R, int32_t offset,
                                             int32_t window, int32_t sinks, int32_t max_tokens, int32_t* ok,
                                             int32_t* start, int32_t* row, int32_t* pos, int32_t* slot, int32_t* err,
                                             void* stream) {
  using namespace dt;
  CacheView v;
  if (const char* why = cache_view(cache, &v)) return cache_fail(DARTREE_ERR_INVALID_ARG, why);
  if (!cache->refs || !table || !lens || !count || !ok || !start || (max_tokens > 0 && (!row || !pos || !slot)))
    return cache_fail(DARTREE_ERR_INVALID_ARG, "null pointer argument");
  if (R < 1 || max_pages < 1 || max_tokens < 0 || window < 0 || sinks < 0)
    return cache_fail(DARTREE_ERR_INVALID_ARG, "bad R, max_pages, max_tokens, window or sinks");
  if (R > kMaxReserveRows) return cache_fail(DARTREE_ERR_UNSUPPORTED, "plan takes at most 4096 rows");
  if (static_cast<long long>(R) * max_pages > 0x7FFFFFFFll)  // (what the rows lack is summed in 32 bits)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "R * max_pages must be below 2^31");
  if ((static_cast<long long>(v.pages) << v.log_page) > 0x7FFFFFFFll)
    return cache_fail(DARTREE_ERR_UNSUPPORTED, "a slot's number must be below 2^31");
  PlanParams p{cache->refs, table, lens, count, ok,     start,  row,   pos,        slot,
               v.pages,     v.log_page, max_pages, R, offset, window, sinks, max_tokens, max_tokens <= kOwnMaps, err};
  static std::atomic<uint64_t> done{0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = opt_in_smem(k_cache_plan, &done);
  if (e == cudaSuccess)
    e = launch_kernel_cluster(k_cache_plan, dim3(kMaxCl), dim3(kPlanThreads), sizeof(PlanSmem), st, true, kMaxCl, p);
  if (e == cudaSuccess && !p.own_maps)
    e = launch_kernel(k_cache_maps, dim3((max_tokens - 1) / 1024 + 1), dim3(256), 0, st, true, p);
  return cache_launched(e);
}
