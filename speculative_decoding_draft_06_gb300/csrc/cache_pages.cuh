// What the kernels that plan pages share.
#pragma once
#include "cache.cuh"

namespace dt {

constexpr int kPlanThreads = 1024;
constexpr int kMaxReserveRows = 4096;

// Exclusive prefix sum of one value per thread over the block (1024
// threads); *total is the block's sum.  sh: 33 numbers.
template <typename N>
__device__ __forceinline__ N block_exclusive(N v, N* sh, N* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  N inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N y = __shfl_up_sync(kFullMask, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) sh[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const N w = sh[lane];
    N wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const N y = __shfl_up_sync(kFullMask, wi, o);
      if (lane >= o) wi += y;
    }
    sh[lane] = wi - w;
    if (lane == 31) sh[32] = wi;
  }
  __syncthreads();
  const N out = sh[warp] + inc - v;
  *total = sh[32];
  __syncthreads();
  return out;
}

}  // namespace dt
