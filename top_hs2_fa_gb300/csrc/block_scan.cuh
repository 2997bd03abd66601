// block_scan.cuh — prefix sums over a block of 1024 threads.
#pragma once
#include "common.cuh"

namespace hs2 {

// Exclusive prefix sum over the block's 1024 threads (all call it); `total` is their sum.
// `sums`: 33 ints of shared memory of this use alone.
HS2_DEVI int block_prefix(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the sums of an earlier call have been read
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int own = sums[lane];
    int s = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s - own;
    if (lane == 31) sums[32] = s;
  }
  __syncthreads();
  total = sums[32];
  return sums[warp] + x - v;
}

}  // namespace hs2
