// Exclusive scan over a block.
#pragma once

#include <stdint.h>

namespace mla {

// Exclusive scan over the block's T threads of one value each; *total = the
// sum.  red holds T / 32 values in shared memory.
template <int T, typename V>
__device__ __forceinline__ V block_scan(V v, V* red, V* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  V x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                                     // an earlier scan's readers of red are done
  if (lane == 31) red[warp] = x;
  __syncthreads();
  V s = lane < T / 32 ? red[lane] : V(0);
#pragma unroll
  for (int o = 1; o < T / 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, T / 32 - 1);
  const V base = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp ? base : V(0)) + x - v;
}

}  // namespace mla
