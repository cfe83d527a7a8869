// Work items of the grouped products: the chunks of rows of the groups that
// have rows, found by every CTA from the offsets (internal).
#pragma once

#include "internal.h"

namespace moe {

// The chunks of rows of the groups that have rows and an expert, in order:
// (group, first row); their number.
template <int WARPS, typename A>
__device__ int find_chunks(const A& a, int2* chunks) {
  __shared__ int count[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int total = 0;
  for (int g0 = 0; g0 < a.n_groups; g0 += WARPS * 32) {
    const int g = g0 + threadIdx.x;
    int n = 0, row = 0;
    if (g < a.n_groups) {
      row = max(0, a.offsets[g]);
      const int rows = min(a.rows, a.offsets[g + 1]) - row;
      if (rows > 0) n = (rows - 1) / a.chunk + 1;
      const int ex = n > 0 && a.map ? a.map[g] : g < a.n_experts ? g : -1;
      if (n > 0 && (ex < 0 || ex >= a.n_experts)) {
        n = 0;
        if (blockIdx.x == 0 && a.status)
          atomicOr(a.status, MOE_DEV_BAD_INDEX);
      }
    }
    int upto = n;  // of this warp's groups, this one's included
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += below;
    }
    if (lane == 31) count[warp] = upto;
    __syncthreads();
    int at = total + upto - n;
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) at += count[w];
      total += count[w];
    }
    // offsets that overlap could make more than there is room for
    for (int i = 0; i < n && at + i < a.chunks; ++i)
      chunks[at + i] = make_int2(g, row + i * a.chunk);
    __syncthreads();
  }
  return min(total, a.chunks);
}
// The end of the chunk's rows.
template <typename A>
__device__ __forceinline__ int chunk_end(const A& a, int2 c) {
  const int end = min(a.rows, a.offsets[c.x + 1]);
  return end - c.y > a.chunk ? c.y + a.chunk : end;
}

}  // namespace moe
