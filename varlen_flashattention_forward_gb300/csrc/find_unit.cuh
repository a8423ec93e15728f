// find_unit.cuh -- which sequence a block's work unit belongs to.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// The sequence and the place within it of work unit x, where sequence b has
// count(b) units, in order.  Called by the whole block (at most 1024 threads,
// whole warps); found.seq is -1 if there is no such unit.
struct FoundUnit {
  int seq, at;
};
template <typename Count>
__device__ __forceinline__ FoundUnit find_unit(int x, int batch, Count count) {
  __shared__ int s_warp[32];
  __shared__ FoundUnit s_found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  if (tid == 0) s_found.seq = -1;
  long long before = 0;  // units of the sequences of earlier turns
  for (int b0 = 0; b0 < batch; b0 += blockDim.x) {
    const int b = b0 + tid;
    const int c = b < batch ? count(b) : 0;
    int sum = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    long long lo = before;
    int all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) lo += s_warp[w];
      all += s_warp[w];
    }
    lo += sum - c;
    if (x >= lo && x < lo + c) {
      s_found.seq = b;
      s_found.at = (int)(x - lo);
    }
    before += all;
    __syncthreads();
    if (before > x) break;
  }
  __syncthreads();
  return s_found;
}

}  // namespace fa
