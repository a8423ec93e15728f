// cost_scan.cuh -- costs of the sequences before each one, in shared memory.
#pragma once

#include <cuda_runtime.h>

#include "named_bar.cuh"
#include "paged_index.h"

namespace fa {

// before[b] = sum of cost(0) .. cost(b - 1), capped, for b up to the batch; by
// the block's first kThreads threads (named barrier 1).
template <int kThreads, typename Cost>
__device__ __forceinline__ void scan_costs(int* before, long long* warp_sum, int batch, Cost cost) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) before[0] = 0;
  long long base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < batch; b0 += kThreads) {
    const int b = b0 + tid;
    long long sum = b < batch ? cost(b) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    named_bar_sync(1, kThreads);
    long long all = 0, lo = base;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) lo += warp_sum[w];
      all += warp_sum[w];
    }
    if (b < batch) before[b + 1] = capped_cost(lo + sum);
    base += all;
    named_bar_sync(1, kThreads);
  }
}

}  // namespace fa
