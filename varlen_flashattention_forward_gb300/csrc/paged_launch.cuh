// paged_launch.cuh -- launches of paged_attn_kernel and its merge.
#pragma once

#include <atomic>
#include <cstring>

#include "paged_attn_kernel.cuh"

namespace fa {

template <int D, int N, int kMask>
cudaError_t launch_attn(const CUtensorMap& k_map, const CUtensorMap& v_map, const PagedAttnArgs& a,
                        int grid, cudaStream_t stream) {
  // Set once per device; concurrent first calls may both set it (the call is
  // idempotent), the flag itself is atomic.
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int smem = (int)paged_smem<D, N>();
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(paged_attn_kernel<D, N, kMask>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_done[dev].store(true, std::memory_order_release);
  }
  paged_attn_kernel<D, N, kMask><<<grid, kPagedThreads, smem, stream>>>(k_map, v_map, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid < 2) return e;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(grid - 1, N);
  cfg.blockDim = dim3(D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, N>, a);
}

// The instantiation for padded head dim `dim` and `rows` rows a tile (16 under a
// mask: more rows go to paged_wide_kernel).
template <int kMask>
cudaError_t launch_attn_shape(int dim, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                              const PagedAttnArgs& a, int grid, cudaStream_t stream) {
  if constexpr (kMask == kNoMask) {
    if (rows == 32)
      return dim == 64 ? launch_attn<64, 32, kMask>(k_map, v_map, a, grid, stream)
                       : launch_attn<128, 32, kMask>(k_map, v_map, a, grid, stream);
  }
  if (rows != 16) return cudaErrorInvalidValue;
  return dim == 64 ? launch_attn<64, 16, kMask>(k_map, v_map, a, grid, stream)
                   : launch_attn<128, 16, kMask>(k_map, v_map, a, grid, stream);
}
// Those of the masked ones, in translation units of their own.
cudaError_t launch_attn_sinks(int dim, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                              const PagedAttnArgs& a, int grid, cudaStream_t stream);
cudaError_t launch_attn_tree(int dim, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             const PagedAttnArgs& a, int grid, cudaStream_t stream);

// Those of paged_wide_kernel and its merge (256 rows a tile), for any of the masks.
cudaError_t launch_attn_wide(int dim, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             const PagedAttnArgs& a, int grid, cudaStream_t stream);

}  // namespace fa
