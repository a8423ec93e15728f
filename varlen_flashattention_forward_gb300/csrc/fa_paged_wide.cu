// Instantiations of the paged attention kernel for many rows a sequence.
#include "paged_launch.cuh"
#include "paged_wide_kernel.cuh"

namespace fa {
namespace {

template <int D>
cudaError_t launch(const CUtensorMap& k_map, const CUtensorMap& v_map, const PagedAttnArgs& a,
                   int grid, cudaStream_t stream) {
  // Set once per device; concurrent first calls may both set it (the call is
  // idempotent), the flag itself is atomic.
  static std::atomic<bool> attr_done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int smem = (int)wide_smem<D>();
  if (!attr_done[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(paged_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e != cudaSuccess) return e;
    attr_done[dev].store(true, std::memory_order_release);
  }
  paged_wide_kernel<D><<<grid, kWideThreads, smem, stream>>>(k_map, v_map, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || grid < 2) return e;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(grid - 1, 16);
  cfg.blockDim = dim3(kWideMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_wide_merge_kernel<D>, a);
}

}  // namespace

cudaError_t launch_attn_wide(int dim, const CUtensorMap& k_map, const CUtensorMap& v_map,
                             const PagedAttnArgs& a, int grid, cudaStream_t stream) {
  return dim == 64 ? launch<64>(k_map, v_map, a, grid, stream)
                   : launch<128>(k_map, v_map, a, grid, stream);
}

}  // namespace fa
