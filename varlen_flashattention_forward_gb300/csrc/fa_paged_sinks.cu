// Instantiations of the paged attention kernel for rows with sinks behind a sliding window.
#include "paged_launch.cuh"

namespace fa {

cudaError_t launch_attn_sinks(int dim, int rows, const CUtensorMap& k_map, const CUtensorMap& v_map,
                              const PagedAttnArgs& a, int grid, cudaStream_t stream) {
  return launch_attn_shape<kSinkMask>(dim, rows, k_map, v_map, a, grid, stream);
}

}  // namespace fa
