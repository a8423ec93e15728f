// paged_host.h -- host-side checks and the tensor map of the paged cache.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "host_common.h"
#include "paged_index.h"

namespace fa {

inline bool cache_dim(int d) { return d == 64 || d == 80 || d == 96 || d == 128; }

// The cache as [num_pages * heads, 64, head_dim] bytes; a box is one (page,
// head), its rows padded with zeros to the kernel's head dim.
inline bool encode_cache(CUtensorMap* m, const void* base, int head_dim, int cells, int row) {
  const EncodeTiledFn fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)kPageTokens, (cuuint64_t)cells};
  cuuint64_t strides[2] = {(cuuint64_t)head_dim, (cuuint64_t)head_dim * kPageTokens};
  cuuint32_t box[3] = {(cuuint32_t)row, (cuuint32_t)kPageTokens, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Sizes of the cache and the arrays that come with it.
inline fa_status check_cache(const void* k_cache, const void* v_cache, const float* k_scale,
                      const float* v_scale, const int* cu, const int* page_table, int batch,
                      int total, int heads_k, int head_dim, int num_pages, int max_pages) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !cu || !page_table) return FA_ERR_INVALID_ARG;
  if (batch < 1 || total < 0 || heads_k < 1 || num_pages < 1 || max_pages < 1)
    return FA_ERR_INVALID_ARG;
  if (!is_aligned(k_cache, 16) || !is_aligned(v_cache, 16) || !is_aligned(k_scale, 4) ||
      !is_aligned(v_scale, 4) || !is_aligned(cu, 4) || !is_aligned(page_table, 4))
    return FA_ERR_INVALID_ARG;
  if (!cache_dim(head_dim)) return FA_ERR_UNSUPPORTED;
  // Positions of a sequence, (page, head) cells and packed rows are 32-bit.
  if ((int64_t)max_pages * kPageTokens > INT32_MAX || (int64_t)num_pages * heads_k > INT32_MAX ||
      (int64_t)total * heads_k > INT32_MAX || heads_k > 32767)
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace fa
