// host_common.h -- host-side facts that the entry points of every translation
// unit share (defined in fa_api.cu).  Internal; the public interface is
// include/fa_gb300.h.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "../../include/fa_gb300.h"

namespace fa {

// SM count, status word address and the pipeline wait limit of the current
// device; FA_ERR_ARCH when it is not sm_103.
struct DeviceFacts {
  int sm_count = 0;
  unsigned int* status = nullptr;
  unsigned long long wait_limit_ns = 0;
};
fa_status device_facts(DeviceFacts* out);

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled of the driver, or nullptr.
EncodeTiledFn tensor_map_encoder();

inline bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// A strided [tokens, heads, dim] view of bf16: innermost dimension
// contiguous, head and token strides multiples of 16 bytes, no element
// reachable two ways.
inline bool is_valid_view(long long row_stride, long long head_stride, int heads, int dim) {
  if (row_stride <= 0 || head_stride <= 0) return false;
  if (row_stride % 8 != 0 || head_stride % 8 != 0) return false;
  if (head_stride < dim) return false;
  if (row_stride < (long long)(heads - 1) * head_stride + dim) return false;
  return row_stride < (1ll << 37) && head_stride < (1ll << 37);
}

}  // namespace fa
