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

// Whether the strides are those of a [rows, heads, dim] view of bf16 (dim a
// multiple of 8): innermost dimension contiguous, head and row strides multiples
// of 16 bytes, no element reachable two ways.  A stride that nothing steps by,
// that of a single head or row, may be anything (a framework leaves what it
// likes there) and is replaced by an ordinary one.
inline bool settle_view(int rows, int heads, int dim, long long* row_stride,
                        long long* head_stride) {
  constexpr long long kMost = 1ll << 37;  // of a tensor map, in elements
  if (heads == 1) *head_stride = dim;
  if (*head_stride < dim || *head_stride % 8 != 0) return false;
  if (heads > 1 && *head_stride > (kMost - dim) / (heads - 1)) return false;
  const long long extent = (heads - 1) * *head_stride + dim;
  if (rows <= 1) *row_stride = extent;
  return *row_stride >= extent && *row_stride % 8 == 0 && *row_stride < kMost;
}

}  // namespace fa
