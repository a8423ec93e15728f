// qk_norm_rope_kernel.cuh -- per-head RMS norm of queries and keys with the
// position rotation, one pass over the data (the arithmetic is in
// rope_row.cuh).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "rope_row.cuh"
#include "sm103_ptx.cuh"

namespace fa {

struct QkSide {
  const uint16_t* in;
  uint16_t* out;
  long long in_row, in_head, out_row, out_head;  // strides in elements
  const float* weight;                           // [dim] or null (no norm)
};

struct QkNormRopeArgs {
  QkSide q, k;
  int heads, heads_k;
  long long units;       // tokens * ceil((heads + heads_k) / ROWS)
  int groups;            // units of a token
  int dim;
  float inv_dim, eps;
  RopeParams rope;
  const int* positions;  // null: no rotation and no token is skipped
  int max_pos;
};

// One group of LANES lanes takes one unit: ROWS neighbouring heads of one
// token (q heads, then k heads), whose rows are all loaded before the first
// is used; the table row is loaded once for all of them.
template <int LANES, int ROWS>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkNormRopeArgs a) {
  const int sub = threadIdx.x % LANES;
  const int dim0 = sub * 8;
  const bool in_dim = dim0 < a.dim;
  const long long unit = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / LANES;
  const bool real = unit < a.units;
  const long long token = real ? unit / a.groups : 0;
  const int head0 = real ? (int)(unit - token * a.groups) * ROWS : 0;
  int pos = 0;
  bool live = real && in_dim;
  if (a.positions) {
    pos = __ldg(a.positions + token);
    live = live && pos >= 0 && pos < a.max_pos;
  }
  uint4 raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = head0 + i;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (live && h < a.heads + a.heads_k) {
      const uint16_t* p = h < a.heads
                              ? a.q.in + token * a.q.in_row + h * a.q.in_head
                              : a.k.in + token * a.k.in_row + (h - a.heads) * a.k.in_head;
      raw[i] = *reinterpret_cast<const uint4*>(p + dim0);
    }
  }
  RopeRow t;
  if (live && a.rope.rot_dim) load_rope(a.rope, pos, dim0, &t);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = head0 + i;
    const bool is_q = h < a.heads;
    const float* wp = is_q ? a.q.weight : a.k.weight;
    float x[8];
    unpack_bf16x8(raw[i], x);
    // (A warp can hold rows of q and of k: every lane goes through the
    // shuffles, those without a weight keep their values.)
    float w[8], y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 1.f;
      y[j] = x[j];
    }
    if (wp && in_dim) {
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(wp + dim0));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(wp + dim0) + 1);
      w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
      w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
    }
    norm_row<LANES>(y, w, a.inv_dim, a.eps);
    if (wp) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = y[j];
    }
    if (a.rope.rot_dim) rotate_row<LANES>(x, a.rope, t, dim0);
    if (live && h < a.heads + a.heads_k) {
      uint16_t* p = is_q ? a.q.out + token * a.q.out_row + h * a.q.out_head
                         : a.k.out + token * a.k.out_row + (h - a.heads) * a.k.out_head;
      *reinterpret_cast<uint4*>(p + dim0) =
          make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                     ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
    }
  }
}

}  // namespace fa
