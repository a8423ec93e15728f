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
  unsigned units;        // tokens * groups
  int groups_q, groups;  // units of a token: of its q heads, of all
  int dim;
  float inv_dim, eps;
  RopeParams rope;
  const int* positions;  // null: no rotation and no token is skipped
  int max_pos;
};

// One group of LANES lanes takes one unit: up to ROWS neighbouring heads of
// one token, of q or of k, whose rows are all loaded before the first is
// used.  The table row and the weights (32 + 32 bytes a lane, against 16 of a
// row) are loaded once for all of them.
template <int LANES, int ROWS>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const QkNormRopeArgs a) {
  const int sub = threadIdx.x % LANES;
  const RowPieces p = row_pieces(a.rope, sub, a.dim);
  const unsigned unit = (blockIdx.x * 256u + threadIdx.x) / LANES;
  const bool real = unit < a.units;
  const unsigned token = real ? unit / (unsigned)a.groups : 0;
  const int group = real ? (int)(unit - token * a.groups) : 0;
  const bool is_q = group < a.groups_q;
  const QkSide& side = is_q ? a.q : a.k;
  const int head0 = (is_q ? group : group - a.groups_q) * ROWS;
  const int rows = (is_q ? a.heads : a.heads_k) - head0;  // (may be over ROWS)
  int pos = 0;
  bool live = real && p.a >= 0;
  if (a.positions) {
    pos = __ldg(a.positions + token);
    live = live && pos >= 0 && pos < a.max_pos;
  }
  const uint16_t* in = side.in + (long long)token * side.in_row + (long long)head0 * side.in_head;
  RowBits raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    raw[i].a = raw[i].b = make_uint2(0u, 0u);
    // (Not through the read-only path: the output may be the input.)
    if (live && i < rows) {
      raw[i].a = *reinterpret_cast<const uint2*>(in + i * side.in_head + p.a);
      raw[i].b = *reinterpret_cast<const uint2*>(in + i * side.in_head + p.b);
    }
  }
  RopeRow t;
  const bool turn = live && p.turns;
  if (turn) t = load_rope(a.rope, a.rope.table + (long long)pos * a.rope.rot_dim, sub);
  const bool any_weight = a.q.weight != nullptr || a.k.weight != nullptr;
  const float* wp = side.weight;
  float w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (wp && p.a >= 0) {
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(wp + p.a));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(wp + p.b));
    w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
    w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
  }
  uint16_t* out = side.out + (long long)token * side.out_row + (long long)head0 * side.out_head;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float x[8];
    unpack_row(raw[i], x);
    // (A warp can hold rows of q and of k: every lane goes through the
    // shuffles, a side without a weight is scaled by 1.)
    if (any_weight) norm_row<LANES>(x, w, a.inv_dim, a.eps, wp != nullptr);
    if (turn) rotate_row(x, a.rope, t);
    if (live && i < rows) {
      *reinterpret_cast<uint2*>(out + i * side.out_head + p.a) =
          make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
      *reinterpret_cast<uint2*>(out + i * side.out_head + p.b) =
          make_uint2(ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
    }
  }
}

}  // namespace fa
