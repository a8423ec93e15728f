// qk_norm_rope_kernel.cuh -- per-head RMS norm of queries and keys with the
// position rotation, one pass over the data (the arithmetic is in
// rope_row.cuh).
//
// Bound by HBM: every row is read and written once.  8192 tokens x 40 heads of
// 128 dims take 30.1 us, 5.7 TB/s; 5003 x 32 of 96 dims 14.6 us, 4.3 TB/s (four
// of a group's 16 lanes are past the row); 64 tokens 2.25 us, the launch.  More
// heads together (eight), more resident blocks or loads of the next unit ahead
// of the stores all measured slower: reads and writes of the same DRAM pages
// then drift apart.
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
  const bool whole = whole_pieces(a.rope);
  const bool any_weight = a.q.weight != nullptr || a.k.weight != nullptr;
  // (Every lane of a warp goes through every turn, for the shuffles.)
  const unsigned per_grid = gridDim.x * (256u / LANES);
  for (unsigned first = (blockIdx.x * 256u + (threadIdx.x & ~31u)) / LANES; first < a.units;
       first += per_grid) {
    const unsigned unit = first + (threadIdx.x & 31u) / LANES;
    const bool real = unit < a.units;
    const unsigned token = real ? unit / (unsigned)a.groups : 0;
    const int group = real ? (int)(unit - token * a.groups) : 0;
    const bool is_q = group < a.groups_q;
    const QkSide& side = is_q ? a.q : a.k;
    const int head0 = (is_q ? group : group - a.groups_q) * ROWS;
    const int rows = (is_q ? a.heads : a.heads_k) - head0;  // (may be over ROWS)
    const int pos = a.positions ? __ldg(a.positions + token) : 0;
    const bool live = real && p.a >= 0 && (!a.positions || (pos >= 0 && pos < a.max_pos));
    const uint16_t* in = side.in + (long long)token * side.in_row + (long long)head0 * side.in_head;
    RowBits raw[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      raw[i].a = raw[i].b = make_uint2(0u, 0u);
      // (Not through the read-only path: the output may be the input.)
      if (live && i < rows) raw[i] = load_row(in + i * side.in_head, p, whole);
    }
    RopeRow t;
    const bool turn = live && p.turns;
    if (turn) t = load_rope(a.rope, a.rope.table + (long long)pos * a.rope.rot_dim, sub);
    const float* wp = side.weight;
    uint64_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = ptx::f2_pack(1.f, 1.f);
    if (wp && p.a >= 0) load_weights(wp, p, w);
    uint16_t* out = side.out + (long long)token * side.out_row + (long long)head0 * side.out_head;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      uint64_t x[4];
      unpack_row(raw[i], x);
      // (A warp can hold rows of q and of k: every lane goes through the
      // shuffles, a side without a weight is scaled by 1.)
      if (any_weight) norm_row<LANES>(x, w, a.inv_dim, a.eps, wp != nullptr);
      if (turn) rotate_row(x, a.rope, t);
      if (live && i < rows) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) ptx::f2_unpack(x[j], f[2 * j], f[2 * j + 1]);
        RowBits v;
        v.a = make_uint2(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]));
        v.b = make_uint2(ptx::pack_bf16x2(f[4], f[5]), ptx::pack_bf16x2(f[6], f[7]));
        store_row(out + i * side.out_head, p, whole, v);
      }
    }
  }
}

}  // namespace fa
