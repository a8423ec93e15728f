// rope_row.cuh -- one head row of q or k: RMS norm and position rotation.
//
//   y = x * w / sqrt(mean(x^2) + eps)          (w == nullptr: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin)   for the pairs of the first
//                                              rot_dim dims
//
// A row is held by a group of LANES neighbouring lanes, 8 dims each, in two
// pieces of 4 (8-byte loads) so chosen that both dims of a pair are in one
// lane: with the half split, lanes below rot_dim / 8 hold dims [4 l, 4 l + 4)
// and the ones rot_dim / 2 further on.  Rotating then takes no shuffles, and a
// lane needs 4 angles of the table row, not 8.  (With 16-byte pieces and
// shuffles, 8192 tokens x 40 heads of 128 dims took 51 us, 38 without.)
//
// Everything is fp32 from the load on; the caller rounds the result once, so
// that norm and rotation add no rounding of their own to the bf16 or e4m3
// result.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fa {

struct RopeParams {
  const float* table;  // [positions, rot_dim]: cos of the pairs, then sin (or null)
  int rot_dim;         // multiple of 16, 0 = no rotation
  int interleaved;     // pairs (2i, 2i + 1) instead of (i, i + rot_dim / 2)
};

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// Dims that lane `sub` of a row holds: [a, a + 4) and [b, b + 4), a < 0: none.
struct RowPieces {
  int a, b;
  bool turns;  // within rot_dim
};
__device__ __forceinline__ RowPieces row_pieces(const RopeParams& r, int sub, int dim) {
  RowPieces p;
  p.turns = sub * 8 < r.rot_dim;
  if (p.turns && !r.interleaved) {
    p.a = sub * 4;
    p.b = sub * 4 + (r.rot_dim >> 1);
  } else {
    p.a = sub * 8;
    p.b = sub * 8 + 4;
  }
  if (sub * 8 >= dim) p.a = -1;
  return p;
}

// A lane's 8 dims of a row, x[0..3] at piece a and x[4..7] at piece b.
struct RowBits {
  uint2 a, b;
};
__device__ __forceinline__ void unpack_row(const RowBits& v, float* x) {
  unpack_bf16x8(make_uint4(v.a.x, v.a.y, v.b.x, v.b.y), x);
}

// The 4 angles of this lane's pairs.
struct RopeRow {
  float4 c, s;
};
__device__ __forceinline__ RopeRow load_rope(const RopeParams& r, const float* row, int sub) {
  RopeRow t;
  t.c = *reinterpret_cast<const float4*>(row + sub * 4);
  t.s = *reinterpret_cast<const float4*>(row + (r.rot_dim >> 1) + sub * 4);
  return t;
}

// Scales the row by w / rms, or where `norm` is false by w.  Lanes past the
// head dim hold zeros; every lane of the warp takes part.
template <int LANES>
__device__ __forceinline__ void norm_row(float* x, const float* w, float inv_dim, float eps,
                                         bool norm = true) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = norm ? rsqrtf(fmaf(sum, inv_dim, eps)) : 1.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
}

// Rotates the lane's pairs in place.
__device__ __forceinline__ void rotate_row(float* x, const RopeParams& r, const RopeRow& t) {
  const float c[4] = {t.c.x, t.c.y, t.c.z, t.c.w}, s[4] = {t.s.x, t.s.y, t.s.z, t.s.w};
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[i], b = x[4 + i];
      x[i] = a * c[i] - b * s[i];
      x[4 + i] = b * c[i] + a * s[i];
    }
  }
}

}  // namespace fa
