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
// lane needs 4 angles of the table row, not 8.  (At 8192
// tokens x 40 heads of 128 dims, 16-byte pieces and shuffles took 51 us where
// this took 33.)
//
// Everything is fp32 from the load on; the caller rounds the result once, so
// that norm and rotation add no rounding of their own to the bf16 or e4m3
// result.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "sm103_ptx.cuh"

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

// A lane's 8 dims of a row as bf16, and as 4 pairs of fp32: x[0], x[1] at piece
// a, x[2], x[3] at piece b.  (Arithmetic is on pairs: half the instructions,
// of which these kernels are as short as of bandwidth.)
struct RowBits {
  uint2 a, b;
};
// Where no pair is split between pieces, every lane's lie together and go with
// one 16-byte access.
__device__ __forceinline__ bool whole_pieces(const RopeParams& r) {
  return r.interleaved || r.rot_dim == 0;
}
__device__ __forceinline__ RowBits load_row(const uint16_t* row, const RowPieces& p, bool whole) {
  RowBits v;
  if (whole) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + p.a);
    v.a = make_uint2(u.x, u.y);
    v.b = make_uint2(u.z, u.w);
  } else {
    v.a = *reinterpret_cast<const uint2*>(row + p.a);
    v.b = *reinterpret_cast<const uint2*>(row + p.b);
  }
  return v;
}
__device__ __forceinline__ void store_row(uint16_t* row, const RowPieces& p, bool whole,
                                          const RowBits& v) {
  if (whole) {
    *reinterpret_cast<uint4*>(row + p.a) = make_uint4(v.a.x, v.a.y, v.b.x, v.b.y);
  } else {
    *reinterpret_cast<uint2*>(row + p.a) = v.a;
    *reinterpret_cast<uint2*>(row + p.b) = v.b;
  }
}
__device__ __forceinline__ void unpack_row(const RowBits& v, uint64_t* x) {
  const uint32_t w[4] = {v.a.x, v.a.y, v.b.x, v.b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = ptx::f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// The 4 angles of this lane's pairs of dims, two by two; ns = -s.
struct RopeRow {
  uint64_t c[2], s[2], ns[2];
};
__device__ __forceinline__ RopeRow load_rope(const RopeParams& r, const float* row, int sub) {
  const float4 c = *reinterpret_cast<const float4*>(row + sub * 4);
  const float4 s = *reinterpret_cast<const float4*>(row + (r.rot_dim >> 1) + sub * 4);
  RopeRow t;
  t.c[0] = ptx::f2_pack(c.x, c.y);
  t.c[1] = ptx::f2_pack(c.z, c.w);
  t.s[0] = ptx::f2_pack(s.x, s.y);
  t.s[1] = ptx::f2_pack(s.z, s.w);
  t.ns[0] = ptx::f2_pack(-s.x, -s.y);
  t.ns[1] = ptx::f2_pack(-s.z, -s.w);
  return t;
}

// Scales the row by w / rms, or where `norm` is false by w.  Lanes past the
// head dim hold zeros; every lane of the warp takes part.
template <int LANES>
__device__ __forceinline__ void norm_row(uint64_t* x, const uint64_t* w, float inv_dim, float eps,
                                         bool norm = true) {
  uint64_t sums = ptx::mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) sums = ptx::fma2(x[i], x[i], sums);
  float lo, hi;
  ptx::f2_unpack(sums, lo, hi);
  float sum = lo + hi;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = norm ? rsqrtf(fmaf(sum, inv_dim, eps)) : 1.f;
  const uint64_t r2 = ptx::f2_pack(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = ptx::mul2(x[i], ptx::mul2(r2, w[i]));
}

// Rotates the lane's pairs of dims in place.
__device__ __forceinline__ void rotate_row(uint64_t* x, const RopeParams& r, const RopeRow& t) {
  if (r.interleaved) {
    float c[4], s[4];
    ptx::f2_unpack(t.c[0], c[0], c[1]);
    ptx::f2_unpack(t.c[1], c[2], c[3]);
    ptx::f2_unpack(t.s[0], s[0], s[1]);
    ptx::f2_unpack(t.s[1], s[2], s[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      ptx::f2_unpack(x[i], a, b);
      x[i] = ptx::f2_pack(a * c[i] - b * s[i], b * c[i] + a * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t a = x[i], b = x[2 + i];
      x[i] = ptx::fma2(a, t.c[i], ptx::mul2(b, t.ns[i]));
      x[2 + i] = ptx::fma2(b, t.c[i], ptx::mul2(a, t.s[i]));
    }
  }
}

// The lane's 8 weights as pairs.
__device__ __forceinline__ void load_weights(const float* w, const RowPieces& p, uint64_t* out) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(w + p.a));
  const float4 v = __ldg(reinterpret_cast<const float4*>(w + p.b));
  out[0] = ptx::f2_pack(u.x, u.y);
  out[1] = ptx::f2_pack(u.z, u.w);
  out[2] = ptx::f2_pack(v.x, v.y);
  out[3] = ptx::f2_pack(v.z, v.w);
}

}  // namespace fa
