// rope_row.cuh -- one head row of q or k: RMS norm and position rotation.
//
//   y = x * w / sqrt(mean(x^2) + eps)          (w == nullptr: y = x)
//   (a, b) -> (a cos - b sin, b cos + a sin)   for the pairs of the first
//                                              rot_dim dims
//
// A row is held by a group of LANES neighbouring lanes, 8 dims (one 16-byte
// load) each.  Everything is fp32 from the load on; the caller rounds the
// result once, so that norm and rotation add no rounding of their own to the
// bf16 or e4m3 result.
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

// cos and sin that this lane's 8 dims need of the position's table row: one
// for each dim (half split), or the 4 of its pairs in c[0..3] and s[0..3].
struct RopeRow {
  float c[8], s[8];
};

__device__ __forceinline__ void load_rope(const RopeParams& r, long long position, int dim0,
                                          RopeRow* out) {
  if (dim0 >= r.rot_dim) return;
  const int half = r.rot_dim >> 1;
  const float* row = r.table + position * r.rot_dim;
  const int at = r.interleaved ? dim0 >> 1 : (dim0 < half ? dim0 : dim0 - half);
  const float4* cp = reinterpret_cast<const float4*>(row + at);
  const float4* sp = reinterpret_cast<const float4*>(row + half + at);
  const float4 c0 = __ldg(cp), s0 = __ldg(sp);
  out->c[0] = c0.x; out->c[1] = c0.y; out->c[2] = c0.z; out->c[3] = c0.w;
  out->s[0] = s0.x; out->s[1] = s0.y; out->s[2] = s0.z; out->s[3] = s0.w;
  if (!r.interleaved) {
    const float4 c1 = __ldg(cp + 1), s1 = __ldg(sp + 1);
    out->c[4] = c1.x; out->c[5] = c1.y; out->c[6] = c1.z; out->c[7] = c1.w;
    out->s[4] = s1.x; out->s[5] = s1.y; out->s[6] = s1.z; out->s[7] = s1.w;
  }
}

// Scales the row by w / rms.  Lanes past the head dim hold zeros; every lane
// of the warp takes part.
template <int LANES>
__device__ __forceinline__ void norm_row(float* x, const float* w, float inv_dim, float eps) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float r = rsqrtf(fmaf(sum, inv_dim, eps));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= r * w[i];
}

// Rotates the row in place; every lane of the warp takes part.
template <int LANES>
__device__ __forceinline__ void rotate_row(float* x, const RopeParams& r, const RopeRow& t,
                                           int dim0) {
  if (r.interleaved) {
    if (dim0 < r.rot_dim) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * t.c[i] - b * t.s[i];
        x[2 * i + 1] = b * t.c[i] + a * t.s[i];
      }
    }
    return;
  }
  // The other dim of each pair is rot_dim / 2 away: the same place of the
  // lane rot_dim / 16 further on, or back.
  const int half = r.rot_dim >> 1;
  const bool first = dim0 < half;
  const int sub = dim0 >> 3;
  const int from = dim0 < r.rot_dim ? (first ? sub + half / 8 : sub - half / 8) : sub;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl_sync(0xffffffffu, x[i], from, LANES);
    if (dim0 < r.rot_dim) x[i] = first ? x[i] * t.c[i] - o * t.s[i] : x[i] * t.c[i] + o * t.s[i];
  }
}

}  // namespace fa
