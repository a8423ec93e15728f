// e4m3.cuh -- the 8-bit cache's numbers: codes, and the scale of a page.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "paged_index.h"
#include "sm103_ptx.cuh"

namespace fa {

constexpr float kE4m3Max = 448.f;
// Scales stay within 2^-64 .. 2^64: the attention's scores, and its sums of
// weights relative to weight times V scale, then stay inside fp32 (where sums
// meet, with root_ex2).
constexpr int kScaleExpMax = 64;

// Smallest power of two s with amax <= 448 s, clamped (amax finite, >= 0).
__device__ __forceinline__ float scale_for(float amax) {
  // amax = 1.m 2^e and 448 = 1.75 2^8.  (Below 2^-126 the exponent is clamped.)
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = imin(imax(e, -kScaleExpMax), kScaleExpMax);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Two fp32 values as e4m3 codes (round to nearest even, saturating at 448,
// NaN kept): lo in bits 0..7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two e4m3 (e5m2) codes as f16x2 (exact).
__device__ __forceinline__ uint32_t unpack_e4m3x2(uint32_t codes) {
  uint32_t d;
  const uint16_t c = (uint16_t)codes;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}
__device__ __forceinline__ uint32_t unpack_e5m2x2(uint32_t codes) {
  uint32_t d;
  const uint16_t c = (uint16_t)codes;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}
__device__ __forceinline__ float2 f16x2_floats(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
      "cvt.f32.f16 %1, h;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// A row of queries as two e4m3 terms: scaled by 2^(7 - e), e the exponent of
// its largest value mx, which puts that in [128, 256), it is hi + lo with hi =
// rn(q) and lo = rn(q - hi).  (Rows below 2^-100 keep a smaller size; their
// scores are zero in fp32 all the same.  mx may be infinite, see terms_scale.)
__device__ __forceinline__ int terms_exponent(float mx) {
  return imax((int)(__float_as_uint(mx) >> 23) - 127, -100);
}
__device__ __forceinline__ void split_terms(const float* x, int e, uint32_t* hi, uint32_t* lo) {
  // As f16 pairs, which hold a scaled bf16 exactly down to 2^-14, far below e4m3's
  // last step, and its difference to hi.  (A conversion takes longer than any
  // product: four of them for two values, through fp32 five.)
  const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t y = ptx::pack_f16x2(x[2 * k] * f, x[2 * k + 1] * f);
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    hi[k] = c;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(y) : "r"(unpack_e4m3x2(hi[k])));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    lo[k] = c;
  }
}
// The same row in three terms, hi in e4m3 and two in e5m2, off by at most 2^-17 (2^-24
// of the row's largest).  A bf16 has four bits behind hi's where hi is normal, which
// e5m2's three hold: they are 0 to 8 steps.  Below that hi leaves up to 2^-10, mid up to
// 2^-14 of it, and rest, whose last step is 2^-16, half of that.  (With mid in e4m3, whose
// last step is 2^-9, 2^-10 would be left to rest, and 2^-14 behind it.)
__device__ __forceinline__ void split_three(const float* x, int e, uint32_t* hi, uint32_t* mid,
                                            uint32_t* rest) {
  const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t y = ptx::pack_f16x2(x[2 * k] * f, x[2 * k + 1] * f);
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    hi[k] = c;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(y) : "r"(unpack_e4m3x2(hi[k])));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    mid[k] = c;
    asm("sub.f16x2 %0, %0, %1;" : "+r"(y) : "r"(unpack_e5m2x2(mid[k])));
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(y));
    rest[k] = c;
  }
}
// What the terms' products are to be multiplied by, for scores times `scale`:
// NaN for a row with an infinity or a NaN (mx infinite).
__device__ __forceinline__ float terms_scale(float mx, int e, float scale) {
  return mx < __int_as_float(0x7f800000) ? scale * __uint_as_float((uint32_t)(e - 7 + 127) << 23)
                                         : __int_as_float(0x7fffffff);
}

}  // namespace fa
