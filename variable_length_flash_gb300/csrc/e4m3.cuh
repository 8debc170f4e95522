// Rounding to e4m3 and back, and the scale that a page of a cache gets.
#pragma once

#include "common.cuh"

namespace vlf {

// Two values as e4m3 (nearest, ties to even; beyond 448 its largest), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// The two e4m3 values of the low 16 bits of x (exact).
__device__ __forceinline__ float2 e4m3_pair(uint32_t x) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)x));
  return __half22float2(*reinterpret_cast<__half2 *>(&h));
}
// x as a page holds it: e4m3, a value that is not finite as a NaN of its sign.
__device__ __forceinline__ uint32_t e4m3_byte(float x, float inv_scale) {
  const uint32_t u = __float_as_uint(x);
  if ((u & 0x7f800000u) == 0x7f800000u) return 0x7fu | u >> 24 & 0x80u;
  return e4m3x2(x * inv_scale, 0.f) & 0xffu;
}

// The smallest power of two, 2^-64 at least, times which 448 is not below amax (finite, >= 0): 448 is
// 1.75 2^8, so it is amax's own exponent less 8, or less 7 where its mantissa is above 1.75.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased
  return __uint_as_float((uint32_t)max(e, 127 - 64) << 23);
}

}  // namespace vlf
