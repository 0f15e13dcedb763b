// Device helpers of the 8-bit paged KV cache: e4m3 codes with a scale for each page and
// kv head (see hspec.h).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace hspec {

// Scale of a page and head whose largest finite magnitude is amax: 0 for amax = 0, else
// 2^k with the least k >= -126 such that amax <= 448 * 2^k = 1.75 * 2^(8 + k): from
// amax = m 2^E, k = E - 8, one more when m > 1.75.
__device__ __forceinline__ float kv8_scale_of(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const int b = __float_as_int(amax);
  const int e = (b >> 23) - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
  return __int_as_float(max(e, 1) << 23);
}

// 1 / s for a scale of kv8_scale_of (a normal power of two, so exact).  1 for s = 0, where the
// finite values are zeros anyway and an infinity has to become the largest code, not 0 * inf.
__device__ __forceinline__ float kv8_inverse(float s) {
  return s > 0.f ? __int_as_float((254 << 23) - __float_as_int(s)) : 1.f;
}

// |v| for the scale's choice: infinities and NaN do not take part.
__device__ __forceinline__ float kv8_mag(float v) {
  const float m = fabsf(v);
  return m <= 3.402823466e38f ? m : 0.f;
}

// Two values to e4m3 (to nearest even, magnitudes above 448 saturate, NaN stays NaN);
// `a` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// The two e4m3 codes in the low 16 bits of `r` as values (exact in fp16).
__device__ __forceinline__ __half2 e4m3x2_to_h2(uint32_t r) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)r));
  return *reinterpret_cast<__half2*>(&h);
}
__device__ __forceinline__ float2 e4m3x2_to_f2(uint32_t r) { return __half22float2(e4m3x2_to_h2(r)); }
__device__ __forceinline__ float e4m3_to_f(uint8_t c) { return e4m3x2_to_f2(c).x; }

}  // namespace hspec
