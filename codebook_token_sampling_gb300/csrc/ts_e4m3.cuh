// ts_e4m3.cuh -- rounding to 8 bits: the quotient by a scale, as the cache's writes
// and the 8-bit rows of the layer operators take it.
#pragma once

#include <cuda_fp8.h>

#include "ts_device.cuh"

namespace ts {

// y = x / scale correctly rounded, given inv = 1 / scale correctly rounded:
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor" (1990): with q within a unit of the quotient, q + (x - q scale) inv
// rounds to it where nothing over- or underflows.  The sign is q's, for zeros.
// Returns whether it serves: the scales that quotient_inverse gives an inverse
// for lie within 2^-90 .. 2^90, so x - q scale underflows only where the quotient
// rounds to an e4m3 zero, and quotients of 2^20 and more, infinite and NaN ones
// are left to the division.
__device__ __forceinline__ bool quotient(float x, float scale, float inv, float &y) {
  const float q = x * inv;
  y = copysignf(fmaf(fmaf(-q, scale, x), inv, q), q);
  return fabsf(q) < 0x1p20f;
}
__device__ __forceinline__ float quotient_inverse(float scale) {
  const float a = fabsf(scale);
  return a >= 0x1p-90f && a <= 0x1p90f ? __fdiv_rn(1.0f, scale) : 0.0f;
}
// The four e4m3 values nearest to y (ties to even, at most 448 in size).
__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ uint8_t e4m3_of(float a) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3));
}

}  // namespace ts
