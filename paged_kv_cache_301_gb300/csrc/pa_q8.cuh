// The 8-bit cache: e4m3 codes with one power-of-two scale per (block, KV head).
//
// A stored value is code * scale.  e4m3 has four significant bits and reaches
// 448, so the scale that fits a block's largest magnitude a is the smallest
// power of two s >= 2^kMinScaleExp with a <= 448 s.  A power of two costs no
// significant bits (the codes are floating point), makes value / s and code * s
// exact, and lets a block that grows token by token move to a larger scale
// without drift: dividing an older code by a power of two only rounds when the
// code becomes subnormal.
#pragma once

#include <cuda_fp8.h>

#include "pa_common.cuh"

namespace pa {

constexpr int kMinScaleExp = -64;   // an all-zero block's scale is 2^-64

// The scale of a block whose largest finite magnitude is a (a >= 0, finite).
// a = m 2^x with 1 <= m < 2, and 448 = 1.75 * 2^8: s = 2^(x - 8) when m <= 1.75,
// twice that otherwise.
__device__ __forceinline__ float scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kMinScaleExp);          // subnormal and zero magnitudes included
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Largest finite magnitude: infinities and NaN do not set a scale (they are
// stored saturated, or as NaN).
__device__ __forceinline__ float finite_mag(float x) {
  const float a = fabsf(x);
  return a < __uint_as_float(0x7F800000u) ? a : 0.f;
}

// Two values rounded to nearest even e4m3 (saturating, NaN kept), a in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Two codes (low half of w) as fp32.
__device__ __forceinline__ float2 e4m3_widen2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Two fp32 values rounded to nearest in one conversion, the first in the low half.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (DT == PA_BFLOAT16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

}  // namespace pa
