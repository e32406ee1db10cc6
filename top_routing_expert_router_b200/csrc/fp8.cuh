// fp8.cuh -- E4M3 conversion of 1 x 128 activation tiles, shared by the row quantiser, the norm
// and the few-token layer.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

// UE8M0 exponent of a tile whose largest magnitude is amax (finite binary32):
// with amax = f * 2^x, f in [0.5, 1), amax <= 448 * 2^e  <=>  f * 2^(x - 8 - e) <= 1.75,
// so e = x - 9 when f <= 0.875 and x - 8 otherwise. For a normal amax = 1.m * 2^(E - 127)
// that is x = E - 126 and f <= 0.875 <=> m <= 0.75, read straight off the bits.
__device__ __forceinline__ int ue8m0_exponent(float amax) {
  if (!(amax > 0.0f)) return 0;
  const uint32_t u = __float_as_uint(amax);
  const int E = (int)(u >> 23);
  int e;
  if (E > 0) {
    e = (u & 0x7FFFFFu) <= 0x600000u ? E - 135 : E - 134;
  } else {  // binary32 subnormal
    int x;
    const float f = frexpf(amax, &x);
    e = f <= 0.875f ? x - 9 : x - 8;
  }
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

// 2^-e as a binary32 (normal for the exponents bf16 inputs produce, -127 <= e <= 119).
__device__ __forceinline__ float pow2_neg(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// E4M3 codes of four values times sc, round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d, float sc) {
  const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * sc, b * sc), __NV_SATFINITE, __NV_E4M3);
  const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * sc, d * sc), __NV_SATFINITE, __NV_E4M3);
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

}  // namespace moe
