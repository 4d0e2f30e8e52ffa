// Values of the 8-bit blocks: e4m3 (four significant bits, exponents from -6,
// largest 448, no infinities) and the block's power-of-two scale.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace shmm_dev {

__device__ __forceinline__ float finite_abs(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? __uint_as_float(b) : 0.0f;
}

// The scale's exponent for a block's largest finite magnitude: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return amax == 0.0f ? 0 : e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two values to e4m3 (the first in the low byte), no infinities among them.
__device__ __forceinline__ uint32_t finite_to_e4m3x2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// ... any values: infinities become NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    if (fabsf(a) == INFINITY) a = NAN;
    if (fabsf(b) == INFINITY) b = NAN;
    return finite_to_e4m3x2(a, b);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xFFFFu), __NV_E4M3);
    return __half22float2(__half2(h));
}

}  // namespace shmm_dev
