// Arithmetic of the 8-bit latent cache's format: e4m3 codes and power-of-two scale bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace kdt {
namespace q8 {

constexpr int kNaN = 255;                 // scale byte of a group that holds an infinity or NaN

// Scale byte of a group whose largest magnitude has the float32 bit pattern `top`: with e the
// least integer such that top <= 448 * 2^e = 1.75 * 2^(e + 8), clamped to [-100, 100], the
// byte is e + 127.
__device__ __forceinline__ int scale_byte(uint32_t top) {
    if (top >= 0x7f800000u) return kNaN;
    const int e = (int)(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return (top == 0u ? -100 : min(max(e, -100), 100)) + 127;
}

// 2^(byte - 127) as float32; NaN for kNaN (a byte of 0, never written, gives 0).
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return __uint_as_float(byte == (uint32_t)kNaN ? 0x7fffffffu : byte << 23);
}

// 2^-(byte - 127); 0 for kNaN.
__device__ __forceinline__ float inverse_scale(int byte) {
    return byte == kNaN ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}

// Four values to four codes (round to nearest even, magnitudes above 448 to 448), value 0 in
// the low byte.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Four codes to their values.
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * h)), __NV_E4M3);
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&r));
        f[2 * h] = v.x;
        f[2 * h + 1] = v.y;
    }
}

}  // namespace q8
}  // namespace kdt
