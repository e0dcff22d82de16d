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

// 16 codes of one group to 16 bf16 values times 2^(byte - 127), exactly, as two 16-byte
// vectors in order; a NaN group gives zeros. The code's exponent and mantissa bits, moved to
// where a bf16 number's sit, are the value times 2^-120 (subnormal codes included: they
// become subnormal bf16 numbers), so one product by 2^(byte - 7) restores it. Scales above
// 2^7 need a second product, as 2^(byte - 7) is then no bf16 number.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ void widen16(const uint4 &codes, uint32_t byte, uint4 &lo, uint4 &hi) {
    const uint32_t top = byte > 134u ? 134u : byte;
    uint32_t f = byte == (uint32_t)kNaN ? 0u : (top + 120u) << 7;
    f |= f << 16;
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // bytes 2h and 2h + 1 to the upper bytes of the two halves: s eeee mmm 0...
            const uint32_t x = __byte_perm(c[k], 0u, h == 0 ? 0x1404 : 0x3424);
            o[2 * k + h] = mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), f);
        }
    }
    if (byte > 134u && byte != (uint32_t)kNaN) {
        uint32_t f2 = (byte - 134u + 127u) << 7;
        f2 |= f2 << 16;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = mul_bf16x2(o[k], f2);
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace q8
}  // namespace kdt
