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

// Widening to bf16 for the matrix instructions, exactly. A code's exponent and mantissa bits,
// moved to where a bf16 number's sit, are the value times 2^-120 (subnormal codes included: they
// become subnormal bf16 numbers), so one product by 2^(byte - 127 + 120) restores it. For bytes
// above kHighByte that is no bf16 number: factor() then stops there and factor_high() is the
// rest, for a second product. A NaN group's factor is 0 (its key is flagged instead).
constexpr uint32_t kHighByte = 134;

__device__ __forceinline__ uint32_t factor(uint32_t byte) {              // bf16 bits
    return byte == (uint32_t)kNaN ? 0u : (min(byte, kHighByte) + 120u) << 7;
}

__device__ __forceinline__ uint32_t factor_high(uint32_t byte) {
    return (max(byte, kHighByte) - kHighByte + 127u) << 7;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Codes (0, 2) and (1, 3) of a word as pairs of bf16 bit patterns times 2^-120. The byte permute
// puts each code in the low byte of its half and copies of its sign in the high byte: 16 times
// that has the sign in bit 15 and exponent and mantissa in bits 4..10, and the rest (more signs,
// and what the lower half carries into the upper one's low bits) is masked away.
__device__ __forceinline__ void spread(uint32_t w, uint32_t &even, uint32_t &odd) {
    asm("prmt.b32 %0, %1, 0, 0xa280;" : "=r"(even) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xb391;" : "=r"(odd) : "r"(w));
    even = (even * 16u) & 0x87f087f0u;
    odd = (odd * 16u) & 0x87f087f0u;
}

// factor() of two scale bytes as a pair, when both are below 128 (no NaN, nothing for factor_high()).
__device__ __forceinline__ uint32_t low_factors(uint32_t b0, uint32_t b1) {
    return (b0 | b1 << 16) * 128u + 120u * 128u * 0x10001u;
}

// Eight codes to eight bf16 values, each four in the order (0, 2, 1, 3); f holds the factor twice.
__device__ __forceinline__ uint4 widen8(const uint2 &codes, uint32_t f) {
    uint4 o;
    spread(codes.x, o.x, o.y);
    spread(codes.y, o.z, o.w);
    o.x = mul_bf16x2(o.x, f);
    o.y = mul_bf16x2(o.y, f);
    o.z = mul_bf16x2(o.z, f);
    o.w = mul_bf16x2(o.w, f);
    return o;
}

// Eight bf16 values in order to the order widen8 gives.
__device__ __forceinline__ uint4 reorder8(const uint4 &v) {
    return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632), __byte_perm(v.z, v.w, 0x5410),
                      __byte_perm(v.z, v.w, 0x7632));
}

}  // namespace q8
}  // namespace kdt
