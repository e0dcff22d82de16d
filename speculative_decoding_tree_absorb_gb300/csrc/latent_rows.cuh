// Rows of latents and rope keys on their way into a cache: what the kernels that write them share.
#pragma once

#include <cmath>

#include "kdt_internal.cuh"

namespace kdt {
namespace rows {

constexpr int kHalf = kDr / 2;

// Frequencies of the rotation in turns: pos * w_j / 2 pi as a fixed-point fraction of a turn
// with 64 fractional bits, so pos * f wraps to the exact angle modulo a full turn.
struct TurnFreqs {
    uint64_t f[kHalf];
};

inline TurnFreqs turn_freqs(double base) {
    TurnFreqs fr;
    for (int j = 0; j < kHalf; ++j) {
        // base^(-2j/64) radians a position, as a fraction of a turn (whole turns drop out)
        const double t = pow(base, -(double)j / kHalf) * 0.15915494309189533577;
        fr.f[j] = (uint64_t)((t - floor(t)) * 18446744073709551616.0);
    }
    return fr;
}

// (k0, k1) rotated by position pos, freq the pair's: the angle in turns, exact modulo 1, rounded to 32 bits,
// is within [-1/2, 1/2); each product and sum rounded on its own.
__device__ __forceinline__ void rotate(float &k0, float &k1, int32_t pos, uint64_t freq) {
    const int32_t turn = (int32_t)(((uint64_t)(int64_t)pos * freq + 0x80000000ull) >> 32);
    float s, c;
    sincospif((float)turn * 4.656612873077393e-10f, &s, &c);     // 2^-31: half turns
    const float r0 = __fsub_rn(__fmul_rn(k0, c), __fmul_rn(k1, s));
    k1 = __fadd_rn(__fmul_rn(k1, c), __fmul_rn(k0, s));
    k0 = r0;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <bool kOnce, typename V> __device__ __forceinline__ V once(const V *p) {
    return kOnce ? __ldcs(p) : __ldg(p);
}

// A lane's 16 latent elements of a row, as kPieces pieces of kPer consecutive ones: piece q
// starts at element q * 32 * kPer + lane * kPer, so every warp load is contiguous.
template <typename E> struct Row;
template <> struct Row<float> {
    static constexpr int kPer = 4, kPieces = 4;
    float4 v[4];
    template <bool kOnce> __device__ __forceinline__ void load(const float *p, int lane) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = once<kOnce>(reinterpret_cast<const float4 *>(p) + 32 * q + lane);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[4 * q] = v[q].x;
            x[4 * q + 1] = v[q].y;
            x[4 * q + 2] = v[q].z;
            x[4 * q + 3] = v[q].w;
        }
    }
};
template <> struct Row<__nv_bfloat16> {
    static constexpr int kPer = 8, kPieces = 2;
    uint4 v[2];
    template <bool kOnce> __device__ __forceinline__ void load(const __nv_bfloat16 *p, int lane) {
#pragma unroll
        for (int q = 0; q < 2; ++q) v[q] = once<kOnce>(reinterpret_cast<const uint4 *>(p) + 32 * q + lane);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[8 * q + 2 * t] = __uint_as_float(w[t] << 16);
                x[8 * q + 2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
            }
        }
    }
};

// y <- y r gamma, r = 1 / sqrt(mean y^2 + eps), in float32; one warp holds the row.
template <typename E>
__device__ __forceinline__ void rms_norm(float (&y)[16], const E *gamma, float eps, int lane) {
    Row<E> gr;                                        // from L1 for each row: 16 registers less
    gr.template load<false>(gamma, lane);
    float ss = 0.f;
#pragma unroll
    for (int t = 0; t < 16; ++t) ss = fmaf(y[t], y[t], ss);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = __frsqrt_rn(fmaf(ss, 1.f / kDc, eps));
    float g[16];
    gr.get(g);
#pragma unroll
    for (int t = 0; t < 16; ++t) y[t] = y[t] * r * g[t];
}

}  // namespace rows
}  // namespace kdt
