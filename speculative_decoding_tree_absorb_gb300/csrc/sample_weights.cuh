// Sampling weights in fixed point: what the kernels that draw tokens share. w = round(2^44 e^y), y a logit's
// distance to its row's largest over the temperature: integer sums do not depend on their order.
#pragma once

#include <math.h>

#include "kdt_internal.cuh"

namespace kdt {
namespace weights {

constexpr int kMaxVocab = 1 << 19;                  // sums of 2^44 weights then fit 63 bits
constexpr int kFrac = 44;

// 2^{k/128}, k = -64 .. 64, in units of 2^-45: hi * 2^45 + lo, hi a multiple of 2^-22 and 0 <= lo < 2^23.
struct Exp2Table {
    float hi[129], lo[129];
};
constexpr int kCopies = 16;                         // of the table in shared memory: a lane's reads meet no other's

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// round(2^44 e^{(l - m) / temperature}), l <= m finite (l may be -inf); tab is the lane's copy of the
// table. Roundings to integers are sums with 1.5 * 2^23 (the integer is then in the low bits): conversions
// run at a fraction of their rate. Without branches, so that several weights are under way at once.
__device__ __forceinline__ uint64_t weight(float l, float m, float c_hi, float c_lo, const float2 *tab) {
    constexpr float kMagic = 12582912.f;
    constexpr int kMagicBits = 0x4b400000;
    const float d = __fsub_rn(l, m);
    const float bb = __fsub_rn(d, l);
    const float dl = __fsub_rn(__fsub_rn(l, __fsub_rn(d, bb)), __fadd_rn(m, bb));   // l - m = d + dl exactly
    const float p = __fmul_rn(d, c_hi);
    const float pl = __fadd_rn(__fmaf_rn(d, c_hi, -p), __fmaf_rn(d, c_lo, __fmul_rn(dl, c_hi)));
    const float t = __fadd_rn(p, kMagic);
    const int n = __float_as_int(t) - kMagicBits;
    const float f = __fsub_rn(p, __fsub_rn(t, kMagic));                               // exact
    const float fh = __fadd_rn(f, pl), fl = __fsub_rn(pl, __fsub_rn(fh, f));         // |f| >= |pl| or both tiny
    const float u = __fmaf_rn(fh, 128.f, kMagic);
    const uint32_t k = min((uint32_t)(__float_as_int(u) - kMagicBits + 64), 128u);    // (beyond it: l = -inf)
    const float r = __fmaf_rn(__fsub_rn(u, kMagic), -0.0078125f, fh);                 // exact
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957768e-09f;   // ln 2 as a pair
    const float q = __fmul_rn(r, kLn2Hi);
    const float ql = __fadd_rn(__fmaf_rn(r, kLn2Hi, -q), __fmaf_rn(r, kLn2Lo, __fmul_rn(fl, kLn2Hi)));
    // e^q - 1 - q
    const float s = __fmul_rn(__fmul_rn(q, q), __fmaf_rn(q, __fmaf_rn(q, 0.0416666679f, 0.166666672f), 0.5f));
    const float2 th = tab[k * kCopies];
    const float a = __fmul_rn(th.x, q);
    const float b = __fadd_rn(__fmaf_rn(th.x, q, -a), __fmul_rn(th.x, __fadd_rn(__fmaf_rn(q, ql, ql), s)));
    // in units of 2^-45: hi + lo + a + b, a in two parts
    const float v = __fmaf_rn(a, 8388608.f, kMagic);
    const float ra = __fmaf_rn(__fsub_rn(v, kMagic), -1.1920928955078125e-07f, a);    // exact
    const int rest = __float2int_rn(__fmaf_rn(th.y, __fadd_rn(q, s), __fmul_rn(__fadd_rn(b, ra), 35184372088832.f)));
    const int hi = __float_as_int(__fmaf_rn(th.x, 4194304.f, 8388608.f)) - 0x4b000000;
    const int lo = __float_as_int(__fadd_rn(th.y, 8388608.f)) - 0x4b000000;
    const int64_t w = (int64_t)hi * (1 << 23) + ((int64_t)(__float_as_int(v) - kMagicBits) * (1 << 22) + (int64_t)(lo + rest));
    const int shift = 45 - kFrac - n;                // 1 .. 48
    return p >= -47.f ? (uint64_t)((w + ((int64_t)1 << ((shift - 1) & 63))) >> (shift & 63)) : 0;   // below -45: half a unit
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

inline Exp2Table make_table() {
    Exp2Table t;
    for (int k = 0; k < 129; ++k) {
        const uint64_t fix = (uint64_t)(exp2((k - 64) / 128.0) * 35184372088832.0 + 0.5);
        t.hi[k] = (float)(fix >> 23) * 2.384185791015625e-07f;                        // 2^-22
        t.lo[k] = (float)(fix & ((1 << 23) - 1));
    }
    return t;
}

}  // namespace weights
}  // namespace kdt
