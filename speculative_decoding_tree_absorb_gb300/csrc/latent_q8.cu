// The 8-bit latent cache: rows quantised as they are written (norm of the latent, rotation
// of the rope key and quantisation in one pass) and rows read back. See include/kdt.h for
// the format: 512 e4m3 codes a row, one power-of-two scale byte for each 32 of them, 64
// bf16 rope values.
//
// Both kernels only stream: a warp takes whole rows, every load and store instruction of a
// warp covers one contiguous stretch (16 bytes a lane where the row holds that much), and
// the grid is sized so that a resident warp takes several rows. Reading keeps the next row's
// loads in flight (40 registers, 40 warps an SM); writing has more to hold, and more warps
// were worth more than a row ahead in each (16 warps of 92 registers: 33 us, 32 of 64: 22 us).
// Measured: 12 prompts of up to 4095 rows in float32 written in 22 us (79 MB: 3.6 TB/s; issue
// slots 58%), 8 sequences of 8256 rows read in 20-25 us (119 MB: 4.8-5.9 TB/s; issue slots
// 67%). Short calls take the 7-9 us of one launch and one row's chain of loads.
#include <cmath>

#include "latent_rows.cuh"
#include "q8.cuh"

namespace kdt {
namespace {

using namespace rows;

constexpr int kWarps = 8;                           // warps a CTA
constexpr int kWriters = 4, kReaders = 5;           // CTAs an SM when there are rows enough

struct WriteParams {
    const void *c, *k, *gamma;
    int64_t c_stride, k_stride;
    const int32_t *pos, *prefix_len, *n_rows;
    uint8_t *c_q8, *c_scale;
    __nv_bfloat16 *k_pe;
    int64_t L;
    int B, T;
    float eps;
};

// One warp a row. y = x r gamma in float32 (r from the row's sum of squares by shuffles); a
// group of 32 is 32 / kPer neighbouring lanes of one piece, its largest magnitude a few
// shuffles (taken over the bit patterns, so infinities and NaN come out on top).
template <typename E>
__global__ void __launch_bounds__(32 * kWarps, kWriters) latent_write_kernel(const WriteParams p,
                                                                   const __grid_constant__ TurnFreqs fr) {
    using R = Row<E>;
    constexpr int kLanes = KDT_Q8_GROUP / R::kPer;        // lanes that share a group
    const int lane = threadIdx.x & 31;
    const uint32_t rows = (uint32_t)p.B * p.T, step = gridDim.x * kWarps;      // (below 2^31: 32-bit divisions)
    const uint64_t freq = fr.f[lane];
    for (uint32_t n = blockIdx.x * kWarps + (threadIdx.x >> 5); n < rows; n += step) {
        const int b = (int)(n / (uint32_t)p.T), i = (int)(n - (uint32_t)b * p.T);
        if (p.n_rows && i >= p.n_rows[b]) continue;
        R c;
        c.template load<true>(static_cast<const E *>(p.c) + (int64_t)n * p.c_stride, lane);
        const E *k = static_cast<const E *>(p.k) + (int64_t)n * p.k_stride;
        const E ka = k[lane], kb = k[lane + kHalf];
        const int32_t pos = p.pos ? p.pos[n] : 0;
        const int64_t row = (int64_t)p.prefix_len[b] + i;
        if (row < 0 || row >= p.L) continue;
        const int64_t dst = (int64_t)b * p.L + row;
        float y[16];
        c.get(y);
        if (p.gamma) rms_norm(y, static_cast<const E *>(p.gamma), p.eps, lane);
        uint8_t *codes = p.c_q8 + dst * kDc;
        uint8_t *scales = p.c_scale + dst * (kDc / KDT_Q8_GROUP);
#pragma unroll
        for (int q = 0; q < R::kPieces; ++q) {
            uint32_t top = 0;
#pragma unroll
            for (int t = 0; t < R::kPer; ++t)
                top = max(top, __float_as_uint(y[R::kPer * q + t]) & 0x7fffffffu);
#pragma unroll
            for (int off = kLanes / 2; off >= 1; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
            const int byte = q8::scale_byte(top);
            const float inv = q8::inverse_scale(byte);     // 0 for a group that reads as NaN
            uint32_t w[R::kPer / 4];
#pragma unroll
            for (int t = 0; t < R::kPer / 4; ++t) {
                const float *z = &y[R::kPer * q + 4 * t];
                w[t] = byte == q8::kNaN ? 0u : q8::encode4(z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv);
            }
            if constexpr (R::kPer == 4)
                reinterpret_cast<uint32_t *>(codes)[32 * q + lane] = w[0];
            else
                reinterpret_cast<uint2 *>(codes)[32 * q + lane] = make_uint2(w[0], w[1]);
            if (lane % kLanes == 0) scales[q * (32 / kLanes) + lane / kLanes] = (uint8_t)byte;
        }
        float k0 = to_f32(ka), k1 = to_f32(kb);
        if (p.pos) rotate(k0, k1, pos, freq);
        __nv_bfloat16 *kd = p.k_pe + dst * kDr;
        kd[lane] = __float2bfloat16_rn(k0);
        kd[lane + kHalf] = __float2bfloat16_rn(k1);
    }
}

struct ReadParams {
    const uint8_t *c_q8, *c_scale;
    const __nv_bfloat16 *k_pe;
    int64_t L;
    int B, R;
    const int32_t *start, *n_rows;
    void *c, *k;
};

// One warp a row: piece q of a lane is kPer consecutive codes (4 for float32, 8 for bf16),
// 16 bytes of output. Every value is a bf16 number, so both types are exact.
template <typename E>
__global__ void __launch_bounds__(32 * kWarps) latent_read_kernel(const ReadParams p) {
    constexpr int kPer = 16 / sizeof(E), kPieces = 16 / kPer;
    const int lane = threadIdx.x & 31;
    const uint32_t rows = (uint32_t)p.B * p.R, step = gridDim.x * kWarps;      // (below 2^31: 32-bit divisions)
    struct Next {
        uint32_t w[4];
        uint8_t s[kPieces];
        uint32_t k;
        bool live;
    };
    auto fetch = [&](uint32_t n, Next &x) {
        x.live = false;
        if (n >= rows) return;
        const int b = (int)(n / (uint32_t)p.R), i = (int)(n - (uint32_t)b * p.R);
        if (p.n_rows && i >= p.n_rows[b]) return;
        x.live = true;
        const int64_t row = (int64_t)(p.start ? p.start[b] : 0) + i;
        if (row < 0 || row >= p.L) {                          // reads as zeros
#pragma unroll
            for (int q = 0; q < 4; ++q) x.w[q] = 0u;
#pragma unroll
            for (int q = 0; q < kPieces; ++q) x.s[q] = 127;
            x.k = 0u;
            return;
        }
        const int64_t src = (int64_t)b * p.L + row;
        if (p.c) {
            const uint8_t *codes = p.c_q8 + src * kDc, *scales = p.c_scale + src * (kDc / KDT_Q8_GROUP);
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                if constexpr (kPer == 4) {
                    x.w[q] = __ldcs(reinterpret_cast<const uint32_t *>(codes) + 32 * q + lane);
                } else {
                    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(codes) + 32 * q + lane);
                    x.w[2 * q] = v.x;
                    x.w[2 * q + 1] = v.y;
                }
                x.s[q] = scales[(q * 32 + lane) * kPer / KDT_Q8_GROUP];
            }
        }
        if (p.k) x.k = __ldcs(reinterpret_cast<const uint32_t *>(p.k_pe + src * kDr) + lane);
    };
    uint32_t n = blockIdx.x * kWarps + (threadIdx.x >> 5);
    Next cur, nxt;
    fetch(n, cur);
    for (; n < rows; n += step) {
        fetch(n + step, nxt);
        if (cur.live) {
            if (p.c) {
                uint4 *dst = reinterpret_cast<uint4 *>(static_cast<E *>(p.c) + (int64_t)n * kDc);
#pragma unroll
                for (int q = 0; q < kPieces; ++q) {
                    const float s = q8::scale_value(cur.s[q]);
                    uint32_t o[4];
#pragma unroll
                    for (int t = 0; t < kPer / 4; ++t) {
                        float f[4];
                        q8::decode4(cur.w[q * (kPer / 4) + t], f);
                        if constexpr (kPer == 4) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[e] = __float_as_uint(f[e] * s);
                        } else {
                            o[2 * t] = q8::pack_bf16(f[0] * s, f[1] * s);
                            o[2 * t + 1] = q8::pack_bf16(f[2] * s, f[3] * s);
                        }
                    }
                    __stcs(dst + 32 * q + lane, make_uint4(o[0], o[1], o[2], o[3]));
                }
            }
            if (p.k) {
                if constexpr (sizeof(E) == 2)
                    reinterpret_cast<uint32_t *>(p.k)[(int64_t)n * (kDr / 2) + lane] = cur.k;
                else
                    reinterpret_cast<float2 *>(p.k)[(int64_t)n * (kDr / 2) + lane] =
                        make_float2(__uint_as_float(cur.k << 16), __uint_as_float(cur.k & 0xffff0000u));
            }
        }
        cur = nxt;
    }
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs for `rows` rows: a warp a row until the device is full (`full` CTAs an SM), then
// resident warps take several rows each.
int grid_for(int64_t rows, int full) {
    const int64_t ctas = (rows + kWarps - 1) / kWarps, most = (int64_t)sm_count() * full;
    return (int)(ctas < most ? ctas : most);
}

}  // namespace
}  // namespace kdt

using namespace kdt;

extern "C" {

kdt_status kdt_latent_write_q8(const kdt_latent_write_args *a, cudaStream_t stream) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->B < 0 || a->T < 1 || (int64_t)a->B * a->T > INT32_MAX) return KDT_ERR_BAD_SHAPE;
    if (a->D_c != kDc || a->D_r != kDr) return KDT_ERR_UNSUPPORTED;
    if (a->dtype != KDT_F32 && a->dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    const int esz = a->dtype == KDT_F32 ? 4 : 2;
    const int64_t cs = a->c_row_stride ? a->c_row_stride : kDc, ks = a->k_row_stride ? a->k_row_stride : kDr;
    if (cs < kDc || (cs * esz) % 16 || ks < kDr || a->kv_row_stride < 1) return KDT_ERR_BAD_SHAPE;
    if (a->gamma && !(a->eps >= 0.f && a->eps < INFINITY)) return KDT_ERR_BAD_SHAPE;
    if (a->pos && !(a->base > 0.0 && a->base <= 1e300)) return KDT_ERR_BAD_SHAPE;
    if (a->B == 0) return KDT_OK;
    if (!a->c || !a->k || !a->prefix_len || !a->c_q8 || !a->c_scale || !a->k_pe) return KDT_ERR_NULL_ARG;
    if (!aligned(a->c, 16) || !aligned(a->gamma, 16) || !aligned(a->k, esz) || !aligned(a->c_q8, 16) ||
        !aligned(a->c_scale, 16) || !aligned(a->k_pe, 16) || !aligned(a->pos, 4) || !aligned(a->prefix_len, 4) ||
        !aligned(a->n_rows, 4))
        return KDT_ERR_BAD_SHAPE;
    const kdt_status st = check_on_current_device(
        {a->c, a->k, a->gamma, a->pos, a->prefix_len, a->n_rows, a->c_q8, a->c_scale, a->k_pe});
    if (st != KDT_OK) return st;
    const TurnFreqs fr = a->pos ? turn_freqs(a->base) : TurnFreqs{};
    const WriteParams p = {a->c,    a->k,       a->gamma, cs, ks, a->pos, a->prefix_len, a->n_rows,
                           a->c_q8, a->c_scale, static_cast<__nv_bfloat16 *>(a->k_pe), a->kv_row_stride,
                           a->B,    a->T,       a->eps};
    const int grid = grid_for((int64_t)a->B * a->T, kWriters);
    if (a->dtype == KDT_F32)
        latent_write_kernel<float><<<grid, 32 * kWarps, 0, stream>>>(p, fr);
    else
        latent_write_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, stream>>>(p, fr);
    return cudaGetLastError() == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

kdt_status kdt_latent_read_q8(const uint8_t *c_q8, const uint8_t *c_scale, const void *k_pe, int64_t kv_row_stride,
                              int B, int R, const int32_t *start, const int32_t *n_rows, kdt_dtype dtype, void *c,
                              void *k, cudaStream_t stream) {
    if (B < 0 || R < 0 || (int64_t)B * R > INT32_MAX || kv_row_stride < 1) return KDT_ERR_BAD_SHAPE;
    if (dtype != KDT_F32 && dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    if (B == 0 || R == 0) return KDT_OK;
    if (!c_q8 || !c_scale || !k_pe || (!c && !k)) return KDT_ERR_NULL_ARG;
    if (!aligned(c_q8, 16) || !aligned(c_scale, 16) || !aligned(k_pe, 16) || !aligned(c, 16) || !aligned(k, 16) ||
        !aligned(start, 4) || !aligned(n_rows, 4))
        return KDT_ERR_BAD_SHAPE;
    const kdt_status st = check_on_current_device({c_q8, c_scale, k_pe, start, n_rows, c, k});
    if (st != KDT_OK) return st;
    const ReadParams p = {c_q8, c_scale, static_cast<const __nv_bfloat16 *>(k_pe), kv_row_stride, B, R, start, n_rows,
                          c, k};
    const int grid = grid_for((int64_t)B * R, kReaders);
    if (dtype == KDT_F32)
        latent_read_kernel<float><<<grid, 32 * kWarps, 0, stream>>>(p);
    else
        latent_read_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
