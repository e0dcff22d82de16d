// K6: tree-verify attention over a paged bf16 latent cache. The simplest kernel that is right: a CTA a query row.
#include <math.h>

#include "kdt_internal.cuh"

namespace kdt {
namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) verify_paged_kernel(const PagedParams p) {
    __shared__ float q[kDqk], s[64];
    __shared__ int64_t row[64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t g = blockIdx.x;                                    // (b, i, h)
    const int b = (int)(g / p.rows_seq), i = (int)(g % p.rows_seq) / p.H;
    const int n = p.n_rows ? min(max(p.n_rows[b], 0), p.T) : p.T;
    if (i >= n) return;
    const int P = min(max(p.prefix_len[b], 0), p.max_kv - n);
    for (int d = tid; d < kDqk; d += kThreads)
        q[d] = d < kDc ? __bfloat162float(p.q_nope[g * p.q_nope_stride + d]) : __bfloat162float(p.q_pe[g * p.q_pe_stride + d - kDc]);
    float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
    for (int k0 = 0; k0 < P + n; k0 += 64) {
        __syncthreads();
        for (int k = warp; k < 64; k += 8) {
            const int j = k0 + k, t = j - P;
            bool see = j < P + n;
            if (see && t >= 0 && p.vis) see = (p.vis[((int64_t)b * p.T + i) * p.W + (t >> 5)] >> (t & 31)) & 1u;
            float x = 0.f;
            int64_t at = -1;
            if (see) {
                const int32_t page = p.table[b * p.table_stride + (j >> p.shift)];
                if (page >= 0 && page < p.n_pages) at = ((int64_t)page << p.shift) + (j & ((1 << p.shift) - 1));
                if (at < 0) {
                    if (lane == 0) record_error(p.err, (int32_t)min((int64_t)INT32_MAX, 1 + (int64_t)p.B * p.T + b));
                } else {
                    for (int d = lane; d < kDc; d += 32) x = fmaf(q[d], __bfloat162float(p.c_kv[at * kDc + d]), x);
                    for (int d = lane; d < kDr; d += 32) x = fmaf(q[kDc + d], __bfloat162float(p.k_pe[at * kDr + d]), x);
                }
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (lane == 0) {
                s[k] = see ? x * p.scale_log2 : -INFINITY;
                row[k] = see ? at : -2;
            }
        }
        __syncthreads();
        float top = m;
        for (int k = 0; k < 64; ++k) top = fmaxf(top, s[k]);
        const float a = m == top ? 1.f : exp2f(m - top);
        l *= a;
        o[0] *= a;
        o[1] *= a;
        m = top;
        for (int k = 0; k < 64; ++k) {
            const float w = s[k] == -INFINITY ? 0.f : exp2f(s[k] - m);
            if (row[k] == -2) continue;                               // (0 times what is not finite is NaN)
            l += w;
            if (row[k] < 0) continue;
            o[0] = fmaf(w, __bfloat162float(p.c_kv[row[k] * kDc + tid]), o[0]);
            o[1] = fmaf(w, __bfloat162float(p.c_kv[row[k] * kDc + tid + 256]), o[1]);
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int h = 0; h < 2; ++h) {
        const int64_t at = g * kDc + tid + 256 * h;
        if (p.out_bf16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(o[h] * inv);
        else static_cast<float *>(p.out)[at] = o[h] * inv;
    }
    if (tid == 0 && p.lse) p.lse[g] = l == 0.f ? -INFINITY : 0.6931471805599453f * (m + log2f(l));
}

}  // namespace

cudaError_t launch_verify_paged(const PagedParams &p, cudaStream_t s) {
    verify_paged_kernel<<<(unsigned)(p.B * (int64_t)p.rows_seq), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace kdt
