// One token a row under temperature, top-k, top-p and min-p, from given random numbers (kdt_sample).
// See include/kdt.h for the definition: weights w = round(2^44 e^{(l - max) / temperature}), and every
// filter keeps a prefix of the row's order (logit descending, index ascending).
#include <math.h>

#include "sample_weights.cuh"

namespace kdt {
namespace {

using namespace weights;

constexpr int kThreads = 1024, kWarps = 32;

struct SampleParams {
    const void *logits;
    int64_t row_stride;
    int R, V;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    double temperature_all, top_p_all, min_p_all;
    int top_k_all;
    int32_t *token, *err;
    float *logp;
};

__device__ __forceinline__ uint32_t order_key(float l) {           // ascending with the logit, one zero
    const uint32_t u = __float_as_uint(l + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }

struct Shared {
    float2 tab[129 * kCopies];
    uint64_t part[kWarps];
    uint64_t total;
    float m[kWarps];
    int found;
};

template <typename T> __device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ uint64_t block_sum(Shared &sh, uint64_t v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.part[warp] = v;
    __syncthreads();
    return warp_sum(sh.part[lane]);
}

// Exclusive prefix sum over the threads; `total` gets the sum.
__device__ uint64_t block_scan(Shared &sh, uint64_t v, uint64_t &total) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
    }
    __syncthreads();
    if (lane == 31) sh.part[warp] = incl;
    __syncthreads();
    uint64_t base = 0;
    total = 0;
    for (int k = 0; k < kWarps; ++k) {
        if (k < warp) base += sh.part[k];
        total += sh.part[k];
    }
    return base + incl - v;
}

// The simplest kernel that is right: a CTA a row, thresholds found by halving the range of keys.
template <typename E>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p, const __grid_constant__ Exp2Table table) {
    __shared__ Shared sh;
    const int r = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const E *x = static_cast<const E *>(p.logits) + (int64_t)r * p.row_stride;
    for (int k = tid; k < 129 * kCopies; k += kThreads) sh.tab[k] = make_float2(table.hi[k / kCopies], table.lo[k / kCopies]);
    const float2 *tab = sh.tab + lane % kCopies;
    const double temp = p.temperature ? (double)p.temperature[r] : p.temperature_all;
    const double top_p = p.top_p ? (double)p.top_p[r] : p.top_p_all;
    const double min_p = p.min_p ? (double)p.min_p[r] : p.min_p_all;
    int top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    if (top_k <= 0 || top_k > p.V) top_k = p.V;
    const bool greedy = temp == 0.0;
    if (greedy) top_k = 1;
    // the largest logit
    float m = -INFINITY;
    bool nan = false;
    for (int i = tid; i < p.V; i += kThreads) {
        const float l = as_f32(x[i]);
        nan |= l != l;
        m = fmaxf(m, l);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh.m[warp] = m;
    nan = __syncthreads_or(nan);
    m = sh.m[lane];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const bool settings = (greedy || (temp >= 1e-3 && temp <= 1e3)) && top_p == top_p && min_p == min_p;
    if (nan || !settings || !(m > -INFINITY && m < INFINITY)) {
        if (tid == 0) {
            p.token[r] = -1;
            if (p.logp) p.logp[r] = 0.f;
            record_error(p.err, r + 1);
        }
        return;
    }
    const double c = 1.4426950408889634074 / (greedy ? 1.0 : temp);
    const float c_hi = (float)c, c_lo = (float)(c - (double)c_hi);
    auto w_of = [&](float l) { return weight(l, m, c_hi, c_lo, tab); };
    // tokens, or their mass, of key x0 or more
    auto count = [&](uint32_t x0) {
        uint64_t n = 0;
        for (int i = tid; i < p.V; i += kThreads) n += order_key(as_f32(x[i])) >= x0;
        return block_sum(sh, n);
    };
    auto mass = [&](uint32_t x0) {
        uint64_t s = 0;
        for (int i = tid; i < p.V; i += kThreads) {
            const float l = as_f32(x[i]);
            if (order_key(l) >= x0) s += w_of(l);
        }
        return block_sum(sh, s);
    };
    // -- kept so far: keys above kx, and the first kr tokens (by index) of key kx
    uint32_t kx = order_key(m);
    uint64_t kr = 1;
    if (!greedy) {
        uint32_t lo = 0, hi = order_key(m);             // the largest key with top_k tokens at or above it
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            if (count(mid) >= (uint64_t)top_k) lo = mid;
            else hi = mid - 1;
        }
        kx = lo;
        kr = (uint64_t)top_k - (kx == 0xffffffffu ? 0 : count(kx + 1));
        if (top_p < 1.0) {
            const uint64_t above = mass(kx + 1);
            const double goal = fmax(top_p, 0.0) * (double)(above + kr * w_of(key_logit(kx)));
            if (goal <= (double)above || kx == order_key(m)) {
                uint32_t a = kx, e = order_key(m);      // the largest key with the goal's mass at or above it
                while (a < e) {
                    const uint32_t mid = a + (e - a + 1) / 2;
                    if ((double)mass(mid) >= goal) a = mid;
                    else e = mid - 1;
                }
                const uint64_t wx = w_of(key_logit(a)), up = mass(a + 1);
                const uint64_t most = a == kx ? kr : (uint64_t)p.V;
                uint64_t n = 1;
                if (wx > 0 && goal > (double)up) {
                    n = (uint64_t)fmax((goal - (double)up) / (double)wx, 1.0);
                    while (n > 1 && (double)(up + (n - 1) * wx) >= goal) --n;
                    while ((double)(up + n * wx) < goal && n < most) ++n;
                }
                kx = a;
                kr = n < most ? n : most;
            } else {
                const uint64_t wx = w_of(key_logit(kx));
                uint64_t n = kr;
                while (n > 1 && (double)(above + (n - 1) * wx) >= goal) --n;
                kr = n;
            }
        }
    }
    const double least = fmin(fmax(min_p, 0.0), 1.0) * 17592186044416.0;
    // -- the draw, tokens in index order
    const int per = (p.V + kThreads - 1) / kThreads, i0 = min(tid * per, p.V), i1 = min(i0 + per, p.V);
    uint64_t equal = 0, all;
    for (int i = i0; i < i1; ++i) equal += order_key(as_f32(x[i])) == kx;
    const uint64_t equal0 = block_scan(sh, equal, all);
    auto kept = [&](int i, uint64_t &e) -> uint64_t {
        const float l = as_f32(x[i]);
        const uint32_t k = order_key(l);
        const bool in = k > kx || (k == kx && e < kr);
        e += k == kx;
        const uint64_t w = in ? w_of(l) : 0;
        return (double)w >= least ? w : 0;
    };
    uint64_t e = equal0, mine = 0, z = 0;
    for (int i = i0; i < i1; ++i) {
        mine += kept(i, e);
        z += w_of(as_f32(x[i]));
    }
    z = block_sum(sh, z);
    const uint64_t before = block_scan(sh, mine, all);
    const double td = (double)p.u[r] * (double)all;
    uint64_t t = td > 0.0 ? (uint64_t)td : 0;
    if (t >= all) t = all - 1;
    if (t >= before && t < before + mine) {
        uint64_t acc = before;
        e = equal0;
        int i = i0;
        for (; i < i1; ++i) {
            acc += kept(i, e);
            if (acc > t) break;
        }
        p.token[r] = i;
        if (p.logp)
            p.logp[r] = greedy ? 0.f : (float)(((double)as_f32(x[i]) - (double)m) / temp - log((double)z / 17592186044416.0));
    }
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace kdt

using namespace kdt;

extern "C" kdt_status kdt_sample(const kdt_sample_args *a, cudaStream_t stream) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->R < 0 || a->V < 1 || a->V > kMaxVocab) return KDT_ERR_BAD_SHAPE;
    if (a->dtype != KDT_F32 && a->dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    const int esz = a->dtype == KDT_F32 ? 4 : 2;
    const int64_t stride = a->row_stride ? a->row_stride : a->V;
    if (stride < a->V) return KDT_ERR_BAD_SHAPE;
    if (!a->temperature && !(a->temperature_all == 0.0 || (a->temperature_all >= 1e-3 && a->temperature_all <= 1e3)))
        return KDT_ERR_BAD_SHAPE;
    if ((!a->top_p && a->top_p_all != a->top_p_all) || (!a->min_p && a->min_p_all != a->min_p_all)) return KDT_ERR_BAD_SHAPE;
    if (a->R == 0) return a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t), stream) != cudaSuccess ? KDT_ERR_CUDA : KDT_OK;
    if (!a->logits || !a->u || !a->token) return KDT_ERR_NULL_ARG;
    if (!aligned(a->logits, esz)) return KDT_ERR_BAD_SHAPE;
    for (const void *q : {(const void *)a->u, (const void *)a->temperature, (const void *)a->top_k, (const void *)a->top_p,
                          (const void *)a->min_p, (const void *)a->token, (const void *)a->logp, (const void *)a->err})
        if (!aligned(q, 4)) return KDT_ERR_BAD_SHAPE;
    const kdt_status st = check_on_current_device(
        {a->logits, a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->token, a->logp, a->err});
    if (st != KDT_OK) return st;
    if (a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t), stream) != cudaSuccess) return KDT_ERR_CUDA;
    const SampleParams p = {a->logits, stride, a->R, a->V, a->u, a->temperature, a->top_p, a->min_p, a->top_k, a->temperature_all,
                            a->top_p_all, a->min_p_all, a->top_k_all, a->token, a->err, a->logp};
    static const Exp2Table table = make_table();
    if (a->dtype == KDT_F32)
        sample_kernel<float><<<a->R, kThreads, 0, stream>>>(p, table);
    else
        sample_kernel<__nv_bfloat16><<<a->R, kThreads, 0, stream>>>(p, table);
    return cudaGetLastError() == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}
