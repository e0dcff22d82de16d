// One token a row under temperature, top-k, top-p and min-p, from given random numbers (kdt_sample).
// See include/kdt.h for the definition: weights w = round(2^44 e^{(l - max) / temperature}), and every
// filter keeps a prefix of the row's order (logit descending, index ascending), so that what is kept is
// told by one key and a number: all logits above the key, and the first `number` tokens equal to it.
//
//  * A cluster of CTAs takes a row, each a contiguous slice, kept in shared memory where it fits.
//  * Bins in the row's order, by the upper 16 bits of a logit's ordered bits (its bf16 value), counted in
//    shared memory: 4096 of them from the maximum down, the values within 2^-10 of zero in one. In bf16 a
//    bin is one value, so that the counts and one weight a bin give every sum exactly: top-k's and top-p's
//    borders come from one scan. A float32 bin's tokens differ: where top-p needs masses their weights are
//    summed (as two 32-bit halves), and the tokens of the bin that a border falls into are gathered in the
//    first CTA, which halves the range of their keys.
//  * The draw: every warp sums what is kept of its part of the slice (weights from the bins' table in
//    bf16), the sums are scanned over warps and CTAs, and the part that holds u times the whole is taken
//    apart again. All sums are integers, the log-probability's too: neither the cluster's size nor the order of the
//    adds shows.
//  * A bin of several values with more tokens than the list holds (2048) is searched by the first CTA alone: it
//    halves the range of the keys, up to 32 passes over the whole row in global memory. This is the slow form, and
//    two kinds of ordinary rows reach it. In float32 a bin is as wide as a bf16 value's last bit, so the bin of a border may
//    hold thousands of tokens where the logits lie far from zero: 160000 of mean 20 and deviation 2 under top-p 0.95
//    take 2.3 ms (64 rows 2.5), of mean 0 0.05 (64 rows 0.11). And -inf lies in the last bin, in bf16 too, where a
//    border falls if top-k asks for more tokens than a mask has left: 30 of 160000 under top-k 50 take 0.36 - 0.38
//    ms (64 rows 0.39 - 0.42), under top-k 20 0.025 - 0.041.
//  * Measured: one row of 32000 tokens in float32 under all filters 29 us, a chain of passes over 4000 tokens a
//    CTA and of a dozen barriers of the cluster. 64 rows of 160000 in bf16 with settings of their own 47 us: two
//    CTAs a row, 80000 tokens each, of its 78 k cycles 11 for the maximum (the row comes from DRAM, 20 MB), 18
//    for the counts (7 cycles for a warp's 32 adds, 20 instructions a token), 12 for bins and borders, 28 for the
//    masses where nothing is filtered (a 64-bit look-up a token), 5 where 60 tokens are kept. The same rows in
//    float32 with settings of their own 111 us; 66 unfiltered, 109 under top-p (a weight a token), 43 under top-k.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "sample_weights.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace weights;

constexpr int kThreads = 1024, kWarps = 32;
constexpr int kBins = 4096;
constexpr int kMaxCluster = 8;
constexpr int kList = 2048, kHold = kList / kThreads; // tokens of one bin that a border falls into
constexpr uint32_t kShort = 256;                    // as many are ranked, a thread each
constexpr size_t kMostSmem = 200 * 1024;            // beside Shared
constexpr uint32_t kPosTiny = 0xba80u, kNegTiny = 0x457fu;     // upper ordered bits of 2^-10 and of -2^-10

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
    int slice;                                      // tokens a CTA takes (a multiple of 16)
    int vec;                                        // rows start on 16-byte boundaries
    int cache;                                      // a slice fits shared memory
};

__device__ __forceinline__ uint32_t order_key(float l) {           // ascending with the logit, one zero
    const uint32_t u = __float_as_uint(l + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t bits_key(float l) {            // the same, but zeros of either sign differ
    const uint32_t u = __float_as_uint(l);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k); }

// Bins in the row's order, the largest logit's first.
struct Bins {
    uint32_t top, low;                              // upper key bits of the maximum; of the first negative bin
    int pos, neg;                                   // bins before the one around zero; and up to the negative ones
    int zero, under;                                // the one around zero, or -1; a negative bin and its upper bits
    __device__ __forceinline__ void set(uint32_t max_key) {
        top = max_key >> 16;
        pos = top >= kPosTiny ? (int)(top - kPosTiny) + 1 : 0;
        neg = pos + (top > kNegTiny ? 1 : 0);
        low = min(top, kNegTiny);
        zero = neg > pos ? pos : -1;
        under = neg + (int)low;
    }
    // top - h for positive ones, `pos` around zero (there under - h <= pos <= top - h), under - h for negative ones
    __device__ __forceinline__ int of(uint32_t key) const {
        const int h = (int)(key >> 16);
        return min(max(min((int)top - h, pos), under - h), kBins - 1);
    }
    // whether a bin holds one bf16 value only, and that value
    __device__ __forceinline__ bool single(int b) const { return b < kBins - 1 && b != zero; }
    __device__ __forceinline__ float value(int b) const {
        const uint32_t h = b < pos ? top - (uint32_t)b : low - (uint32_t)(b - neg);
        return key_logit(h & 0x8000u ? h << 16 : (h << 16) | 0xffffu);
    }
};

struct Border {                                     // what a filter keeps: keys above `key`, and `ties` of it
    uint32_t key;
    uint32_t ties;
};

struct Shared {
    float2 tab[129 * kCopies];
    uint64_t part[kWarps];
    uint32_t part2[kWarps];
    uint64_t total;
    uint32_t total2;
    float wm[kWarps];
    // written by other CTAs of the cluster
    float m[kMaxCluster];
    uint64_t sum[kMaxCluster];                      // kept above the border, and ties, by CTA
    uint32_t ties[kMaxCluster];
    uint64_t z[kMaxCluster];
    Border border[2];                               // top-k's, top-p's
    uint64_t above[2];                              // mass that the border keeps
    uint64_t mass_of[kMaxCluster];                  // of the CTAs' shares of the bins
    uint32_t count_of[kMaxCluster];
    int bin[2];                                     // where a border falls
    uint32_t before[2], in_bin[2];                  // tokens in front of it, and in it
    uint64_t mass_before[2];
    uint32_t list_n[2];
    // of this CTA
    int found;
    uint64_t at;
    uint32_t ties_at;
    // settings and thresholds, found by one thread: an FP64 operation of all warps takes 500 clocks
    float c_hi, c_lo;
    int good;
    uint64_t least, goal, t;
};

template <typename T> __device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ uint64_t block_sum(Shared &sh, uint64_t v) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.part[warp] = v;
    __syncthreads();
    return warp_sum(sh.part[lane]);
}

// Exclusive prefix sums of (a, c) over the threads; `ta`, `tc` get the sums.
__device__ __forceinline__ void block_scan(Shared &sh, uint64_t a, uint32_t c, uint64_t &ea, uint32_t &ec, uint64_t &ta, uint32_t &tc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t ia = a;
    uint32_t ic = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, ia, off);
        const uint32_t y = __shfl_up_sync(0xffffffffu, ic, off);
        if (lane >= off) {
            ia += x;
            ic += y;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.part[warp] = ia;
        sh.part2[warp] = ic;
    }
    __syncthreads();
    if (warp == 0) {                                           // (the warps' sums by one warp: by each of 32 it costs more)
        const uint64_t pa = sh.part[lane];
        const uint32_t pc = sh.part2[lane];
        uint64_t sa = pa;
        uint32_t sc = pc;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t x = __shfl_up_sync(0xffffffffu, sa, off);
            const uint32_t y = __shfl_up_sync(0xffffffffu, sc, off);
            if (lane >= off) {
                sa += x;
                sc += y;
            }
        }
        sh.part[lane] = sa - pa;
        sh.part2[lane] = sc - pc;
        if (lane == 31) {
            sh.total = sa;
            sh.total2 = sc;
        }
    }
    __syncthreads();
    ea = sh.part[warp] + ia - a;
    ec = sh.part2[warp] + ic - c;
    ta = sh.total;
    tc = sh.total2;
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// w added to a 64-bit sum held as two words: the low word's old value tells the carry.
__device__ __forceinline__ void add_to(uint32_t *lo, uint32_t *hi, uint64_t w) {
    const uint32_t l = (uint32_t)w, old = atomicAdd(lo, l);
    const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
    if (h) atomicAdd(hi, h);
}
// The same in another CTA of the cluster, by shared::cluster addresses.
__device__ __forceinline__ uint32_t add_cluster(uint32_t addr, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void add_to_cluster(uint32_t lo, uint32_t hi, uint64_t w) {
    const uint32_t l = (uint32_t)w, old = add_cluster(lo, l);
    const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
    if (h) add_cluster(hi, h);
}

// Dynamic shared memory. The slice's bins are counted here (their weights' sums where a bin has several values), then
// added up in the CTA whose share of the bins they fall into.
struct Dyn {
    uint32_t count[kBins], lo[kBins], hi[kBins];    // of the slice
    uint32_t all_count[kBins], all_lo[kBins], all_hi[kBins];       // of the row: this CTA's share
    uint64_t w[kBins];                              // bf16: a bin's weight
    uint64_t list_w[kShort];                        // of a short list's tokens
};

template <typename E>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleParams p, const __grid_constant__ Exp2Table table) {
    extern __shared__ __align__(16) unsigned char dyn_raw[];
    __shared__ Shared sh;
    Dyn &dy = *reinterpret_cast<Dyn *>(dyn_raw);
    constexpr bool kSingle = sizeof(E) == 2;
    uint64_t *list = reinterpret_cast<uint64_t *>(dyn_raw + sizeof(Dyn));
    E *row = reinterpret_cast<E *>(dyn_raw + sizeof(Dyn) + 2 * kList * sizeof(uint64_t));
    uint32_t rank, size;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int r = blockIdx.x / size, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int v0 = min((int)rank * p.slice, p.V), n = min(p.slice, p.V - v0);
    const E *src = static_cast<const E *>(p.logits) + (int64_t)r * p.row_stride + v0;
    for (int k = tid; k < 129 * kCopies; k += kThreads) sh.tab[k] = make_float2(table.hi[k / kCopies], table.lo[k / kCopies]);
    for (int k = tid; k < 6 * kBins / 4; k += kThreads) reinterpret_cast<uint4 *>(dyn_raw)[k] = make_uint4(0u, 0u, 0u, 0u);
    if (tid < 2) sh.list_n[tid] = 0;
    const float2 *tab = sh.tab + lane % kCopies;
    const double unit = 17592186044416.0;                      // 2^44
    int top_k = p.top_k ? p.top_k[r] : p.top_k_all;
    const bool greedy = p.temperature ? p.temperature[r] == 0.f : p.temperature_all == 0.0;
    if (greedy) top_k = 1;
    const bool by_count = top_k > 0 && top_k < p.V, by_mass = !greedy && (p.top_p ? p.top_p[r] < 1.f : p.top_p_all < 1.0);
    if (tid == kThreads - 1) {
        const double temp = p.temperature ? (double)p.temperature[r] : p.temperature_all;
        const double top_p = p.top_p ? (double)p.top_p[r] : p.top_p_all;
        const double min_p = p.min_p ? (double)p.min_p[r] : p.min_p_all;
        const double c = 1.4426950408889634074 / (greedy ? 1.0 : temp);
        sh.c_hi = (float)c;
        sh.c_lo = (float)(c - (double)sh.c_hi);
        sh.least = (uint64_t)ceil(fmin(fmax(min_p, 0.0), 1.0) * unit);
        sh.good = (greedy || (temp >= 1e-3 && temp <= 1e3)) && top_p == top_p && min_p == min_p;
    }

    // -- the largest logit (NaN wins), the slice to shared memory on the way
    constexpr int kPer = 16 / (int)sizeof(E);
    const int nv = n / kPer;
    float m = -INFINITY;
    bool nan = false;
    auto see = [&](float x) {
        nan |= x != x;
        m = fmaxf(m, x);
    };
    if (p.vec) {
#pragma unroll 4
        for (int i = tid; i < nv; i += kThreads) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            if (p.cache) reinterpret_cast<uint4 *>(row)[i] = v;
            const E *e = reinterpret_cast<const E *>(&v);
#pragma unroll
            for (int k = 0; k < kPer; ++k) see(as_f32(e[k]));
        }
        for (int i = nv * kPer + tid; i < n; i += kThreads) {
            if (p.cache) row[i] = src[i];
            see(as_f32(src[i]));
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < n; i += kThreads) {
            const E v = src[i];
            if (p.cache) row[i] = v;
            see(as_f32(v));
        }
    }
    auto top = [](float a, float c) { return a != a ? a : (c != c ? c : fmaxf(a, c)); };
    if (nan) m = __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) sh.wm[warp] = m;
    tc::cluster_sync();        // every CTA runs before another writes to its shared memory
    if (warp == 0) {
        m = sh.wm[lane];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane < (int)size) tc::st_cluster_f32(tc::map_to_rank(&sh.m[rank], (uint32_t)lane), m);
    }
    tc::cluster_sync();
    m = lane < (int)size ? sh.m[lane] : -INFINITY;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (!sh.good || !(m > -INFINITY && m < INFINITY)) {      // (the cluster as one)
        if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.logp) p.logp[r] = 0.f;
            record_error(p.err, r + 1);
        }
        return;
    }
    const E *data = p.cache ? row : src;
    const float c_hi = sh.c_hi, c_lo = sh.c_lo;
    const uint64_t least = sh.least;
    auto w_of = [&](float l) { return weight(l, m, c_hi, c_lo, tab); };
    Bins bins;
    bins.set(order_key(m));
    // every token of the slice, 16 bytes at a time where they can be had so. The loop is unrolled: `f` is short,
    // and says of which tokens `rest` has to see (32 copies of a weight's code do not fit the instruction cache:
    // 75 instructions' time a token).
    auto each = [&](auto &&f, auto &&rest) {
        if (p.cache || p.vec) {
            for (int i0 = tid; i0 < nv; i0 += 4 * kThreads) {
                uint32_t more = 0;
                uint4 v[4];                                    // (their latency is what a pass takes)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (i0 + u * kThreads < nv) v[u] = reinterpret_cast<const uint4 *>(data)[i0 + u * kThreads];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i0 + u * kThreads >= nv) break;
                    const E *e = reinterpret_cast<const E *>(&v[u]);
#pragma unroll
                    for (int k = 0; k < kPer; ++k) more |= (f(as_f32(e[k]), (i0 + u * kThreads) * kPer + k) ? 1u : 0u) << (u * kPer + k);
                }
                while (more) {
                    const int k = __ffs(more) - 1;
                    more &= more - 1;
                    rest(as_f32(data[(i0 + k / kPer * kThreads) * kPer + k % kPer]));
                }
            }
#pragma unroll 1
            for (int i = nv * kPer + tid; i < n; i += kThreads)
                if (f(as_f32(data[i]), i)) rest(as_f32(data[i]));
        } else
#pragma unroll 1
            for (int i = tid; i < n; i += kThreads)
                if (f(as_f32(data[i]), i)) rest(as_f32(data[i]));
    };
    auto none = [](float) {};
    auto each_weighed = [&](auto &&f) {                        // one by one, for what is long
#pragma unroll 1
        for (int i = tid; i < n; i += kThreads) f(as_f32(data[i]));
    };

    // -- tokens a bin; in float32 also the sum of all weights in units of 2^-42, good enough for a log-probability. A
    // token's weight is rounded to them by itself, so that this sum has no order either: a multiple of 2^-20 and
    // the rest, both the low bits of a sum with 1.5 * 2^23 of their units (|rest| <= 2^21 of them, and a thread has
    // 512 tokens and a tail's at most).
    uint64_t z = 0;
    int32_t z_hi = 0, z_lo = 0;
    static_assert((kMaxVocab / kThreads + 8) * ((int64_t)1 << 21) < INT32_MAX, "a thread's sums");
    const bool sums = !kSingle && p.logp && !greedy, binned = !greedy && (kSingle || by_count || by_mass);
    auto add_z = [&](float l) {
        constexpr float kHi = 12.f, kLo = 2.86102294921875e-06f;             // 1.5 * 2^23 of 2^-20, of 2^-42
        const float d = __fsub_rn(l, m), y = __fmul_rn(d, c_hi), e2 = ex2(y);
        const float e = y < -60.f ? 0.f : __fmaf_rn(e2, __fmul_rn(0.6931471805599453f, __fmaf_rn(d, c_lo, __fmaf_rn(d, c_hi, -y))), e2);
        const float h = __fadd_rn(e, kHi), rest = __fsub_rn(e, __fsub_rn(h, kHi));           // exact
        z_hi += __float_as_int(h) - 0x41400000;
        z_lo += __float_as_int(__fadd_rn(rest, kLo)) - 0x36400000;
    };
    if (sums && !binned)
        each([&](float l, int) {
            add_z(l);
            return false;
        }, none);
    Border border = {0u, (uint32_t)p.V};                       // everything
    if (greedy) border = {order_key(m), 1u};
    const bool table_w = kSingle && !greedy;                   // bins have weights
    if (binned) {
        // (the last bin has what lies far below, a mask's -inf too: counted apart, as a word that all add to is slow)
        const bool weighs = kSingle || (by_mass && !by_count);
        uint32_t n_last = 0;
        uint64_t w_last = 0, w_zero = 0;
        if (!weighs || kSingle)
            each([&](float l, int) {
                if (sums) add_z(l);
                const int b = bins.of(bits_key(l));
                if (b == kBins - 1) {
                    ++n_last;
                    return weighs && l > -INFINITY;
                }
                atomicAdd(&dy.count[b], 1u);
                return kSingle && b == bins.zero;
            }, [&](float l) {
                const int b = bins.of(bits_key(l));
                if (b == kBins - 1 && l > -INFINITY) w_last += w_of(l);
                if (b == bins.zero) w_zero += w_of(l);
            });
        else
            each_weighed([&](float l) {
                if (sums) add_z(l);
                const int b = bins.of(bits_key(l));
                if (b == kBins - 1) {
                    ++n_last;
                    if (l > -INFINITY) w_last += w_of(l);
                } else {
                    atomicAdd(&dy.count[b], 1u);
                    add_to(&dy.lo[b], &dy.hi[b], w_of(l));
                }
            });
        n_last = warp_sum(n_last);
        w_last = warp_sum(w_last);
        if (kSingle) w_zero = warp_sum(w_zero);
        if (lane == 0) {
            if (n_last) atomicAdd(&dy.count[kBins - 1], n_last);
            if (w_last) add_to(&dy.lo[kBins - 1], &dy.hi[kBins - 1], w_last);
            if (kSingle && w_zero) add_to(&dy.lo[bins.zero], &dy.hi[bins.zero], w_zero);
        }
        // the row's bins: each CTA adds what it counted to the CTAs whose share of the bins that is
        const int share = kBins / (int)size, first = (int)rank * share, per = (share + kThreads - 1) / kThreads;
        auto push = [&](bool counts, int from, int to) {           // (behind a barrier)
            for (int b = from + tid; b < to; b += kThreads) {
                const uint32_t o = (uint32_t)(b / share), n0 = dy.count[b], l = dy.lo[b], h = dy.hi[b];
                if (counts && n0) add_cluster(tc::map_to_rank(&dy.all_count[b], o), n0);
                if (l | h) add_to_cluster(tc::map_to_rank(&dy.all_lo[b], o), tc::map_to_rank(&dy.all_hi[b], o), ((uint64_t)h << 32) | l);
            }
            tc::cluster_sync();
        };
        // this thread's bins, `per` from b0 on, at most four; tokens and mass of the bins before them, and of all
        const int b0 = first + tid * per, b1 = min(b0 + per, first + share);
        uint32_t cnt[4];
        uint64_t mass[4], ma, mt;
        uint32_t ca, ct;
        auto total_up = [&]() {
            uint64_t sm = 0;
            uint32_t sc = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = b0 + k;
                cnt[k] = b < b1 ? dy.all_count[b] : 0;
                mass[k] = b < b1 ? ((uint64_t)dy.all_hi[b] << 32) + dy.all_lo[b] : 0;
                if (kSingle && cnt[k] && bins.single(b)) mass[k] = w_of(bins.value(b)) * cnt[k];
                sc += cnt[k];
                sm += mass[k];
            }
            block_scan(sh, sm, sc, ma, ca, mt, ct);
            if (tid < (int)size) {
                st_cluster(tc::map_to_rank(&sh.mass_of[rank], (uint32_t)tid), mt);
                st_cluster(tc::map_to_rank(&sh.count_of[rank], (uint32_t)tid), ct);
            }
            tc::cluster_sync();
            mt = 0;
            for (uint32_t o = 0; o < size; ++o) {
                if (o < rank) {
                    ma += sh.mass_of[o];
                    ca += sh.count_of[o];
                }
                mt += sh.mass_of[o];
            }
        };
        __syncthreads();
        if (table_w)                                           // weights of the slice's own values
            for (int b = tid; b < kBins; b += kThreads)
                if (dy.count[b] && bins.single(b)) dy.w[b] = w_of(bins.value(b));
        push(true, 0, kBins);
        total_up();
        if (kSingle && rank == 0 && tid == 0) z = mt >> 2;     // (bf16: every token's weight)
        // ties of weight wx to keep so that `up` and they reach the goal: one at least, `cap` at most
        auto ties_for = [&](uint64_t goal, uint64_t up, uint64_t wx, uint64_t cap) -> uint64_t {
            if (wx == 0 || goal <= up) return 1;
            return min((goal - up + wx - 1) / wx, cap);
        };
        // Where a border falls (stage 0: top-k's, 1: top-p's), told to the cluster by the one thread that finds it; for a
        // bin of one value the border itself.
        auto here = [&](int stage, int b, uint32_t before, uint32_t in, uint64_t m0, uint32_t want, uint64_t goal, const Border &most) {
            Border bd = {0u, 0u};
            uint64_t kept = 0;
            if (kSingle && bins.single(b)) {
                const uint64_t wx = w_of(bins.value(b));
                bd.key = order_key(bins.value(b));
                bd.ties = want ? want - before : (uint32_t)ties_for(goal, m0, wx, bd.key == most.key ? most.ties : in);
                kept = m0 + bd.ties * wx;
            }
            for (uint32_t o = 0; o < size; ++o) {
                st_cluster(tc::map_to_rank(&sh.bin[stage], o), (uint32_t)b);
                st_cluster(tc::map_to_rank(&sh.before[stage], o), before);
                st_cluster(tc::map_to_rank(&sh.in_bin[stage], o), in);
                st_cluster(tc::map_to_rank(&sh.mass_before[stage], o), m0);
                st_cluster(tc::map_to_rank(&sh.border[stage].key, o), bd.key);
                st_cluster(tc::map_to_rank(&sh.border[stage].ties, o), bd.ties);
                st_cluster(tc::map_to_rank(&sh.above[stage], o), kept);
            }
        };
        // the bin that holds the last token of `want`, or the first with `goal` of mass up to and with it
        auto find_count = [&](uint32_t want) {
            uint32_t n0 = ca;
            uint64_t m0 = ma;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (n0 < want && want <= n0 + cnt[k]) here(0, b0 + k, n0, cnt[k], m0, want, 0, Border{0u, 0u});
                n0 += cnt[k];
                m0 += mass[k];
            }
            tc::cluster_sync();
        };
        auto find_mass = [&](uint64_t goal, const Border &most) {
            uint32_t n0 = ca;
            uint64_t m0 = ma;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (cnt[k] && m0 + mass[k] >= goal && !(n0 > 0 && m0 >= goal)) here(1, b0 + k, n0, cnt[k], m0, 0u, goal, most);
                n0 += cnt[k];
                m0 += mass[k];
            }
            tc::cluster_sync();
        };
        // the tokens of a stage's bin to the first CTA, as (key, token)
        auto gather = [&](int stage) {
            const int b = sh.bin[stage];
            const uint32_t counter = tc::map_to_rank(&sh.list_n[stage], 0), base = tc::map_to_rank(list + stage * kList, 0);
            each([&](float l, int i) {
                const uint32_t key = order_key(l);
                if (bins.of(key) == b) {
                    const uint32_t at = add_cluster(counter, 1u);
                    if (at < kList) st_cluster(base + 8 * at, ((uint64_t)key << 32) | (uint32_t)(v0 + i));
                }
                return false;
            }, none);
            tc::cluster_sync();
        };
        // What the cluster is told: the border, and the mass up to and with it.
        auto tell = [&](int stage, uint32_t o, uint32_t key, uint64_t ties, uint64_t kept) {
            st_cluster(tc::map_to_rank(&sh.border[stage].key, o), key);
            st_cluster(tc::map_to_rank(&sh.border[stage].ties, o), (uint32_t)ties);
            st_cluster(tc::map_to_rank(&sh.above[stage], o), kept);
        };
        // In the first CTA: of the listed tokens in order the least number with `want` tokens, or (want 0) with a mass
        // that with `before` reaches the goal, of those that `most` keeps. Short lists: a thread a token, which counts
        // and weighs those before its own; the one at the border tells. Others: the range of keys is halved, the tokens
        // in registers.
        auto select = [&](int stage, uint32_t want, uint64_t goal, uint64_t before, const Border &most) {
            const uint32_t ln = sh.list_n[stage];
            const uint64_t *li = list + stage * kList;
            if (rank == 0 && ln <= kShort) {
                if ((tid & ~31u) < ln) {
                    const uint64_t w = w_of(key_logit(tid < ln ? (uint32_t)(li[tid] >> 32) : order_key(m)));
                    if (tid < ln) dy.list_w[tid] = w;
                }
                __syncthreads();
                if (tid < ln) {
                    const uint32_t key = (uint32_t)(li[tid] >> 32), at = (uint32_t)li[tid];
                    const uint64_t w = dy.list_w[tid];
                    uint64_t up = before;                      // mass of larger ones
                    uint32_t larger = 0, equal = 0;            // and their number; equal ones before this
#pragma unroll 4
                    for (uint32_t i = 0; i < ln; ++i) {
                        const uint64_t e = li[i], we = dy.list_w[i];
                        const uint32_t k = (uint32_t)(e >> 32);
                        if (k > key) {
                            ++larger;
                            up += we;
                        }
                        equal += k == key && (uint32_t)e < at;
                    }
                    bool border;
                    if (want) border = larger + equal + 1 == want;
                    else {
                        const bool may = key > most.key || (key == most.key && equal < most.ties);
                        border = may && (larger + equal == 0 || up + equal * w < goal) && up + (equal + 1) * w >= goal;
                    }
                    if (border)
                        for (uint32_t o = 0; o < size; ++o) tell(stage, o, key, equal + 1, up + (equal + 1) * w);
                }
            } else if (rank == 0) {
                uint32_t lo = 0u, hi = order_key(m);
                const int b = sh.bin[stage];
                if (bins.single(b)) {                          // its keys share their upper half
                    const uint32_t h = b < bins.pos ? bins.top - (uint32_t)b : bins.low - (uint32_t)(b - bins.neg);
                    lo = h << 16;
                    hi = min(hi, lo | 0xffffu);
                }
                lo = max(lo, most.key);
                uint32_t key[kHold];
                uint64_t w[kHold], t = 0;
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    const uint32_t i = tid + k * kThreads;
                    key[k] = i < ln ? (uint32_t)(li[i] >> 32) : 0u;        // 0 is no number's key
                    w[k] = w_of(key_logit(i < ln ? key[k] : order_key(m)));
                    if (i >= ln || key[k] < most.key) key[k] = 0u;
                    if (key[k] && key[k] == most.key) ++t;
                    if (key[k] <= most.key) w[k] = 0;          // (the border's own: `equal`, as many as are kept)
                }
                uint64_t equal = 0;
                if (most.key) equal = min(block_sum(sh, t), (uint64_t)most.ties) * w_of(key_logit(most.key));
                auto measure = [&](uint32_t x, bool mass_of) -> uint64_t {     // of keys x and above
                    uint64_t s = 0;
#pragma unroll
                    for (int k = 0; k < kHold; ++k) s += key[k] >= x && key[k] ? (mass_of ? w[k] : 1) : 0;
                    return block_sum(sh, s) + (mass_of && x <= most.key ? equal : 0);
                };
                const bool mm = want == 0;
                while (lo < hi) {                              // the largest key with enough at or above it
                    const uint32_t mid = lo + (hi - lo + 1) / 2;
                    const uint64_t s = measure(mid, mm);
                    if (mm ? before + s >= goal : s >= want) lo = mid;
                    else hi = mid - 1;
                }
                const uint64_t up = before + measure(lo + 1, true), wx = w_of(key_logit(lo));
                const uint64_t ties = mm ? ties_for(goal, up, wx, lo == most.key ? most.ties : 0xffffffffu) : want - measure(lo + 1, false);
                if (tid < (int)size) tell(stage, (uint32_t)tid, lo, ties, up + ties * wx);
            }
            tc::cluster_sync();
        };
        // the same over the whole row, for bins that the list cannot hold (slow, see above)
        auto search_row = [&](int stage, uint32_t want, uint64_t goal, const Border &most) {
            if (rank == 0) {
                const E *whole = src;                          // (rank 0's slice starts the row)
                auto measure = [&](uint32_t x, bool mm) -> uint64_t {
                    uint64_t s = 0, t = 0;
                    for (int i = tid; i < p.V; i += kThreads) {
                        const float l = as_f32(whole[i]);
                        const uint32_t k = order_key(l);
                        if (k < x || k < most.key) continue;
                        if (!mm) ++s;
                        else if (k == most.key) ++t;
                        else s += w_of(l);
                    }
                    s = block_sum(sh, s);
                    if (mm) {
                        t = block_sum(sh, t);
                        if (t) s += min(t, (uint64_t)most.ties) * w_of(key_logit(most.key));
                    }
                    return s;
                };
                const bool mm = want == 0;
                uint32_t lo = most.key, hi = order_key(m);
                while (lo < hi) {
                    const uint32_t mid = lo + (hi - lo + 1) / 2;
                    const uint64_t s = measure(mid, mm);
                    if (mm ? s >= goal : s >= want) lo = mid;
                    else hi = mid - 1;
                }
                const uint64_t up = lo == 0xffffffffu ? 0 : measure(lo + 1, mm), wx = w_of(key_logit(lo));
                const uint64_t ties = mm ? ties_for(goal, up, wx, lo == most.key ? most.ties : 0xffffffffu) : want - up;
                const uint64_t up_mass = mm ? up : (lo == 0xffffffffu ? 0 : measure(lo + 1, true));
                if (tid < (int)size) tell(stage, (uint32_t)tid, lo, ties, up_mass + ties * wx);
            }
            tc::cluster_sync();
        };
        uint64_t kept_mass = mt;                               // of the top-k's tokens
        if (by_count) {
            find_count((uint32_t)top_k);
            const bool listed = sh.in_bin[0] <= kList;
            if (!(kSingle && bins.single(sh.bin[0]))) {
                if (listed) {
                    gather(0);
                    select(0, (uint32_t)top_k - sh.before[0], 0, kSingle ? sh.mass_before[0] : 0, Border{0u, 0u});
                } else
                    search_row(0, (uint32_t)top_k, 0, Border{0u, 0u});
            }
            border = sh.border[0];
            kept_mass = sh.above[0];
            if (!kSingle && by_mass) {                         // the masses of what top-k keeps, the border's bin whole
                const int last = bins.of(border.key);
                auto add = [&](float l) {
                    const int q = bins.of(bits_key(l));
                    if (q < last) add_to(&dy.lo[q], &dy.hi[q], w_of(l));
                };
                each([&](float l, int) { return bins.of(bits_key(l)) < last; }, add);
                __syncthreads();
                push(false, 0, last);
                total_up();
                // (the border's bin: what the list, or the row, has kept)
                kept_mass = listed ? mt + sh.above[0] : sh.above[0];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (b0 + k == last && b0 + k < b1) mass[k] = kept_mass - mt;
            }
        }
        if (by_mass) {
            if (tid == 0) {
                const double top_p = p.top_p ? (double)p.top_p[r] : p.top_p_all;
                sh.goal = (uint64_t)ceil(fmax(top_p, 0.0) * (double)kept_mass);
            }
            __syncthreads();
            const uint64_t goal = sh.goal;
            const Border most = by_count ? border : Border{0u, (uint32_t)p.V};
            find_mass(goal, most);
            if (!(kSingle && bins.single(sh.bin[1]))) {
                if (sh.in_bin[1] <= kList) {
                    gather(1);
                    select(1, 0u, goal, sh.mass_before[1], most);
                } else
                    search_row(1, 0u, goal, most);
            }
            border = sh.border[1];
        }
    }
    __syncthreads();

    // -- what is kept of each warp's part: mass above the border, and its ties
    const int part = (p.slice / 16 + kWarps - 1) / kWarps * 16;
    const uint64_t wx = w_of(key_logit(border.key));
    const bool ties_kept = wx >= least;
    auto exact = [&](float l, uint32_t key) -> uint64_t {      // of a token above the border or below
        const uint64_t w = key > border.key && l > -INFINITY ? w_of(l) : 0;
        return w >= least ? w : 0;
    };
    constexpr uint64_t kNone = ~0ull;                          // a bin of several values
    if (table_w) {                                             // the table's weights are what is kept of them
        for (int b = tid; b < kBins; b += kThreads)
            if (dy.count[b])
                dy.w[b] = !bins.single(b) ? kNone : (order_key(bins.value(b)) > border.key && dy.w[b] >= least ? dy.w[b] : 0);
        __syncthreads();
    }
    auto table_of = [&](float l) -> uint64_t { return table_w ? dy.w[bins.of(bits_key(l))] : kNone; };
    auto weigh = [&](float l) -> uint64_t {
        const uint64_t w = table_of(l);
        return (uint32_t)(w >> 32) != ~0u ? w : exact(l, order_key(l));
    };
    const float at_border = key_logit(border.key);             // (everything: NaN, equal to none and below none)
    auto measure = [&](int i0, int i1, uint64_t &sum, uint32_t &ties) {      // (a warp's lanes side by side)
        uint64_t s = 0;
        uint32_t t = 0;
        // like `each`: what the table has at once, the others one by one
        auto take = [&](float l) -> bool {
            t += l == at_border;
            const uint64_t w = table_of(l);
            const bool has = (uint32_t)(w >> 32) != ~0u;
            s += has ? w : 0;
            return !has && !(l <= at_border);
        };
        int i = i0;
        if ((p.cache || p.vec) && i0 % kPer == 0) {            // (the slices' and the warps' parts start so)
            const int nq = (i1 - i0) / kPer;
            const uint4 *q = reinterpret_cast<const uint4 *>(data + i0);
            for (int j0 = lane; j0 < nq; j0 += 4 * 32) {
                uint4 v[4];
                uint32_t more = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (j0 + 32 * u < nq) v[u] = q[j0 + 32 * u];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (j0 + 32 * u >= nq) break;
                    const E *e = reinterpret_cast<const E *>(&v[u]);
                    float most;                                // nothing kept: most vectors, where few tokens are
                    if constexpr (kSingle) {
                        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&v[u]);
                        const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
                        most = fmaxf(f.x, f.y);
                    } else
                        most = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                    if (most < at_border) continue;
#pragma unroll
                    for (int k = 0; k < kPer; ++k) more |= (take(as_f32(e[k])) ? 1u : 0u) << (u * kPer + k);
                }
                while (more) {
                    const int k = __ffs(more) - 1;
                    more &= more - 1;
                    const float l = as_f32(data[i0 + (j0 + 32 * (k / kPer)) * kPer + k % kPer]);
                    s += exact(l, order_key(l));
                }
            }
            i += nq * kPer;
        }
#pragma unroll 1
        for (i += lane; i < i1; i += 32) {
            const float l = as_f32(data[i]);
            if (take(l)) s += exact(l, order_key(l));
        }
        sum = warp_sum(s);
        ties = warp_sum(t);
    };
    uint64_t sum;
    uint32_t ties;
    const int w0 = min(warp * part, n), w1 = min(w0 + part, n);
    measure(w0, w1, sum, ties);
    __syncthreads();
    if (lane == 0) {
        sh.part[warp] = sum;
        sh.part2[warp] = ties;
    }
    if (!kSingle) z = warp_sum((uint64_t)((int64_t)z_hi * (1 << 22) + z_lo));
    __shared__ uint64_t zs[kWarps];
    if (lane == 0) zs[warp] = z;
    __syncthreads();
    if (warp == 0) {
        const uint64_t s = warp_sum(sh.part[lane]);
        const uint32_t t = warp_sum(sh.part2[lane]);
        const uint64_t zz = warp_sum(zs[lane]);
        if (lane < (int)size) {
            st_cluster(tc::map_to_rank(&sh.sum[rank], (uint32_t)lane), s);
            st_cluster(tc::map_to_rank(&sh.ties[rank], (uint32_t)lane), t);
            st_cluster(tc::map_to_rank(&sh.z[rank], (uint32_t)lane), zz);
        }
    }
    tc::cluster_sync();
    // ties are kept in index order: `left` of them from a place on
    auto of_ties = [&](uint32_t left, uint32_t t) { return ties_kept ? (uint64_t)min(left, t) * wx : 0; };
    uint64_t all = 0, before = 0, mine = 0;
    uint32_t left = border.ties, left_mine = 0;
    for (uint32_t o = 0; o < size; ++o) {
        const uint64_t k = sh.sum[o] + of_ties(left, sh.ties[o]);
        if (o == rank) {
            before = all;
            mine = k;
            left_mine = left;
        }
        all += k;
        left -= min(left, sh.ties[o]);
    }
    if (tid == 0) {
        const double td = (double)p.u[r] * (double)all;
        const uint64_t t = td > 0.0 ? (uint64_t)td : 0;
        sh.t = t >= all ? all - 1 : t;
    }
    __syncthreads();
    uint64_t t = sh.t;
    if (t < before || t >= before + mine) return;              // another CTA's (nothing of this one is read from now on)
    t -= before;
    // which warp's part, then which of its 32 pieces, then which token
    auto locate = [&](uint64_t base, uint32_t lf) {            // by every warp alike, over sh.part and sh.part2
        const uint64_t s = sh.part[lane];
        const uint32_t q = sh.part2[lane];
        uint32_t iq = q;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, iq, off);
            if (lane >= off) iq += y;
        }
        const uint32_t lf0 = lf - min(lf, iq - q);
        uint64_t k = s + of_ties(lf0, q), ik = k;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, ik, off);
            if (lane >= off) ik += y;
        }
        const bool here = t >= base + ik - k && t < base + ik;
        const int o = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
        __syncthreads();
        if (warp == 0 && lane == o) {
            sh.found = o;
            sh.at = base + ik - k;
            sh.ties_at = lf0;
        }
        __syncthreads();
    };
    locate(0, left_mine);
    const int p0 = min(sh.found * part, n), p1 = min(p0 + part, n), piece = (p1 - p0 + kWarps - 1) / kWarps;
    uint64_t base = sh.at;
    uint32_t lf = sh.ties_at;
    const int q0 = min(p0 + warp * piece, p1), q1 = min(q0 + piece, p1);
    measure(q0, q1, sum, ties);
    __syncthreads();
    if (lane == 0) {
        sh.part[warp] = sum;
        sh.part2[warp] = ties;
    }
    __syncthreads();
    locate(base, lf);
    if (warp != sh.found) return;
    base = sh.at;
    lf = sh.ties_at;
    for (int i0 = q0; i0 < q1; i0 += 32) {
        const int i = i0 + lane;
        const float l = i < q1 ? as_f32(data[i]) : -INFINITY;
        const uint32_t key = order_key(l);
        const bool tie = i < q1 && key == border.key;
        const uint32_t tm = __ballot_sync(0xffffffffu, tie), tb = __popc(tm & ((1u << lane) - 1));
        uint64_t w = 0;
        if (i < q1 && key > border.key) w = weigh(l);
        if (tie && tb < lf && ties_kept) w = wx;
        uint64_t ik = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, ik, off);
            if (lane >= off) ik += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, base + ik > t);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                p.token[r] = v0 + i;
                if (p.logp) {
                    uint64_t zz = 0;                           // in units of 2^-42
                    for (uint32_t o = 0; o < size; ++o) zz += sh.z[o];
                    const double temp = p.temperature ? (double)p.temperature[r] : p.temperature_all;
                    p.logp[r] = greedy ? 0.f : (float)(((double)l - (double)m) / temp - log((double)zz * 2.2737367544323206e-13));
                }
            }
            return;
        }
        base += __shfl_sync(0xffffffffu, ik, 31);
        lf -= min(lf, (uint32_t)__popc(tm));
    }
}

// Clusters of C CTAs that the device holds at once.
template <typename E> int resident(cudaLaunchConfig_t cfg, int C) {
    static std::atomic<int> cached[64][kMaxCluster + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) dev = 0;
    std::atomic<int> &slot = cached[dev & 63][C];
    int n = slot.load(std::memory_order_relaxed);
    if (n > 0) return n;
    cfg.gridDim = dim3((unsigned)C);
    cfg.dynamicSmemBytes = kMostSmem;
    cfg.attrs[0].val.clusterDim.x = (unsigned)C;
    if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<E>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();                                    // clear the query's error
        return sm_count() / C;
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

template <typename E> cudaError_t launch(SampleParams p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kMaxCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // CTAs a row: as many as the device holds at once for the batch, of 2048 tokens or more each
    int C = kMaxCluster;
    while (C > 1 && (p.V < 2048 * C || p.R > resident<E>(cfg, C))) C >>= 1;
    p.slice = ((p.V + C - 1) / C + 15) / 16 * 16;
    const size_t fixed = sizeof(Dyn) + 2 * kList * sizeof(uint64_t), slice = (size_t)p.slice * sizeof(E);
    p.cache = fixed + slice <= kMostSmem;
    at[0].val.clusterDim.x = (unsigned)C;
    cfg.gridDim = dim3((unsigned)(p.R * C));
    cfg.dynamicSmemBytes = fixed + (p.cache ? slice : 0);
    static const Exp2Table table = make_table();
    return cudaLaunchKernelEx(&cfg, sample_kernel<E>, p, table);
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
    if (a->R == 0) return clear_error(a->err, stream);
    if (!a->logits || !a->u || !a->token) return KDT_ERR_NULL_ARG;
    if (!aligned(a->logits, esz)) return KDT_ERR_BAD_SHAPE;
    for (const void *q : {(const void *)a->u, (const void *)a->temperature, (const void *)a->top_k, (const void *)a->top_p,
                          (const void *)a->min_p, (const void *)a->token, (const void *)a->logp, (const void *)a->err})
        if (!aligned(q, 4)) return KDT_ERR_BAD_SHAPE;
    const kdt_status st = check_on_current_device(
        {a->logits, a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->token, a->logp, a->err});
    if (st != KDT_OK) return st;
    if (a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t), stream) != cudaSuccess) return KDT_ERR_CUDA;
    SampleParams p = {a->logits, stride, a->R, a->V, a->u, a->temperature, a->top_p, a->min_p, a->top_k, a->temperature_all,
                            a->top_p_all, a->min_p_all, a->top_k_all, a->token, a->err, a->logp, 0, 0, 0};
    p.vec = aligned(a->logits, 16) && (stride * esz) % 16 == 0;
    const cudaError_t e = a->dtype == KDT_F32 ? launch<float>(p, stream) : launch<__nv_bfloat16>(p, stream);
    return e == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}
