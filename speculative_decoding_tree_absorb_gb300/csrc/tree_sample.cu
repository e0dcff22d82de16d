// Sampled verification of a draft tree: which drafted tokens stand under the target's
// probabilities, decided from given random numbers (kdt_tree_sample).
//
// At a node the target's distribution over the vocabulary is p = softmax(logits / temperature).
// The children are tried in index order: child c stands with probability p(c) / (1 - the
// probability of the siblings tried before), that is when u_c (Z - sum of their weights) <
// w_c with w = e^{(l - max l) / temperature} and Z the sum of all w. If none stands, the
// token after the path is drawn from what is left of p without the children, as the first
// token whose running sum exceeds u_bonus times the rest. Tokens so emitted are distributed
// as the target's own samples, whatever tree was drafted.
//
//  * A cluster of CTAs takes one sequence, each a contiguous slice of the vocabulary, and
//    walks down together: only the rows on the path are read, once, kept in shared memory
//    where they fit. A step is one pass for the slice's maximum and sum, one exchange of
//    (maximum, sum) through distributed shared memory, and the children's tests, which every
//    CTA makes alike from the same numbers.
//  * The walk's sums use the fast exponential and float32; a test closer than kMargin of Z is
//    made again with the exact sums. The fast Z is off by at most 1.9e-5 of itself: 264 roundings
//    in a row (V = 524288 in float32 with one CTA a sequence: 256 vectors a thread, 3 sums within
//    one, 5 shuffles; bf16 140) give 1.58e-5; a weight 2^-|y| is off by 2^-22 and by
//    2.1 2^-24 |y| (three roundings of y), with |y| at most 14.3 on average over the sum (V tokens
//    of 2^-|y| beside the largest), 1.8e-6; the slices' factors 3e-7. A test in float32 adds
//    three roundings a child, 5.8e-6 for kFewKids: together below kMargin. An accepted
//    token's log-probability is made from the fast Z.
//  * Drawing from the rest needs more: the threshold falls between two of V running sums, and
//    with float32 weights (errors of 1e-7) neighbours of small probability would be mixed up.
//    Weights are fixed-point numbers there, w = round(2^44 e^y): integer sums do not depend on
//    their order, so any split gives the same token. weight() computes them from pairs of
//    float32 numbers (an FP64 operation of one warp takes 16 clocks here): y log2(e) = n + k / 128
//    + r, e^y = 2^n 2^{k/128} (1 + q + q^2/2 + ...), q = r ln 2 <= 0.0028, the leading terms as
//    pairs. Its error is below 2^-40 of the weight.
//  * What bounds it is the chain of a step, not its bytes: about 2.5 us of loads, two block sums,
//    the exchange and the tests, 0.8 us for 160000 tokens over 8 CTAs, and once a sequence
//    8 us of weights and 3 of sums for the draw. Measured: 8 sequences, 64 nodes, 160000 tokens
//    in bf16 (paths of up to 6) 41 us, one sequence, 9 nodes, 32000 tokens in float32 19 us.
#include <math.h>

#include <atomic>

#include "sample_weights.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace weights;

constexpr int kNT = 512, kNW = kNT / 32;            // threads, warps a CTA
constexpr int kMaxCluster = 8;
constexpr size_t kMostSmem = 208 * 1024;            // beside Shared
constexpr double kMargin = 4e-5;
constexpr int kKeep = 32;                           // log-probabilities written at a time
constexpr int kFewKids = 32;                        // children whose first tests are made in float32

struct SampleParams {
    const int32_t *parent, *tok;
    const void *logits;
    const float *u_node, *u_bonus;
    int T, V;
    int64_t row_stride;                             // elements between rows of logits
    float c_hi, c_lo;                               // log2(e) / temperature as a pair
    double inv_temp;
    int slice;                                      // tokens a CTA takes (a multiple of 16)
    int vec;                                        // rows start on 16-byte boundaries
    int cache;                                      // a slice fits shared memory
    int32_t *acc_nodes, *n_acc, *bonus, *err;
    float *logp;
};

struct alignas(16) Slot {
    float m;                                        // slice maximum (-inf: nothing), or NaN
    float pad;
    double z;                                       // its sum, relative to m
};

struct Shared {
    float2 tab[129 * kCopies];
    Slot slot[2][kMaxCluster];                      // by exchange parity
    uint64_t exact[2][kMaxCluster];
    double z;
    double keep_z[kKeep];                           // what the path's log-probabilities are made of
    float keep_l[kKeep], keep_m[kKeep];
    float wz[kNW];
    float wm[kNW];
    uint64_t wx[kNW];                               // exact sums of the warps' parts
    uint64_t scan[kNW];
    int n_child, decision, found;
};

__host__ __device__ constexpr size_t list_bytes(int T) { return ((size_t)T * 36 + 15) / 16 * 16; }

// One cluster a sequence.
template <typename E>
__global__ void __launch_bounds__(kNT, 1) tree_sample_kernel(const SampleParams p,
                                                             const __grid_constant__ Exp2Table table) {
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ Shared sh;
    // children of the node at hand: exact weight (0 for a repeated token), node, token (INT32_MIN when
    // it is none), logit, random number; and the
    // tree's parents, tokens and random numbers
    uint64_t *cw = reinterpret_cast<uint64_t *>(dyn);
    int32_t *cn = reinterpret_cast<int32_t *>(cw + p.T), *ct = cn + p.T;
    float *cl = reinterpret_cast<float *>(ct + p.T), *cu = cl + p.T;
    int32_t *par = reinterpret_cast<int32_t *>(cu + p.T), *tok = par + p.T;
    float *un = reinterpret_cast<float *>(tok + p.T);
    E *row = reinterpret_cast<E *>(dyn + list_bytes(p.T));
    uint32_t rank, size;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int b = blockIdx.x / size, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t tb = (int64_t)b * p.T;
    const int v0 = min((int)rank * p.slice, p.V), n = min(p.slice, p.V - v0);
    for (int k = tid; k < 129 * kCopies; k += kNT) sh.tab[k] = make_float2(table.hi[k / kCopies], table.lo[k / kCopies]);
    const float2 *tab = sh.tab + lane % kCopies;
    for (int i = tid; i < p.T; i += kNT) {
        const int32_t pa = p.parent[tb + i];
        par[i] = pa;
        tok[i] = p.tok[tb + i];
        un[i] = p.u_node[tb + i];
        if (rank == 0) {
            p.acc_nodes[tb + i] = -1;
            if (p.logp) p.logp[tb + i] = 0.f;
            if (pa < -1 || pa >= i) record_error(p.err, (int32_t)(tb + i + 1));
        }
    }
    tc::cluster_arrive();      // every CTA runs before another writes to its shared memory (waited for there)
    __syncthreads();
    // a warp's part of the slice, in whole groups of 16 tokens
    const int part = (p.slice / 16 + kNW - 1) / kNW * 16;
    const int w0 = min(warp * part, n), w1 = min(w0 + part, n);

    // natural log of the probability of a token of logit l, M the row's maximum, z the sum of weights. The
    // FP64 log takes 2 k clocks: log z = log 2^e + logf(mantissa as float32) + the rest, to a unit of float32
    auto log_p = [&](float l, float M, double z) {
        const long long bits = __double_as_longlong(z);
        const int e = (int)(bits >> 52) - 1023;
        const double mant = __longlong_as_double((bits & 0xfffffffffffffll) | 0x3ff0000000000000ll);
        const float mf = (float)mant;
        const double log_mant = (double)logf(mf) + (double)__fdividef((float)(mant - (double)mf), mf);
        return (float)(((double)l - (double)M) * p.inv_temp - (log_mant + (e - kFrac) * 0.69314718055994530942));
    };
    auto write_kept = [&](int first, int count) {              // by the warp of the thread that kept them
        if (rank || warp || !p.logp) return;
        __syncwarp();
        if (lane < count) p.logp[tb + first + lane] = log_p(sh.keep_l[lane], sh.keep_m[lane], sh.keep_z[lane]);
        __syncwarp();
    };
    int node = 0, depth = 0;
    uint32_t step = 0;
    for (;;) {
        const E *src = static_cast<const E *>(p.logits) + (tb + node) * p.row_stride + v0;
        // -- the children, in index order (the last warp), and their logits
        if (warp == kNW - 1) {
            int c = 0;
            for (int i0 = node + 1; i0 < p.T; i0 += 32) {
                const int i = i0 + lane;
                const bool kid = i < p.T && par[i] == node;
                const uint32_t mask = __ballot_sync(0xffffffffu, kid);
                if (kid) cn[c + __popc(mask & ((1u << lane) - 1))] = i;
                c += __popc(mask);
            }
            __syncwarp();
            for (int k = lane; k < c; k += 32) {
                const int32_t t = tok[cn[k]];
                const bool good = t >= 0 && t < p.V;
                if (!good && rank == 0) record_error(p.err, (int32_t)(tb + cn[k] + 1));
                ct[k] = good ? t : INT32_MIN;
                cu[k] = un[cn[k]];
                cl[k] = good ? as_f32(static_cast<const E *>(p.logits)[(tb + node) * p.row_stride + t]) : -INFINITY;
            }
            if (lane == 0) sh.n_child = c;
        }
        // -- the slice's maximum (NaN wins), rows to shared memory on the way
        float m = -INFINITY;
        bool nan = false;
        auto see = [&](float x) {
            nan |= x != x;
            m = fmaxf(m, x);
        };
        constexpr int kPer = 16 / (int)sizeof(E);
        if (p.vec) {
            const int nv = n / kPer;
#pragma unroll 4
            for (int i = tid; i < nv; i += kNT) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
                if (p.cache) reinterpret_cast<uint4 *>(row)[i] = v;
                const E *e = reinterpret_cast<const E *>(&v);
#pragma unroll
                for (int k = 0; k < kPer; ++k) see(as_f32(e[k]));
            }
            for (int i = nv * kPer + tid; i < n; i += kNT) {
                if (p.cache) row[i] = src[i];
                see(as_f32(src[i]));
            }
        } else {
#pragma unroll 4
            for (int i = tid; i < n; i += kNT) {
                const E v = src[i];
                if (p.cache) row[i] = v;
                see(as_f32(v));
            }
        }
        if (nan) m = __uint_as_float(0x7fffffffu);
        auto top = [](float a, float c) { return a != a ? a : (c != c ? c : fmaxf(a, c)); };
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) sh.wm[warp] = m;
        __syncthreads();                                       // also: the row and the children are in place
        m = sh.wm[lane % kNW];
#pragma unroll
        for (int off = kNW / 2; off >= 1; off >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, off));
        const E *data = p.cache ? row : src;
        // -- the slice's sum relative to its maximum
        // (in float32 by vectors of 16 bytes, threads and warps: at most 264 roundings in a row; then in 64 bits)
        float z = 0.f;
        if (m > -INFINITY && m < INFINITY) {
            auto term = [&](float x) { return ex2((x - m) * p.c_hi); };
            if (p.cache || p.vec) {
                const int nv = n / kPer;
#pragma unroll 4
                for (int i = tid; i < nv; i += kNT) {
                    const uint4 v = reinterpret_cast<const uint4 *>(data)[i];
                    const E *e = reinterpret_cast<const E *>(&v);
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < kPer; ++k) s += term(as_f32(e[k]));
                    z += s;
                }
                for (int i = nv * kPer + tid; i < n; i += kNT) z += term(as_f32(data[i]));
            } else {
                for (int i0 = tid; i0 < n; i0 += 8 * kNT) {
                    float s = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (i0 + k * kNT < n) s += term(as_f32(data[i0 + k * kNT]));
                    z += s;
                }
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
        if (lane == 0) sh.wz[warp] = z;
        __syncthreads();
        // -- one exchange over the cluster
        Slot *slots = sh.slot[step & 1];
        if (step == 0) tc::cluster_wait();
        if (warp == 0) {
            double s = lane < kNW ? (double)sh.wz[lane] : 0.0;
#pragma unroll
            for (int off = kNW / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (lane < (int)size)
                tc::st_cluster_v4(tc::map_to_rank(&slots[rank], (uint32_t)lane), __float_as_uint(m), 0u,
                                  (uint32_t)__double2loint(s), (uint32_t)__double2hiint(s));
        }
        tc::cluster_sync();
        float M = lane % kMaxCluster < (int)size ? slots[lane % kMaxCluster].m : -INFINITY;
#pragma unroll
        for (int off = kMaxCluster / 2; off >= 1; off >>= 1) M = top(M, __shfl_xor_sync(0xffffffffu, M, off));
        if (!(M > -INFINITY && M < INFINITY)) {                // no distribution: the walk ends here
            if (rank == 0 && tid == 0) {
                record_error(p.err, (int32_t)(tb + node + 1));
                p.acc_nodes[tb + depth] = node;
                p.n_acc[b] = depth + 1;
                p.bonus[b] = -1;
            }
            break;
        }
        if (warp == 0) {                                       // Z in units of the weights, the same in every CTA
            double s = 0.0;
            if (lane < (int)size && slots[lane].m > -INFINITY)
                s = slots[lane].z * ((double)exp2f((slots[lane].m - M) * p.c_hi) * (double)(1ull << kFrac));
#pragma unroll
            for (int off = kMaxCluster / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if (lane == 0) sh.z = s;
        }
        // -- the children's weights; a repeated token counts once
        const int nc = sh.n_child;
        for (int k = tid >= 32 ? tid - 32 : kNT - 32 + tid; k < nc; k += kNT) {   // (warp 0 is at the sum)
            cw[k] = ct[k] < 0 ? 0 : weight(cl[k], M, p.c_hi, p.c_lo, tab);
            for (int j = 0; j < k && cw[k]; ++j)
                if (ct[j] == ct[k]) cw[k] = 0;
        }
        __syncthreads();
        // -- the tests; with exact sums when one is too close (and for the draw)
        bool exact = false;
        int take = -1;
        for (;;) {
            if (tid == 0) {
                double rem = sh.z;
                int d = -1;                                    // -1: none stands, -2: too close
                // FP64 operations in a row take long here; float32 adds at most 3 roundings a child
                if (!exact && nc <= kFewKids) {
                    float left = (float)rem;
                    const float margin = (float)kMargin * left;
                    for (int k = 0; k < nc; ++k) {
                        const float w = (float)cw[k], t = cu[k] * left;
                        if (cw[k] == 0) continue;
                        if (fabsf(t - w) <= margin || t < w) {
                            d = fabsf(t - w) <= margin ? -2 : k;
                            break;
                        }
                        left -= w;
                    }
                } else {
                const double margin = exact ? -1.0 : kMargin * rem;
                for (int k = 0; k < nc; ++k) {
                    const double w = (double)cw[k];
                    if (cw[k] == 0) continue;
                    const double t = (double)cu[k] * rem;
                    if (fabs(t - w) <= margin) {
                        d = -2;
                        break;
                    }
                    if (t < w) {
                        d = k;
                        break;
                    }
                    rem -= w;
                }
                }
                sh.decision = d;
            }
            __syncthreads();
            take = sh.decision;
            if (take >= 0 || exact) break;
            // exact sums of the warps' parts, children included
            uint64_t x = 0;
#pragma unroll 4
            for (int i = w0 + lane; i < w1; i += 32) x += weight(as_f32(data[i]), M, p.c_hi, p.c_lo, tab);
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            if (lane == 0) sh.wx[warp] = x;
            __syncthreads();
            if (tid < (int)size) {
                uint64_t s = 0;
                for (int k = 0; k < kNW; ++k) s += sh.wx[k];
                const uint32_t dst = tc::map_to_rank(&sh.exact[step & 1][rank], (uint32_t)tid);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(dst), "l"(s) : "memory");
            }
            tc::cluster_sync();
            if (tid == 0) {
                uint64_t s = 0;
                for (uint32_t k = 0; k < size; ++k) s += sh.exact[step & 1][k];
                sh.z = (double)s;
            }
            exact = true;
            if (take == -1) break;                             // no test was close: none stands
        }
        if (rank == 0 && tid == 0) {
            p.acc_nodes[tb + depth] = node;
            if (take >= 0) {                                   // their FP64 log is off the walk's path
                sh.keep_z[depth % kKeep] = sh.z;
                sh.keep_l[depth % kKeep] = cl[take];
                sh.keep_m[depth % kKeep] = M;
            }
        }
        ++step;
        if (take >= 0) {
            node = cn[take];
            ++depth;
            if (depth % kKeep == 0) write_kept(depth - kKeep, kKeep);
            __syncthreads();                                   // the children's arrays are rewritten next
            continue;
        }
        // -- the draw from the rest: the least token with running sum > t, children left out
        uint64_t before = 0, mine = 0, all = 0, kids = 0;
        for (uint32_t k = 0; k < size; ++k) {
            const uint64_t x = sh.exact[(step - 1) & 1][k];
            if (k < rank) before += x;
            if (k == rank) mine = x;
            all += x;
        }
        for (int k = 0; k < nc; ++k) {
            if (!cw[k]) continue;
            kids += cw[k];
            if (ct[k] < v0) before -= cw[k];
            else if (ct[k] < v0 + n) mine -= cw[k];
        }
        const uint64_t rest = all - kids;
        if (tid == 0) {
            const double td = (double)p.u_bonus[b] * (double)rest;
            const uint64_t t = td > 0.0 ? (uint64_t)td : 0;
            sh.scan[0] = rest > 0 && t >= rest ? rest - 1 : t;
        }
        __syncthreads();
        uint64_t t = sh.scan[0];
        if (rank == 0 && tid == 0) {
            p.n_acc[b] = depth + 1;
            if (rest == 0) {                                   // only with a u_node of 1 or more
                p.bonus[b] = -1;
                record_error(p.err, (int32_t)(tb + node + 1));
            }
        }
        if (rest == 0 || t < before || t >= before + mine) break;     // not this CTA's slice
        t -= before;
        // which warp's part (children taken out of the parts' sums), then which token of it
        __syncthreads();
        if (tid == 0) {
            for (int k = 0; k < nc; ++k)
                if (cw[k] && ct[k] >= v0 && ct[k] < v0 + n) sh.wx[(ct[k] - v0) / part] -= cw[k];
            int o = 0;
            uint64_t acc = 0;
            while (o < kNW - 1 && t >= acc + sh.wx[o]) acc += sh.wx[o++];
            sh.found = o;
            sh.scan[0] = acc;
        }
        __syncthreads();
        t -= sh.scan[0];
        const int o0 = min(sh.found * part, n), o1 = min(o0 + part, n), per = (o1 - o0 + kNT - 1) / kNT;
        const int e0 = min(o0 + tid * per, o1), e1 = min(e0 + per, o1);
        auto left = [&](int i) -> uint64_t {                   // weight of slice token i, 0 for a child's
            for (int k = 0; k < nc; ++k)
                if (ct[k] == v0 + i) return 0;
            return weight(as_f32(data[i]), M, p.c_hi, p.c_lo, tab);
        };
        uint64_t sum = 0;
        for (int i = e0; i < e1; ++i) sum += left(i);
        uint64_t incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        __syncthreads();
        if (lane == 31) sh.scan[warp] = incl;
        __syncthreads();
        uint64_t base = incl - sum;
        for (int k = 0; k < warp; ++k) base += sh.scan[k];
        if (t >= base && t < base + sum) {
            int i = e0;
            uint64_t acc = base;
            for (; i < e1; ++i) {
                acc += left(i);
                if (acc > t) break;
            }
            p.bonus[b] = v0 + i;
            if (p.logp) p.logp[tb + depth] = log_p(as_f32(data[i]), M, sh.z);
        }
        break;
    }
    write_kept(depth - depth % kKeep, depth % kKeep);
    tc::cluster_sync();        // no CTA leaves while another may still write to its shared memory
}

// Clusters of C CTAs that the device holds at once (a cluster lies within one GPC: 15 of 8, 36 of 4, 76 of 2).
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
    if (cudaOccupancyMaxActiveClusters(&n, tree_sample_kernel<E>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();                                    // clear the query's error
        return sm_count() / C;
    }
    slot.store(n, std::memory_order_relaxed);
    return n;
}

template <typename E> cudaError_t launch(SampleParams p, int B, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(tree_sample_kernel<E>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kMaxCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kNT);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // CTAs a sequence: as many as the device holds at once for the batch, of 1024 tokens or more each
    // (16 gave one sequence of 32000 tokens nothing, and only 7 such clusters are held)
    int C = kMaxCluster;
    while (C > 1 && (p.V < 1024 * C || B > resident<E>(cfg, C))) C >>= 1;
    p.slice = ((p.V + C - 1) / C + 15) / 16 * 16;
    const size_t lists = list_bytes(p.T), slice = (size_t)p.slice * sizeof(E);
    p.cache = lists + slice <= kMostSmem;
    const size_t smem = lists + (p.cache ? slice : 0);
    at[0].val.clusterDim.x = (unsigned)C;
    cfg.gridDim = dim3((unsigned)(B * C));
    cfg.dynamicSmemBytes = smem;
    static const Exp2Table table = make_table();
    return cudaLaunchKernelEx(&cfg, tree_sample_kernel<E>, p, table);
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace kdt

using namespace kdt;

extern "C" {

kdt_status kdt_tree_sample(const int32_t *parent, const int32_t *tok, const void *logits, kdt_dtype dtype, int B, int T,
                           int V, int64_t row_stride, double temperature, const float *u_node, const float *u_bonus,
                           int32_t *acc_nodes, int32_t *n_acc, int32_t *bonus, float *logp, int32_t *err,
                           cudaStream_t stream) {
    if (B < 0 || B > 65535 || T < 1 || T > kMaxT || V < 1 || V > kMaxVocab) return KDT_ERR_BAD_SHAPE;
    if (dtype != KDT_F32 && dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    const int esz = dtype == KDT_F32 ? 4 : 2;
    const int64_t stride = row_stride ? row_stride : V;
    if (stride < V) return KDT_ERR_BAD_SHAPE;
    if (!(temperature >= 1e-3 && temperature <= 1e3)) return KDT_ERR_BAD_SHAPE;
    if (B > 0 && (!parent || !tok || !logits || !u_node || !u_bonus || !acc_nodes || !n_acc || !bonus))
        return KDT_ERR_NULL_ARG;
    if (!aligned(logits, esz)) return KDT_ERR_BAD_SHAPE;
    for (const void *q : {(const void *)parent, (const void *)tok, (const void *)u_node, (const void *)u_bonus,
                          (const void *)acc_nodes, (const void *)n_acc, (const void *)bonus, (const void *)logp,
                          (const void *)err})
        if (!aligned(q, 4)) return KDT_ERR_BAD_SHAPE;
    if (B == 0) return clear_error(err, stream);
    const kdt_status st =
        check_on_current_device({parent, tok, logits, u_node, u_bonus, acc_nodes, n_acc, bonus, logp, err});
    if (st != KDT_OK) return st;
    if (err && cudaMemsetAsync(err, 0, sizeof(int32_t), stream) != cudaSuccess) return KDT_ERR_CUDA;
    SampleParams p = {};
    p.parent = parent;
    p.tok = tok;
    p.logits = logits;
    p.u_node = u_node;
    p.u_bonus = u_bonus;
    p.T = T;
    p.V = V;
    p.row_stride = stride;
    const double c = 1.4426950408889634074 / temperature;
    p.c_hi = (float)c;
    p.c_lo = (float)(c - (double)p.c_hi);
    p.inv_temp = 1.0 / temperature;
    p.vec = aligned(logits, 16) && (stride * esz) % 16 == 0;
    p.acc_nodes = acc_nodes;
    p.n_acc = n_acc;
    p.bonus = bonus;
    p.logp = logp;
    p.err = err;
    const cudaError_t e = dtype == KDT_F32 ? launch<float>(p, B, stream) : launch<__nv_bfloat16>(p, B, stream);
    return e == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
