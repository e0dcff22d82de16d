// K5: tree-verify attention over the 8-bit latent cache for few query rows a sequence
// (single tokens, small trees): tcgen05 with the KEYS on the M side.
//
// The definition is kdt_verify_attn's over the cache's values: scores s_j = scale (q_nope .
// c_j + q_pe . k_j) of a row over its visible keys, softmax, out = sum p_j c_j, lse.
//
//  * A work item is up to 64 query rows (heads x tree nodes) of one sequence over a run of
//    128-key blocks. With so few rows the tensor cores are filled from the other side:
//    S^T = K Q^T has M = 128 keys, N = 64 rows, and O^T = V^T P^T has M = 128 latent dims
//    (four tiles), N = 64 rows. A row tile of 64 on the M side would leave half of every
//    MMA idle.
//  * The cache is read once, in 8 bits. Converter warps load codes to registers, widen them
//    to bf16 (exact: e4m3 times a power of two is a bf16 number) and store them as 128-byte
//    swizzled [128 keys x 64 dims] tiles. ONE copy serves both contractions: K-major A
//    operand of S^T, MN-major A operand of O^T. Four pairs of tiles (128 dims each) are
//    released one by one as O^T's four tiles are issued, so the next block's conversion and
//    scores follow pair by pair.
//  * Rope keys take a ninth tile; once a block's scores are done its space holds P^T
//    (128 keys x 64 rows, bf16, an MN-major B operand: a thread, owning one key, writes one
//    128-byte row).
//  * In S^T a thread owns one key and 32 rows, so a row's maximum lies across threads. The
//    running maximum is lazy: a block only votes whether some score exceeds its row's
//    reference by more than 2^20; the exact maxima (shuffles) and the rescale of O^T are
//    taken when one does, which the first block of an item always makes it do. p <= 2^20
//    keeps l and O (float32) far from overflow, and the result does not depend on the
//    reference. l is summed per key and reduced once an item.
//  * The (row tile, key block) pairs of the batch are cut into equal contiguous shares, one
//    CTA an SM; tiles cut by a share boundary leave normalised pieces that a second kernel
//    joins by log-sum-exp.
//  * A group of codes marked NaN is stored as zeros and its key flagged: the flag makes the
//    key's visible scores NaN, so a row that sees it becomes NaN and a row that does not
//    see it is untouched (0 * NaN never enters a product).
//  * Every wait is bounded; one that runs out records a status in the error word and the
//    kernel drains its MMAs, frees tensor memory and returns.
#include <math.h>

#include "kdt_internal.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace tc;

constexpr int kRowsT = kQ8Rows;                     // query rows of a tile (N)
constexpr int kKeysB = kQ8Keys;                     // keys of a block (M)
// Warps: 0 issues the MMAs (1-3 idle), 4-11 softmax, 12-19 converters. The launch gives each
// of the five warpgroups 96 registers a thread; they trade: 40 + 2 * 136 + 2 * 80 <= 5 * 96.
constexpr int kSoftWarps = 8, kConvWarps = 8, kSoft0 = 4, kConv0 = 12;
constexpr int kThreads = 32 * (kConv0 + kConvWarps);
constexpr int kRegsMma = 40, kRegsSoft = 136, kRegsConv = 80;
static_assert(kRegsMma + 2 * kRegsSoft + 2 * kRegsConv <= 5 * 96, "the warpgroups' shares exceed the launch's registers");
constexpr int kPairs = 4;                           // pairs of 64-dim tiles (128 latent dims each)
constexpr int kKTile = kKeysB * 128;                // [128 keys x 64 dims] bf16: 16 KB
constexpr int kQTile = kRowsT * 128;                // [64 rows x 64 dims] bf16: 8 KB
constexpr int kOffR = 8 * kKTile;                   // rope tile, then P^T
constexpr int kOffQ = kOffR + kKTile;               // nine Q tiles
constexpr int kSmem = kOffQ + 9 * kQTile + 1024;    // + alignment slack
constexpr uint32_t kColS = 256;                     // S^T columns; O^T tile q at 64 q
constexpr float kRaise = 20.f;                      // log2 units
constexpr uint64_t kWait = 200000000ull;            // ns
constexpr int kAhead = 2;                           // blocks the L2 prefetch runs ahead

struct Bars {
    uint64_t kfull[kPairs];     // a pair of latent tiles converted (8 warps)
    uint64_t kempty[kPairs];    // O^T's MMAs read it
    uint64_t rfull;             // rope tile stored (8 warps)
    uint64_t sfull;             // scores of the block in tensor memory
    uint64_t pfull;             // P^T stored, O^T rescaled if needed (8 warps)
    uint64_t pdone;             // the block's O^T complete, P^T's space free
    uint64_t qfull;             // Q tiles of the item stored (8 warps)
    uint64_t qempty;            // the item's last score MMAs ran
    uint64_t ofree;             // O^T of the item read out (8 warps)
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int work[4];                // this CTA's share: blocks, first sequence, tile, block
};

struct Shared {
    Bars bar;
    alignas(16) float m[kRowsT];   // read as float4
    alignas(16) float alpha[kRowsT];
    alignas(16) float inv[kRowsT];
    float red[4][kRowsT];       // per key quadrant
    uint32_t bad[2][kKeysB];    // keys with a NaN group, by block parity
};

__device__ __forceinline__ bool wait_for(Bars &bar, uint64_t *b, uint32_t parity, int32_t *err, int code) {
    if (*reinterpret_cast<volatile int *>(&bar.abort_flag)) return false;
    if (mbar_wait(b, parity, kWait)) return true;
    bar.abort_flag = 1;
    if (err) atomicCAS(err, 0, code);
    return false;
}

__device__ __forceinline__ bool warp_wait(Bars &bar, uint64_t *b, uint32_t parity, int32_t *err, int code) {
    return __all_sync(0xffffffffu, wait_for(bar, b, parity, err, code));
}

template <int kId, int kCount>
__device__ __forceinline__ bool barrier_or(bool flag) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pin, pout;\n\t"
        "setp.ne.u32 pin, %1, 0;\n\t"
        "bar.red.or.pred pout, %2, %3, pin;\n\t"
        "selp.u32 %0, 1, 0, pout;\n\t}"
        : "=r"(r)
        : "r"(flag ? 1u : 0u), "n"(kId), "n"(kCount)
        : "memory");
    return r != 0;
}

template <int kN> __device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN> __device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int blocks_of(const Q8Params &p, int b) {
    return (p.prefix_len[b] + p.T + kKeysB - 1) / kKeysB;
}

// The item a role is at: blocks [kb, kb + nb) of row tile rt of sequence b. The share's items
// follow in order; an item ends where its tile or the share does.
struct Item {
    int left;               // blocks of the share from this item on
    int b, rt, kb, nb;
    int P;                  // the sequence's prefix length
};

__device__ __forceinline__ bool fill(const Q8Params &p, Item &it) {
    if (it.left <= 0) return false;
    it.P = p.prefix_len[it.b];
    it.nb = min((it.P + p.T + kKeysB - 1) / kKeysB - it.kb, it.left);
    return true;
}

__device__ __forceinline__ bool advance(const Q8Params &p, Item &it) {
    it.left -= it.nb;
    it.kb = 0;
    if (++it.rt == p.tiles_seq) {
        it.rt = 0;
        ++it.b;
    }
    return fill(p, it);
}

// Positions: sequence-major, tile-major, block order; W of them. CTA c takes
// [W c / C, W (c + 1) / C). One warp finds its share's first item {left, b, rt, kb}.
__device__ __forceinline__ void find_share(const Q8Params &p, int64_t C, int64_t c, int lane, int *out) {
    int64_t W = 0;
    for (int b = lane; b < p.B; b += 32) W += (int64_t)p.tiles_seq * blocks_of(p, b);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
    const int64_t s0 = W * c / C, s1 = W * (c + 1) / C;
    if (lane == 0) {
        out[0] = (int)(s1 - s0);
        out[1] = out[2] = out[3] = 0;
    }
    __syncwarp();
    int64_t before = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        const int nb = b < p.B ? blocks_of(p, b) : 1;
        const int64_t w = b < p.B ? (int64_t)p.tiles_seq * nb : 0;
        int64_t incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const int64_t at = before + incl - w;
        const bool hit = s0 >= at && s0 < at + w;
        if (hit) {
            out[1] = b;
            out[2] = (int)((s0 - at) / nb);
            out[3] = (int)((s0 - at) % nb);
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (__any_sync(0xffffffffu, hit)) break;
    }
    __syncwarp();
}

// x[r] of 32 lanes reduced over the lanes for all 32 r at once: lane r gets row r's result.
// Step `off` exchanges the half of the array that the other lane keeps.
template <typename Op>
__device__ __forceinline__ float transpose_reduce(const float (&x)[32], int lane, Op op) {
    float v[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const bool up = lane & 16;
        const float send = up ? x[k] : x[k + 16], keep = up ? x[k + 16] : x[k];
        v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int k = 0; k < off; ++k) {
            const float send = up ? v[k] : v[k + off], keep = up ? v[k + off] : v[k];
            v[k] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
        }
    }
    return v[0];
}

__device__ __forceinline__ uint32_t lane_addr(uint32_t base, int warp, uint32_t col) {
    return base + ((uint32_t)(32 * (warp & 3)) << 16) + col;
}

template <bool kBf16Out>
__global__ void __launch_bounds__(kThreads, 1) verify_q8_rows_kernel(const Q8Params p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    Bars &bar = sh.bar;
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    if (warp == 4) find_share(p, gridDim.x, blockIdx.x, lane, bar.work);
    if (threadIdx.x == 32) {
        for (int i = 0; i < kPairs; ++i) {
            mbar_init(&bar.kfull[i], kConvWarps);
            mbar_init(&bar.kempty[i], 1);
        }
        mbar_init(&bar.rfull, kConvWarps);
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.pfull, kSoftWarps);
        mbar_init(&bar.pdone, 1);
        mbar_init(&bar.qfull, kConvWarps);
        mbar_init(&bar.qempty, 1);
        mbar_init(&bar.ofree, kSoftWarps);
        mbar_init(&bar.drain, 1);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x >= 256 && threadIdx.x < 512) sh.bad[(threadIdx.x >> 7) & 1][threadIdx.x & 127] = 0u;
    if (warp == 0) tmem_relinquish();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    Item it = {bar.work[0], bar.work[1], bar.work[2], bar.work[3], 0, 0};
    bool have = fill(p, it);
    uint32_t g = 0, ii = 0;                                  // blocks and items so far

    if (warp >= kSoft0 && warp < kSoft0 + kSoftWarps) {
        // ------------------------- softmax, correction and epilogue -------------------------
        // key = lane of S^T; half = which 32 rows of the tile; srow: one row a thread of the first 64
        regs_inc<kRegsSoft>();
        const int half = (warp - kSoft0) >> 2, key = 32 * (warp & 3) + lane;
        const int srow = (int)threadIdx.x - 32 * kSoft0;
        unsigned char *prow = smem + kOffR + key * 128;
        bool ok = true, vis_ready = false;
        for (; have; have = advance(p, it), ++ii) {
            const int row0 = it.rt * kRowsT + 32 * half;     // first of this warp's 32 rows
            float l[32];
#pragma unroll
            for (int r = 0; r < 32; ++r) l[r] = 0.f;
            if (srow < kRowsT) sh.m[srow] = -INFINITY;
            barrier_or<1, 256>(false);
            bool fail = false;
            for (int j = 0; j < it.nb; ++j, ++g) {
                ok = ok && warp_wait(bar, &bar.sfull, g & 1, p.err, -41);
                float x[32];
                bool raise = false;
                if (ok) {
                    tc_fence_after();
                    uint32_t raw[32];
                    tmem_ld32(lane_addr(tmem + kColS, warp, 32 * half), raw);
                    tmem_wait_ld();
                    tc_fence_before();
                    const int key0 = (it.kb + j) * kKeysB, kk = key0 + key;
#pragma unroll
                    for (int r = 0; r < 32; ++r) x[r] = __uint_as_float(raw[r]) * p.scale_log2;
                    if (sh.bad[g & 1][key]) {                // NaN wherever it is seen
#pragma unroll
                        for (int r = 0; r < 32; ++r) x[r] = __uint_as_float(0x7fffffffu);
                    }
                    if (key0 + kKeysB > it.P) {              // the block holds tree keys, or rows behind them
                        if (!vis_ready) {
                            griddep_wait();
                            vis_ready = true;
                        }
                        const int t = kk - it.P;             // this key's tree index
                        if (t >= p.T) {
#pragma unroll
                            for (int r = 0; r < 32; ++r) x[r] = -INFINITY;
                        } else if (t >= 0) {
                            int i = min(row0, p.rows_seq - 1) / p.H, left = p.H - (row0 - i * p.H);
                            const uint32_t *word = p.vis + ((int64_t)it.b * p.T + i) * p.W + (t >> 5);
                            uint32_t bits = __ldg(word);
#pragma unroll
                            for (int r = 0; r < 32; ++r) {
                                if (left == 0 && i + 1 < p.T) {
                                    ++i;
                                    left = p.H;
                                    word += p.W;
                                    bits = __ldg(word);
                                }
                                --left;
                                if (!((bits >> (t & 31)) & 1u)) x[r] = -INFINITY;
                            }
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 m4 = reinterpret_cast<const float4 *>(sh.m + 32 * half)[q];
                        raise |= x[4 * q] > m4.x + kRaise || x[4 * q + 1] > m4.y + kRaise || x[4 * q + 2] > m4.z + kRaise ||
                                 x[4 * q + 3] > m4.w + kRaise;
                    }
                }
                if (barrier_or<1, 256>(raise || !ok)) {
                    fail = barrier_or<1, 256>(!ok);
                    if (fail) break;
                    // some row's reference has to rise: the block's maxima, quadrant by quadrant
                    const float mx = transpose_reduce(x, lane, [](float a, float b) { return fmaxf(a, b); });
                    sh.red[warp & 3][32 * half + lane] = mx;
                    barrier_or<1, 256>(false);
                    if (srow < kRowsT) {
                        const int r = srow;
                        const float top = fmaxf(fmaxf(sh.red[0][r], sh.red[1][r]), fmaxf(sh.red[2][r], sh.red[3][r]));
                        const float m = sh.m[r];
                        float a = 1.f;
                        if (top > m + kRaise) {
                            a = m == -INFINITY ? 1.f : ex2(m - top);
                            sh.m[r] = top;
                        }
                        sh.alpha[r] = a;
                    }
                    barrier_or<1, 256>(false);
                    if (j > 0) {                             // O^T and l of the blocks before
                        ok = warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -42);
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < kPairs; ++q) {
                                uint32_t o[32];
                                const uint32_t addr = lane_addr(tmem, warp, kRowsT * q + 32 * half);
                                tmem_ld32(addr, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int r = 0; r < 32; ++r)
                                    o[r] = __float_as_uint(__uint_as_float(o[r]) * sh.alpha[32 * half + r]);
                                tmem_st32(addr, o);
                            }
                            tmem_wait_st();
                            tc_fence_before();
                        }
#pragma unroll
                        for (int r = 0; r < 32; ++r) l[r] *= sh.alpha[32 * half + r];
                    }
                }
                if (ok) {
                    sh.bad[g & 1][key] = 0u;                 // (both halves write the same)
                    // p = 2^(x - m) to this key's row of P^T; a row with no visible key yet has m = -inf
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t o[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float2 m2 = reinterpret_cast<const float2 *>(sh.m + 32 * half)[4 * u + v];
                            const int r = 8 * u + 2 * v;
                            const float p0 = m2.x == -INFINITY ? x[r] + INFINITY : ex2(x[r] - m2.x);
                            const float p1 = m2.y == -INFINITY ? x[r + 1] + INFINITY : ex2(x[r + 1] - m2.y);
                            // (x = -inf there, or NaN: a hidden key's NaN never gets here)
                            const float q0 = m2.x == -INFINITY && x[r] == -INFINITY ? 0.f : p0;
                            const float q1 = m2.y == -INFINITY && x[r + 1] == -INFINITY ? 0.f : p1;
                            l[r] += q0;
                            l[r + 1] += q1;
                            o[v] = q8::pack_bf16(q0, q1);
                        }
                        *reinterpret_cast<uint4 *>(prow + (((4 * half + u) ^ (key & 7)) << 4)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.pfull);
                }
            }
            if (fail) break;
            // l over the keys, then out = O / l and lse = ln2 (m + log2 l)
            const float ls = transpose_reduce(l, lane, [](float a, float b) { return a + b; });
            sh.red[warp & 3][32 * half + lane] = ls;
            ok = ok && warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -43);
            if (barrier_or<1, 256>(!ok)) break;
            // all blocks of the tile: final rows; else a piece, in slot 2c for the share's first item
            const bool whole = it.kb == 0 && it.nb == (it.P + p.T + kKeysB - 1) / kKeysB;
            const int64_t first = whole ? (int64_t)it.b * p.rows_seq + it.rt * kRowsT
                                        : (2 * (int64_t)blockIdx.x + (ii ? 1 : 0)) * kRowsT;
            if (srow < kRowsT) {
                const int r = srow;
                const float lt = sh.red[0][r] + sh.red[1][r] + sh.red[2][r] + sh.red[3][r];
                sh.inv[r] = lt == 0.f ? 0.f : 1.f / lt;
                float *lse = whole ? p.lse : p.part_lse;
                if (lse && it.rt * kRowsT + r < p.rows_seq)
                    lse[first + r] = lt == 0.f ? -INFINITY : 0.6931471805599453f * (sh.m[r] + log2f(lt));
            }
            barrier_or<1, 256>(false);
            tc_fence_after();
            const int rows = min(32, p.rows_seq - row0);     // of this warp's 32 (may be <= 0)
#pragma unroll 1
            for (int q = 0; q < kPairs; ++q) {
                uint32_t o[32];
                tmem_ld32(lane_addr(tmem, warp, kRowsT * q + 32 * half), o);
                tmem_wait_ld();
                const int64_t at = (first + 32 * half) * kDc + 128 * q + key;
                if (whole && kBf16Out) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at;
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        if (r < rows) dst[r * kDc] = __float2bfloat16_rn(__uint_as_float(o[r]) * sh.inv[32 * half + r]);
                } else {
                    float *dst = (whole ? static_cast<float *>(p.out) : p.part_o) + at;
#pragma unroll
                    for (int r = 0; r < 32; ++r)
                        if (r < rows) dst[r * kDc] = __uint_as_float(o[r]) * sh.inv[32 * half + r];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ofree);
        }
    } else if (warp >= kConv0) {
        // --------------------------------- converters ---------------------------------
        // A step is 128 keys x 128 bytes: one pair of latent tiles (codes), or the rope tile. Warp
        // cw takes keys 16 cw .. + 16, four at a time: 8 lanes a key, 16 bytes a lane.
        regs_dec<kRegsConv>();
        const int cw = warp - kConv0, sub = lane & 7, kq = lane >> 3;
        struct Regs {
            uint4 v[4];
            uint32_t s[4];
        };
        bool ok = true;
        Regs cur;
        auto load = [&](int j, int step, Regs &x) {
            const int kv = it.P + p.T, key0 = (it.kb + j) * kKeysB + 16 * cw + kq;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int kk = key0 + 4 * t;
                x.v[t] = make_uint4(0u, 0u, 0u, 0u);
                x.s[t] = 127u;
                if (kk < kv) {
                    const int64_t row = (int64_t)it.b * p.L + kk;
                    if (step < kPairs) {
                        x.v[t] = __ldg(reinterpret_cast<const uint4 *>(p.c_q8 + row * kDc) + 8 * step + sub);
                        x.s[t] = __ldg(p.c_scale + row * (kDc / KDT_Q8_GROUP) + 4 * step + (sub >> 1));
                    } else {
                        x.v[t] = __ldg(reinterpret_cast<const uint4 *>(p.k_pe + row * kDr) + sub);
                    }
                }
            }
        };
        if (have) load(0, 0, cur);
        while (have && ok) {
            // the item's rows of Q: warp cw takes rows 8 cw .. + 8
            ok = ii == 0 || warp_wait(bar, &bar.qempty, (ii - 1) & 1, p.err, -44);
            if (!ok) break;
            {
                const int r0 = 8 * cw, R0 = it.rt * kRowsT + r0;
                const int64_t base = (int64_t)it.b * p.rows_seq + R0;
#pragma unroll 2
                for (int r = 0; r < 8; ++r) {
                    const bool live = R0 + r < p.rows_seq;
                    const uint4 *src = reinterpret_cast<const uint4 *>(p.q_nope + (base + r) * p.q_nope_stride);
                    unsigned char *dst = smem + kOffQ + (r0 + r) * 128;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = 32 * h + lane;         // 16-byte chunk of the row's 64
                        const uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(dst + (c >> 3) * kQTile + (((c & 7) ^ ((r0 + r) & 7)) << 4)) = v;
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 4 * h + kq;
                    const bool live = R0 + r < p.rows_seq;
                    const uint4 v = live ? __ldg(reinterpret_cast<const uint4 *>(p.q_pe + (base + r) * p.q_pe_stride) + sub)
                                         : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(smem + kOffQ + 8 * kQTile + (r0 + r) * 128 + ((sub ^ ((r0 + r) & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.qfull);
            }
            const int nb = it.nb;
            for (int j = 0; j < nb && ok; ++j, ++g) {
#pragma unroll
                for (int step = 0; step <= kPairs; ++step) {
                    Regs nxt;
                    if (step < kPairs) {
                        load(j, step + 1, nxt);
                    } else if (j + 1 < nb) {
                        load(j + 1, 0, nxt);
                    } else if ((have = advance(p, it))) {
                        load(0, 0, nxt);
                    }
                    // the tile's space: read by O^T's MMAs of the block before
                    if (g > 0) {
                        uint64_t *b = step < kPairs ? &bar.kempty[step] : &bar.pdone;
                        if (!(ok = warp_wait(bar, b, (g - 1) & 1, p.err, step < kPairs ? -45 : -46))) break;
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int kr = 16 * cw + 4 * t + kq;     // key of the block
                        if (step < kPairs) {
                            if (cur.s[t] == (uint32_t)q8::kNaN) sh.bad[g & 1][kr] = 1u;
                            uint4 lo, hi;
                            q8::widen16(cur.v[t], cur.s[t], lo, hi);
                            // chunks 2 (sub % 4) and + 1 of tile sub / 4; the lanes of the second tile
                            // store theirs in the other order, so that eight lanes cover all banks
                            unsigned char *dst = smem + (2 * step + (sub >> 2)) * kKTile + kr * 128;
                            const int c0 = 2 * (sub & 3), sw = kr & 7, second = sub >> 2;
                            *reinterpret_cast<uint4 *>(dst + (((c0 + second) ^ sw) << 4)) = second ? hi : lo;
                            *reinterpret_cast<uint4 *>(dst + (((c0 + 1 - second) ^ sw) << 4)) = second ? lo : hi;
                        } else {
                            *reinterpret_cast<uint4 *>(smem + kOffR + kr * 128 + ((sub ^ (kr & 7)) << 4)) = cur.v[t];
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(step < kPairs ? &bar.kfull[step] : &bar.rfull);
                    cur = nxt;
                }
            }
            ++ii;
        }
    } else {
        regs_dec<kRegsMma>();
        if (warp == 0 && elect_one()) {
        // -------------------------------- MMA issuer --------------------------------
        const uint32_t id_s = idesc_bf16_f32(kKeysB, kRowsT, 0, 0), id_o = idesc_bf16_f32(kKeysB, kRowsT, 1, 1);
        // Descriptors differ only in their low words (address and leading stride); each use adds a
        // constant to a base the compiler cannot see through, or it would keep all of them live.
        const uint64_t d0 = sdesc_sw128(0, 0, 1024);
        const uint32_t dhi = (uint32_t)(d0 >> 32);
        const uint32_t base = smem_u32(smem) >> 4, lbo_k = (16u >> 4) << 16, lbo_mn = ((uint32_t)kKTile >> 4) << 16;
        auto desc = [&](uint32_t lo) { return ((uint64_t)dhi << 32) | lo; };
        auto opaque = [](uint32_t v) {
            asm volatile("" : "+r"(v));
            return v;
        };
        // warms L2 kAhead blocks ahead of the one whose scores are issued
        Item pf = it;
        int pj = 0;
        bool pmore = have;
        auto prefetch = [&]() {
            if (!pmore) return;
            const int key0 = (pf.kb + pj) * kKeysB, n = min(kKeysB, pf.P + p.T - key0);
            const int64_t row = (int64_t)pf.b * p.L + key0;
            prefetch_l2_bulk(p.c_q8 + row * kDc, (uint32_t)n * kDc);
            prefetch_l2_bulk(p.c_scale + row * (kDc / KDT_Q8_GROUP), (uint32_t)n * (kDc / KDT_Q8_GROUP));
            prefetch_l2_bulk(p.k_pe + row * kDr, (uint32_t)n * kDr * 2);
            if (++pj == pf.nb) {
                pj = 0;
                pmore = advance(p, pf);
            }
        };
        for (int k = 0; k < kAhead; ++k) prefetch();
        bool ok = true;
        for (; ok && have; have = advance(p, it), ++ii) {
            if (!(ok = wait_for(bar, &bar.qfull, ii & 1, p.err, -47))) break;
            for (int j = 0; j < it.nb && ok; ++j, ++g) {
#pragma unroll 1
                for (int c = 0; c < kPairs; ++c) {
                    if (!(ok = wait_for(bar, &bar.kfull[c], g & 1, p.err, -48))) break;
                    tc_fence_after();
                    const uint32_t kd = opaque(base + lbo_k + 2 * c * (kKTile >> 4));
                    const uint32_t qd = opaque(base + lbo_k + (kOffQ >> 4) + 2 * c * (kQTile >> 4));
#pragma unroll
                    for (int t = 0; t < 8; ++t)              // tile 2c + t / 4, 16 dims each
                        mma_ss(tmem + kColS, desc(kd + (((t >> 2) * kKTile + (t & 3) * 32) >> 4)),
                               desc(qd + (((t >> 2) * kQTile + (t & 3) * 32) >> 4)), id_s, (c > 0 || t > 0) ? 1u : 0u);
                }
                if (!ok || !(ok = wait_for(bar, &bar.rfull, g & 1, p.err, -49))) break;
                tc_fence_after();
                const uint32_t rd = opaque(base + lbo_k + (kOffR >> 4));
                const uint32_t qr = opaque(base + lbo_k + ((kOffQ + 8 * kQTile) >> 4));
#pragma unroll
                for (int t = 0; t < 4; ++t) mma_ss(tmem + kColS, desc(rd + 2 * t), desc(qr + 2 * t), id_s, 1u);
                mma_commit(&bar.sfull);
                prefetch();
                if (j == it.nb - 1) mma_commit(&bar.qempty);
                if (!(ok = wait_for(bar, &bar.pfull, g & 1, p.err, -50))) break;
                // the item before: its O^T has been read out
                if (j == 0 && ii > 0 && !(ok = wait_for(bar, &bar.ofree, (ii - 1) & 1, p.err, -51))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < kPairs; ++c) {
                    const uint32_t vd = opaque(base + lbo_mn + 2 * c * (kKTile >> 4));
                    const uint32_t pd = opaque(base + lbo_mn + (kOffR >> 4));
#pragma unroll
                    for (int t = 0; t < 8; ++t)              // 16 keys each
                        mma_ss(tmem + kRowsT * c, desc(vd + (t * 2048 >> 4)), desc(pd + (t * 2048 >> 4)), id_o,
                               (j > 0 || t > 0) ? 1u : 0u);
                    mma_commit(&bar.kempty[c]);
                }
                mma_commit(&bar.pdone);
            }
        }
        mma_commit(&bar.drain);                              // every MMA done before tensor memory goes
        mbar_wait(&bar.drain, 0, kWait);
        }
        __syncwarp();
    }
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the tiles that a share boundary cut: CTA (tile, y) takes rows 8 y ..
// + 8, a warp a row. The tile spans positions [t0, t1), the shares meeting it are c_a .. c_b
// (one: it was written whole), each with a normalised state (o, lse): o = sum_k e^(lse_k -
// M) o_k / sum_k e^(lse_k - M). A NaN in a piece's lse reaches the row.
template <bool kBf16Out>
__global__ void __launch_bounds__(256) merge_q8_rows_kernel(const Q8Params p) {
    griddep_wait();
    const int tile = blockIdx.x, b = tile / p.tiles_seq, rt = tile % p.tiles_seq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t C = p.ctas;
    int64_t tot = 0, bef = 0;
    for (int k = lane; k < p.B; k += 32) {
        const int64_t w = (int64_t)p.tiles_seq * blocks_of(p, k);
        tot += w;
        if (k < b) bef += w;
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        tot += __shfl_xor_sync(0xffffffffu, tot, off);
        bef += __shfl_xor_sync(0xffffffffu, bef, off);
    }
    const int64_t W = tot;
    const int nblk = blocks_of(p, b);
    const int64_t t0 = bef + (int64_t)rt * nblk, t1 = t0 + nblk;
    const int64_t ca = ((t0 + 1) * C - 1) / W, cb = (t1 * C - 1) / W;      // shares of positions t0 and t1 - 1
    if (ca == cb) return;
    const int row = blockIdx.y * 8 + warp, r = rt * kRowsT + row;
    if (r >= p.rows_seq) return;
    // share c's slot: 2c when the share starts at or after t0 (the tile is its first item), else 2c + 1
    auto slot = [&](int64_t c) -> int64_t {
        const int64_t s = W * c / C;
        return c > cb || s == W * (c + 1) / C ? -1 : (s >= t0 ? 2 * c : 2 * c + 1);
    };
    float M = -INFINITY;
    bool nan = false;
    for (int64_t base = ca; base <= cb; base += 32) {
        const int64_t sl = slot(base + lane);
        const float v = sl >= 0 ? p.part_lse[sl * kRowsT + row] : -INFINITY;
        nan |= v != v;
        M = fmaxf(M, v);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __any_sync(0xffffffffu, nan);
    float4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    float S = nan ? __uint_as_float(0x7fffffffu) : 0.f;
    if (M > -INFINITY)
        for (int64_t base = ca; base <= cb; base += 32) {
            const int64_t sl = slot(base + lane);
            const float v = sl >= 0 ? p.part_lse[sl * kRowsT + row] : -INFINITY;
            const float wt = v == -INFINITY ? 0.f : __expf(v - M);
            float ws = wt;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
            S += ws;
            const int cnt = (int)min((int64_t)32, cb - base + 1);
#pragma unroll 4
            for (int k = 0; k < cnt; ++k) {
                const float wk = __shfl_sync(0xffffffffu, wt, k);
                const int64_t sk = __shfl_sync(0xffffffffu, sl, k);
                if (sk < 0 || wk == 0.f) continue;           // the same for the whole warp
                const float4 *src = reinterpret_cast<const float4 *>(p.part_o + (sk * kRowsT + row) * kDc) + lane;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v4 = src[32 * q];
                    acc[q].x = fmaf(wk, v4.x, acc[q].x);
                    acc[q].y = fmaf(wk, v4.y, acc[q].y);
                    acc[q].z = fmaf(wk, v4.z, acc[q].z);
                    acc[q].w = fmaf(wk, v4.w, acc[q].w);
                }
            }
        }
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const int64_t grow = (int64_t)b * p.rows_seq + r;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 v = make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv);
        if (kBf16Out)
            reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + grow * kDc)[32 * q + lane] =
                make_uint2(q8::pack_bf16(v.x, v.y), q8::pack_bf16(v.z, v.w));
        else
            reinterpret_cast<float4 *>(static_cast<float *>(p.out) + grow * kDc)[32 * q + lane] = v;
    }
    if (lane == 0 && p.lse) p.lse[grow] = S == 0.f ? -INFINITY : M + logf(S);
}

template <bool kBf16Out> cudaError_t launch(const Q8Params &p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(verify_q8_rows_kernel<kBf16Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // starts while the visibility kernel of the same call runs, and waits for it before it
    // reads the bits; the merge starts at this kernel's end
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = p.overlap_vis ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, verify_q8_rows_kernel<kBf16Out>, p)) != cudaSuccess) return e;
    if (p.ctas > 1) {
        cudaLaunchConfig_t mc = {};
        mc.gridDim = dim3((unsigned)((int64_t)p.B * p.tiles_seq), kRowsT / 8);
        mc.blockDim = dim3(256);
        mc.stream = s;
        mc.attrs = pdl;
        mc.numAttrs = 1;
        e = cudaLaunchKernelEx(&mc, merge_q8_rows_kernel<kBf16Out>, p);
    }
    return e;
}

}  // namespace

cudaError_t launch_verify_q8_rows(const Q8Params &p, cudaStream_t s) {
    return p.out_bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace kdt
