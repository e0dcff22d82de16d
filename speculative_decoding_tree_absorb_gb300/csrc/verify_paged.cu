// K6: tree-verify attention over a paged bf16 latent cache (single tokens, small trees): tcgen05 with the
// KEYS on the M side.
//
// The definition is kdt_verify_attn's, key j of a sequence read from the page its table names: scores s_j =
// scale (q_nope . c_j + q_pe . k_j) of a row over its visible keys, softmax, out = sum p_j c_j, lse.
//
//  * A tile is up to 64 query rows (heads x tree nodes) of one sequence, 16 or 32 when it has no more. The
//    tensor cores are filled from the keys' side: S^T = K Q^T with M = 64 keys, N = rows, and O^T = V^T P^T
//    with M = 128 latent dims (four accumulators), N = rows. O^T takes 4 N of tensor memory's 512 columns and
//    S^T 2 N, so that a block's scores are made while the one before is in its softmax.
//  * A block is 64 keys: 576 dims as nine 128-byte swizzled tiles, the latent in four stages of two tiles.
//    ONE copy serves both contractions: K-major A operand of S^T, MN-major A operand of O^T. TMA boxes of
//    min(64, page) rows bring it, a box a page where pages are smaller; the stages form a ring of two blocks
//    or more, and each is given back as soon as its part of O^T is done. Boxes behind the last row, and pages
//    that are none, lie outside the tensor map: zeros, no traffic.
//  * One warp issues the scores' MMAs and another the output's, so that neither a late page holds up O^T, which
//    frees the ring, nor softmax the scores. The whole warp walks the loop and waits in step, and one lane
//    issues: descriptors computed by a lone thread, which polled for both kinds of work, took 75 - 100 cycles an
//    MMA where the MMAs take 31 (scores) and 47 (output): 4.3 k cycles a block, now 2.6 k.
//  * What bounds a block (64 rows, 64 keys) in a CTA alone: the operands of 36 + 16 MMAs pass shared memory at
//    128 bytes a cycle, 1.9 k cycles, and the ring of two blocks makes every second block wait for the chain
//    load - scores - softmax - output, 5.2 k: 2.6 k a block. With all 152 at work and nothing in L2 2.8 - 3.3 k;
//    DRAM would give each its own block every 3.1 k. Copies ahead into L2 (by TMA, by a warp of their own or by
//    the loading warp, two to six blocks) made every case 1 - 30 % slower, and two buffers for P^T with one for
//    the rope keys 2 %. Boxes of 16 rows (pages of 16) pass the copy engine at 5 cycles a row: 3.9 k a block.
//  * In S^T a thread owns two keys and a few rows, so a row's maximum lies across threads. The running
//    maximum is lazy: a block only votes whether some score exceeds its row's reference by more than 2^20;
//    exact maxima and the rescale of O^T are taken when one does, and for the first block of an item. p <=
//    2^20 keeps l and O (float32) far from overflow, and the result does not depend on the reference. Sums
//    stay with the threads until the item's end.
//  * Row tiles of a sequence (a "group" of up to 8) walk the same keys side by side, a CTA each, so that DRAM
//    is read once and the others hit L2. The (group, key block) pairs of the batch are cut into equal
//    contiguous shares; groups cut by a share's end leave normalised pieces that a second kernel joins by
//    log-sum-exp.
//  * Measured, both kernels (bf16 out, pages not in L2): 64 single tokens of 64 heads over 1024 - 8192 keys 84 us,
//    351 MB of cache at 4.2 TB/s, of which 8 us pass before the first scores (lengths, then the page table, then
//    the first pages, none of them in L2) and 10 us join 38 MB of pieces; two of 128 heads over 60001 and 99990
//    keys 72 us; eight trees of 13 nodes of 32 heads over 2500 - 12000 keys in pages of 16 99 us; one token of
//    16 heads over 700 14 us. Many rows a sequence: eight trees of 64 nodes of 64 heads over 8192 keys 621 us,
//    0.94 PFLOP/s; the contiguous cache's kernel, whose clusters share a block's keys among 256 rows, takes 420.
//  * Masks, rows of other sequences' leftovers behind the last key, and latents that are not finite concern
//    the blocks with tree keys only: there the softmax warps zero what may not enter a product (0 * NaN), and
//    mark its key, whose score is NaN for the rows that see it.
//  * Every wait is bounded; one that runs out records a status in the error word and the kernel drains its
//    MMAs, frees tensor memory and returns.
#include <cuda.h>
#include <float.h>
#include <math.h>
#include <string.h>

#include "kdt_internal.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace tc;

constexpr int kKeysB = kPagedKeys;                  // keys of a block (M of S^T)
// Warps: 0 loads keys, 1 issues the scores' MMAs, 2 loads queries, 3 issues the output's MMAs, 4-11 softmax.
constexpr int kSoft0 = 4, kSoftWarps = 8, kSoftThreads = 32 * kSoftWarps;
constexpr int kThreads = 32 * (kSoft0 + kSoftWarps);
constexpr int kStages = 4;                          // of a block's latent
constexpr int kTileBytes = kKeysB * 128;            // [64 keys x 64 dims] bf16
constexpr int kStageBytes = 2 * kTileBytes;
constexpr uint32_t kColS = 256;                     // S^T columns (two buffers of N); O^T part q at N q
constexpr float kRaise = 20.f;                      // log2 units
// Minus the reference of a row that has seen no score yet but -inf: large enough that any other score votes
// for a rise, and finite, so that -inf stays -inf, of weight 0.
constexpr float kNoReference = FLT_MAX;
constexpr uint64_t kWait = 200000000ull;            // ns

template <int kRows> struct Layout {
    static constexpr int kRing = kRows == 64 ? 8 : (kRows == 32 ? 10 : 11);         // latent stages
    static constexpr int kRopeRing = kRows == 64 ? 2 : 3;
    static constexpr int kQTile = kRows * 128;      // [rows x 64 dims] bf16
    static constexpr int kOffR = kRing * kStageBytes;
    static constexpr int kOffQ = kOffR + kRopeRing * kTileBytes;
    static constexpr int kOffP = kOffQ + 9 * kQTile;
    static constexpr int kSmem = kOffP + kRows * 128 + 1024;                        // + alignment slack
};

struct Bars {
    uint64_t kfull[11], kempty[11];     // a stage landed; O^T's MMAs have read it
    uint64_t rfull[3], rempty[3];       // rope keys
    uint64_t sfull[2];                  // scores of the block in tensor memory
    uint64_t sempty[2];                 // and read out of it
    uint64_t pfull;                     // P^T stored, O^T rescaled if needed
    uint64_t pdone;                     // the block's O^T complete, P^T's space free
    uint64_t qfull, qempty;             // queries of the item landed; its scores are all made
    uint64_t ofree;                     // O^T of the item read out
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int work[6];                        // this share: blocks; its first item: sequence, group, block, nodes, prefix
};

template <int kRows> struct Shared {
    Bars bar;
    alignas(16) float m[kRows];         // the reference, log2 units
    alignas(16) float alpha[kRows];     // of a rise; at an item's end 1 / l
    float red[4][kRows];                // by keys' quarter
    uint32_t bad[2];                    // keys whose latent is not finite
    uint32_t up[32];                    // a short tree's nodes and their ancestors
};

__device__ __forceinline__ bool wait_for(Bars &bar, uint64_t *b, uint32_t parity, int32_t *err, int code) {
    uint64_t t0 = 0;
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(b, parity)) return true;
        if (*reinterpret_cast<volatile int *>(&bar.abort_flag)) return false;
        const uint64_t now = global_ns();
        if (!t0) t0 = now;
        if (now - t0 > kWait) break;
    }
    bar.abort_flag = 1;
    if (err) atomicCAS(err, 0, code);
    return false;
}

// By a whole warp, all of it in step: a loop that lanes may leave one by one costs 100 cycles a wait, and a
// block's chain has a dozen of them. What comes after the first try is a call: inlined in every place, it took the
// roles' loops out of the instruction caches (eight trees of 64 nodes of 64 heads over 8192 keys 660 us, 621 so).
__device__ __noinline__ bool wait_on(Bars &bar, uint64_t *b, uint32_t parity, int32_t *err, int code) {
    uint64_t t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
        const uint64_t now = global_ns();
        if (!t0) t0 = now;
        const bool late = __any_sync(0xffffffffu, now - t0 > kWait) != 0;
        if (late && (threadIdx.x & 31) == 0) {
            bar.abort_flag = 1;
            if (err) atomicCAS(err, 0, code);
        }
        if (late || __any_sync(0xffffffffu, *reinterpret_cast<volatile int *>(&bar.abort_flag) != 0)) return false;
    }
}

__device__ __forceinline__ bool warp_wait(Bars &bar, uint64_t *b, uint32_t parity, int32_t *err, int code) {
    if (__all_sync(0xffffffffu, mbar_try_wait(b, parity))) return true;
    return wait_on(bar, b, parity, err, code);
}

__device__ __forceinline__ bool soft_or(bool flag) {       // over the softmax warps
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred pin, pout;\n\t"
        "setp.ne.u32 pin, %1, 0;\n\t"
        "bar.red.or.pred pout, 1, %2, pin;\n\t"
        "selp.u32 %0, 1, 0, pout;\n\t}"
        : "=r"(r)
        : "r"(flag ? 1u : 0u), "n"(kSoftThreads)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Tree nodes and prefix of sequence b, brought into the caller's bounds.
__device__ __forceinline__ int nodes_of(const PagedParams &p, int b) {
    return p.n_rows ? min(max(p.n_rows[b], 0), p.T) : p.T;
}
__device__ __forceinline__ int prefix_of(const PagedParams &p, int b, int n) {
    return min(max(p.prefix_len[b], 0), p.max_kv - n);
}
__device__ __forceinline__ int groups_of(const PagedParams &p, int n) {
    return (n * p.H + p.tile * p.group - 1) / (p.tile * p.group);
}

// The item a role is at: blocks [kb, kb + nb) of group grp of sequence b. The share's items follow in order;
// an item ends where its group or the share does.
struct Item {
    int left;               // blocks of the share from this item on
    int b, grp, kb, nb;
    int n, P, kv;           // nodes, prefix, keys of the sequence
    int idx;                // items of the share before this one
};

__device__ __forceinline__ bool fill(const PagedParams &p, Item &it) {
    if (it.left <= 0) return false;
    while (it.b < p.B && (it.n = nodes_of(p, it.b)) == 0) ++it.b;
    if (it.b >= p.B) return false;
    it.P = prefix_of(p, it.b, it.n);
    it.kv = it.P + it.n;
    it.nb = min((it.kv + kKeysB - 1) / kKeysB - it.kb, it.left);
    return true;
}

__device__ __forceinline__ bool advance(const PagedParams &p, Item &it) {
    it.left -= it.nb;
    it.kb = 0;
    ++it.idx;
    if (++it.grp >= groups_of(p, it.n)) {
        it.grp = 0;
        ++it.b;
    }
    return fill(p, it);
}

__device__ __forceinline__ bool first_item(const PagedParams &p, const int *work, Item &it) {
    it.left = work[0];
    it.b = work[1];
    it.grp = work[2];
    it.kb = work[3];
    it.n = work[4];
    it.P = work[5];
    it.kv = it.P + it.n;
    it.nb = min((it.kv + kKeysB - 1) / kKeysB - it.kb, it.left);
    it.idx = 0;
    return it.left > 0;
}

// The row tile of this CTA (g-th of the group), or -1 when the sequence has none there.
__device__ __forceinline__ int tile_of(const PagedParams &p, const Item &it, int g) {
    const int rt = it.grp * p.group + g;
    return rt * p.tile < it.n * p.H ? rt : -1;
}

// a / b for 0 <= a, 0 < b < 2^31: a 64-bit division costs hundreds of cycles of a kernel's start.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return a >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Positions: sequence-major, group-major, block order; W of them in G groups, cut into up to p.shares equal
// shares: one a group, or more of p.least blocks or more.
struct Shares {
    int64_t W, each;
    int C, more;                                              // the first `more` shares have a block more
    __device__ __forceinline__ Shares(const PagedParams &p, int64_t w, int64_t G) : W(w) {
        C = (int)min((int64_t)p.shares, max(max(quotient(W + p.least - 1, p.least), G), (int64_t)1));
        each = quotient(W, C);
        more = (int)(W - each * C);
    }
    __device__ __forceinline__ int64_t start(int c) const { return c < C ? each * c + min(c, more) : W; }
    __device__ __forceinline__ int of(int64_t at) const {     // the share that has position `at` < W
        const int64_t longer = more * (each + 1);
        return (int)(at < longer ? quotient(at, each + 1) : more + quotient(at - longer, each));
    }
};

// One warp finds share c's first item. Where share c is the first to begin inside a group, it leaves that
// group's rows and the number of its pieces for the merge.
__device__ __forceinline__ void find_share(const PagedParams &p, int c, bool writes, int lane, int *out) {
    int64_t W = 0, G = 0;
    for (int b = lane; b < p.B; b += 32) {
        const int n = nodes_of(p, b);
        if (n) {
            G += groups_of(p, n);
            W += (int64_t)groups_of(p, n) * ((prefix_of(p, b, n) + n + kKeysB - 1) / kKeysB);
        }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        W += __shfl_xor_sync(0xffffffffu, W, off);
        G += __shfl_xor_sync(0xffffffffu, G, off);
    }
    const Shares shares(p, W, G);
    const int64_t s0 = shares.start(c), s1 = shares.start(c + 1);
    if (lane == 0) {
        out[0] = (int)(s1 - s0);
        out[1] = out[2] = out[3] = out[4] = out[5] = 0;
        if (writes) p.cuts[c].pieces = 0;                     // unless share c is the first to begin inside a group
    }
    __syncwarp();
    int64_t before = 0;
    for (int base = 0; base < p.B && s0 < s1; base += 32) {
        const int b = base + lane;
        const int n = b < p.B ? nodes_of(p, b) : 0;
        const int P = n ? prefix_of(p, b, n) : 0, nb = n ? (P + n + kKeysB - 1) / kKeysB : 1;
        const int64_t w = n ? (int64_t)groups_of(p, n) * nb : 0;
        int64_t incl = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += y;
        }
        const int64_t at = before + incl - w;
        const bool hit = s0 >= at && s0 < at + w;
        if (hit) {
            const int grp = (int)quotient(s0 - at, nb);
            out[1] = b;
            out[2] = grp;
            out[3] = (int)(s0 - at - (int64_t)grp * nb);
            out[4] = n;
            out[5] = P;
            const int64_t t0 = at + (int64_t)grp * nb;        // where the group begins, and the share before
            const int64_t before_it = c > 0 ? shares.start(c - 1) : s0;
            if (writes && s0 > t0 && before_it <= t0) {
                const int row = grp * p.group * p.tile;
                p.cuts[c].row0 = (int64_t)b * p.rows_seq + row;
                p.cuts[c].rows = min(n * p.H - row, p.group * p.tile);
                p.cuts[c].second = before_it < t0 ? 1 : 0;
                p.cuts[c].pieces = shares.of(t0 + nb - 1) - c + 2;
            }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (__any_sync(0xffffffffu, hit)) break;
    }
    __syncwarp();
}

// A value that all lanes of a warp have, known to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory descriptors differ in their low words only: address and leading stride in 16 bytes.
constexpr uint32_t kLeadK = 1u << 16, kLeadMn = (uint32_t)(kTileBytes >> 4) << 16;
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return (sdesc_sw128(0, 0, 1024) >> 32 << 32) | lo; }

// By a warp: the words of a short tree's nodes, as the visibility kernel makes them. (A call: inlined, its code
// costs the loop around it 1 %.)
__device__ __noinline__ void walk_tree(const int32_t *parent, int32_t *err, int b, int T, int lane, uint32_t *up) {
    const int32_t par = lane < T ? __ldg(parent + (int64_t)b * T + lane) : -1;
    uint32_t acc = 1u << lane;
    int at = lane;
    bool walks = lane < T;
    while (__any_sync(0xffffffffu, walks)) {
        const int32_t next = __shfl_sync(0xffffffffu, par, at);
        if (walks && (next < -1 || next >= at)) {            // malformed: the walk stops here
            record_error(err, (int32_t)((int64_t)b * T + at + 1));
            walks = false;
        }
        walks = walks && next >= 0;
        if (walks) {
            at = next;
            acc |= 1u << at;
        }
    }
    up[lane] = acc;
}

__device__ __forceinline__ uint32_t lane_addr(uint32_t base, int warp, uint32_t col) {
    return base + ((uint32_t)(32 * (warp & 3)) << 16) + col;
}

template <int kRows, bool kBf16Out>
__global__ void __launch_bounds__(kThreads, 1)
    verify_paged_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_qn, const __grid_constant__ CUtensorMap map_qp, const PagedParams p) {
    using L = Layout<kRows>;
    constexpr int kHalf = kRows / 2;                // rows of a softmax warpgroup
    constexpr int kCols = kHalf / 8;                // groups of 8 of them
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared<kRows> sh;
    Bars &bar = sh.bar;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = blockIdx.x / p.group, g_of = blockIdx.x % p.group;

    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    if (warp == 4) find_share(p, share, p.pieces && g_of == 0, lane, bar.work);
    if (threadIdx.x == 32) {
        for (int i = 0; i < L::kRing; ++i) {
            mbar_init(&bar.kfull[i], 1);
            mbar_init(&bar.kempty[i], 1);
        }
        for (int i = 0; i < L::kRopeRing; ++i) {
            mbar_init(&bar.rfull[i], 1);
            mbar_init(&bar.rempty[i], 1);
        }
        mbar_init(&bar.sfull[0], 1);
        mbar_init(&bar.sfull[1], 1);
        mbar_init(&bar.sempty[0], kSoftWarps);
        mbar_init(&bar.sempty[1], kSoftWarps);
        mbar_init(&bar.pfull, kSoftWarps);
        mbar_init(&bar.pdone, 1);
        mbar_init(&bar.qfull, 1);
        mbar_init(&bar.qempty, 1);
        mbar_init(&bar.ofree, kSoftWarps);
        mbar_init(&bar.drain, 2);
        bar.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&map_c);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_qn);
        tma_prefetch_desc(&map_qp);
    }
    if (warp == 0) tmem_relinquish();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    if (warp >= kSoft0) {
        // ------------------------- softmax, correction and epilogue -------------------------
        // A warp has 16 keys of S^T and half of the rows: this thread keys ka and ka + 8, rows row_of(i, e).
        Item it;
        bool have = first_item(p, bar.work, it);
        uint32_t g = 0;                                      // blocks so far
        const int w4 = warp & 3, half = (warp - kSoft0) >> 2, ka = 16 * w4 + (lane >> 2);
        const int srow = (int)threadIdx.x - 32 * kSoft0;
        const float scale = p.scale_log2;
        bool ok = true, vis_ready = false;
        auto row_of = [&](int i, int e) { return kHalf * half + 8 * i + 2 * (lane & 3) + e; };
        // where this lane's 16 bytes of stmatrix go: matrix 2 i + (keys + 8), row r of it
        const int mrow = lane & 7, mhalf = (lane >> 3) & 1, mi = (lane >> 4) & 1;
        const uint32_t pdst = smem + L::kOffP + (kHalf * half + mrow) * 128 + (((2 * w4 + mhalf) ^ mrow) << 4);
        for (; have; have = advance(p, it)) {
            const int rt = tile_of(p, it, g_of);
            if (rt < 0) continue;
            float l[2 * kCols], nm[2 * kCols];
#pragma unroll
            for (int k = 0; k < 2 * kCols; ++k) l[k] = 0.f;
            if (srow < kRows) sh.m[srow] = -INFINITY;        // (read by others behind the first block's barriers)
            if (p.parent && (it.kb + it.nb) * kKeysB > it.P) {   // the item has tree keys
                if (warp == kSoft0) walk_tree(p.parent, p.err, it.b, p.T, lane, sh.up);
                soft_or(false);
            }
            bool fail = false;
            for (int j = 0; j < it.nb; ++j, ++g) {
                const int key0 = (it.kb + j) * kKeysB;
                const bool masked = key0 + kKeysB > it.P;
                // bit 2 k + h: row k of this thread's sees key ka + 8 h
                uint32_t see = ~0u;
                if (masked) {
                    see = 0u;
                    const int ta = key0 + ka - it.P;
                    if (p.vis && !vis_ready) {
                        griddep_wait();
                        vis_ready = true;
                    }
#pragma unroll
                    for (int k = 0; k < 2 * kCols; ++k) {
                        const int node = (rt * kRows + row_of(k >> 1, k & 1)) / p.H;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int t = ta + 8 * h;
                            bool v = t < 0;
                            if (t >= 0 && t < it.n && node < it.n) {
                                if (p.parent) v = (sh.up[node] >> t) & 1u;
                                else v = !p.vis || ((__ldcg(p.vis + ((int64_t)it.b * p.T + node) * p.W + (t >> 5)) >> (t & 31)) & 1u);
                            }
                            see |= (v ? 1u : 0u) << (2 * k + h);
                        }
                    }
                }
                ok = ok && warp_wait(bar, &bar.sfull[g & 1], (g >> 1) & 1, p.err, -61);
                tc_fence_after();
                uint32_t is_bad = 0u;
                if (masked) {
                    // rows behind the last key are zeroed, and, where nodes hide keys, what is not finite
                    const uint32_t u0 = kStages * g;
                    for (int c = 0; c < kStages; ++c)        // (long since: this thread's view of what landed)
                        ok = ok && warp_wait(bar, &bar.kfull[(u0 + c) % L::kRing], ((u0 + c) / L::kRing) & 1, p.err, -62);
                    auto at = [&](int r, int x) {            // 16-byte chunk x of 64 of key row r
                        return smem + ((u0 + (x >> 4)) % L::kRing) * kStageBytes + ((x >> 3) & 1) * kTileBytes + r * 128 + ((x & 7) << 4);
                    };
                    const int first = min(it.kv - key0, kKeysB);
                    for (int x = srow; x < (kKeysB - first) * 64; x += kSoftThreads) st_shared_v4(at(first + (x >> 6), x & 63), 0u, 0u, 0u, 0u);
                    if (p.vis || p.parent) {
                        if (srow < 2) sh.bad[srow] = 0u;
                        soft_or(false);
                        const int from = max(it.P - key0, 0);
                        for (int x = srow; x < (first - from) * 64; x += kSoftThreads) {
                            const int r = from + (x >> 6);
                            uint32_t v[4];
                            ld_shared_v4(at(r, x & 63), v);
                            bool inf = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                inf |= (v[k] & 0x7f800000u) == 0x7f800000u || (v[k] & 0x7f80u) == 0x7f80u;
                            if (inf) {
                                st_shared_v4(at(r, x & 63), 0u, 0u, 0u, 0u);
                                atomicOr(&sh.bad[r >> 5], 1u << (r & 31));
                            }
                        }
                        soft_or(false);
                        is_bad = ((sh.bad[ka >> 5] >> (ka & 31)) & 1u) | (((sh.bad[(ka + 8) >> 5] >> ((ka + 8) & 31)) & 1u) << 1);
                    }
                }
                uint32_t raw[4 * kCols];
                tmem_ld_frag(lane_addr(tmem + kColS + (g & 1) * kRows, warp, kHalf * half), raw);
                loaded(raw);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sempty[g & 1]);
                float x[4 * kCols];                          // [i][key][e]
                auto scores = [&](bool shifted) {
#pragma unroll
                    for (int k = 0; k < 4 * kCols; ++k)
                        x[k] = fmaf(__uint_as_float(raw[k]), scale, shifted ? nm[2 * (k >> 2) + (k & 1)] : 0.f);
                    if (masked) {
#pragma unroll
                        for (int k = 0; k < 4 * kCols; ++k) {
                            const int r = 2 * (k >> 2) + (k & 1), h = (k >> 1) & 1;
                            if ((is_bad >> h) & 1u) x[k] = __uint_as_float(0x7fffffffu);
                            x[k] = (see >> (2 * r + h)) & 1u ? x[k] : -INFINITY;
                        }
                    }
                };
                bool rise = j == 0;                          // (no reference yet)
                if (j > 0) {
                    scores(true);
                    float top = x[0];
#pragma unroll
                    for (int k = 1; k < 4 * kCols; ++k) top = fmaxf(top, x[k]);
                    rise = soft_or(top > kRaise || !ok);
                }
                if (rise) {
                    scores(false);
#pragma unroll
                    for (int k = 0; k < 2 * kCols; ++k) {
                        float v = fmaxf(x[4 * (k >> 1) + (k & 1)], x[4 * (k >> 1) + 2 + (k & 1)]);
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                        if (lane < 4) sh.red[w4][row_of(k >> 1, k & 1)] = v;
                    }
                    // O^T of the block before is complete
                    if (j > 0) ok = ok && warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -63);
                    if ((fail = soft_or(!ok))) break;
                    if (srow < kRows) {
                        const float to = fmaxf(fmaxf(sh.red[0][srow], sh.red[1][srow]), fmaxf(sh.red[2][srow], sh.red[3][srow]));
                        const float m = sh.m[srow];
                        float a = 1.f;
                        if (to > m + kRaise) {
                            a = m == -INFINITY ? 1.f : ex2(m - to);
                            sh.m[srow] = to;
                        }
                        sh.alpha[srow] = a;
                    }
                    soft_or(false);
                    if (j > 0) {
#pragma unroll 1
                        for (int q = 0; q < 4 * kCols; ++q) {
                            const int col = kHalf * half + 8 * (q % kCols);
                            const uint32_t addr = lane_addr(tmem, warp, kRows * (q / kCols) + col);
                            uint32_t o[8];
                            tc_fence_after();
                            tmem_ld8(addr, o);
                            loaded(o);
#pragma unroll
                            for (int r = 0; r < 8; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * sh.alpha[col + r]);
                            tmem_st8(addr, o);
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int k = 0; k < 2 * kCols; ++k) l[k] *= sh.alpha[row_of(k >> 1, k & 1)];
                    }
#pragma unroll
                    for (int k = 0; k < 2 * kCols; ++k) {
                        const float m = sh.m[row_of(k >> 1, k & 1)];
                        nm[k] = m == -INFINITY ? kNoReference : -m;
                    }
                    scores(true);
                }
                // p = 2^(score - m), to P^T's place once O^T's MMAs of the block before have read it
                uint32_t pk[2 * kCols];                      // [i][key]
#pragma unroll
                for (int k = 0; k < 2 * kCols; ++k) {
                    x[2 * k] = ex2(x[2 * k]);
                    x[2 * k + 1] = ex2(x[2 * k + 1]);
                    pk[k] = q8::pack_bf16(x[2 * k], x[2 * k + 1]);
                }
                if (g > 0) ok = ok && warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -64);
                tc_fence_before();
                if constexpr (kCols == 1) {
                    stmatrix_trans(pdst, pk);                // (two matrices: lanes 0 - 15 give the addresses)
                } else {
#pragma unroll
                    for (int i = 0; i < kCols; i += 2) {
                        const uint32_t four[4] = {pk[2 * i], pk[2 * i + 1], pk[2 * i + 2], pk[2 * i + 3]};
                        stmatrix_trans(pdst + (i + mi) * 1024, four);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pfull);
#pragma unroll
                for (int k = 0; k < 2 * kCols; ++k) l[k] += x[4 * (k >> 1) + (k & 1)] + x[4 * (k >> 1) + 2 + (k & 1)];
            }
            if (fail) break;
            // l over the keys, then out = O / l and lse = ln2 (m + log2 l)
#pragma unroll
            for (int k = 0; k < 2 * kCols; ++k) {
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
                if (lane < 4) sh.red[w4][row_of(k >> 1, k & 1)] = l[k];
            }
            ok = ok && warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -65);
            if (soft_or(!ok)) break;
            // all blocks of the group: final rows; else a piece, in slot 2 x for the share's first item
            const bool whole = it.kb == 0 && it.nb == (it.kv + kKeysB - 1) / kKeysB;
            const int live = min(kRows, it.n * p.H - rt * kRows);
            const int64_t first = whole ? (int64_t)it.b * p.rows_seq + rt * kRows
                                        : (2 * (int64_t)blockIdx.x + (it.idx ? 1 : 0)) * kRows;
            if (srow < kRows) {
                const float lt = sh.red[0][srow] + sh.red[1][srow] + sh.red[2][srow] + sh.red[3][srow];
                sh.alpha[srow] = lt == 0.f ? 0.f : 1.f / lt;
                float *lse = whole ? p.lse : p.part_lse;
                if (lse && srow < live) lse[first + srow] = lt == 0.f ? -INFINITY : 0.6931471805599453f * (sh.m[srow] + log2f(lt));
            }
            soft_or(false);
            tc_fence_after();
            // A thread has one dim of kHalf rows. Float32: a warp stores 128 bytes of a row at once. bf16: of two
            // rows, lanes in pairs trade a dim of one for the other's dim of the other.
            const int rows = min(max(live - kHalf * half, 0), kHalf);
            const int64_t at = (first + kHalf * half) * kDc + 32 * w4;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t raw[kCols][8];
                float o[kHalf];
#pragma unroll
                for (int k = 0; k < kCols; ++k) tmem_ld8(lane_addr(tmem, warp, kRows * q + kHalf * half + 8 * k), raw[k]);
#pragma unroll
                for (int k = 0; k < kCols; ++k) loaded(raw[k]);
#pragma unroll
                for (int r = 0; r < kHalf; ++r) o[r] = __uint_as_float(raw[r >> 3][r & 7]) * sh.alpha[kHalf * half + r];
                if (whole && kBf16Out) {
                    const int odd = lane & 1;
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at + 128 * q + (int64_t)odd * kDc + (lane & ~1);
#pragma unroll
                    for (int r = 0; r < kHalf; r += 2) {
                        const float mine = odd ? o[r + 1] : o[r];
                        const float other = __shfl_xor_sync(0xffffffffu, odd ? o[r] : o[r + 1], 1);
                        if (r + odd < rows)
                            *reinterpret_cast<uint32_t *>(dst + (int64_t)r * kDc) = q8::pack_bf16(odd ? other : mine, odd ? mine : other);
                    }
                } else {
                    float *dst = (whole ? static_cast<float *>(p.out) : p.part_o) + at + 128 * q + lane;
#pragma unroll
                    for (int r = 0; r < kHalf; ++r)
                        if (r < rows) dst[(int64_t)r * kDc] = o[r];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ofree);
        }
    } else if (warp == 0) {
        // ------------------------------------ keys ------------------------------------
        // Lane k has the cache row of the block's k-th box (of min(64, page) rows); one lane issues all copies.
        const int box = min(kKeysB, 1 << p.shift), boxes = kKeysB / box;
        const int nowhere = p.n_pages << p.shift;            // a row outside the tensor maps
        auto place = [&](const Item &i, int j) {
            const int key = (i.kb + j) * kKeysB + lane * box;
            if (lane >= boxes || key >= i.kv) return nowhere;
            const int32_t page = __ldg(p.table + i.b * p.table_stride + (key >> p.shift));
            if (page >= 0 && page < p.n_pages) return (page << p.shift) + (key & ((1 << p.shift) - 1));
            record_error(p.err, (int32_t)min((int64_t)INT32_MAX, 1 + (int64_t)p.B * p.T + i.b));
            return nowhere;
        };
        const bool lead = elect_one();
        Item it;
        bool ok = true;
        uint32_t slot = 0, phase = 1, rslot = 0, rphase = 1;
        for (bool have = first_item(p, bar.work, it); have && ok; have = advance(p, it)) {
            if (tile_of(p, it, g_of) < 0) continue;
            int next = place(it, 0);
            for (int j = 0; j < it.nb; ++j) {
                const int rows = next;
                if (j + 1 < it.nb) next = place(it, j + 1);
                if (!(ok = warp_wait(bar, &bar.rempty[rslot], rphase, p.err, -66))) break;
                if (lead) mbar_arrive_expect_tx(&bar.rfull[rslot], kTileBytes);
                int row[kKeysB / 8];
#pragma unroll
                for (int k = 0; k < kKeysB / 8; ++k) {
                    if (k >= boxes) break;
                    row[k] = __shfl_sync(0xffffffffu, rows, k);
                    if (lead) tma_load_2d_at(smem + L::kOffR + rslot * kTileBytes + k * box * 128, &map_k, &bar.rfull[rslot], 0, row[k]);
                }
                if (++rslot == L::kRopeRing) {
                    rslot = 0;
                    rphase ^= 1;
                }
#pragma unroll 1
                for (int c = 0; c < kStages; ++c) {
                    if (!(ok = warp_wait(bar, &bar.kempty[slot], phase, p.err, -67))) break;
                    const uint32_t dst = smem + slot * kStageBytes;
                    if (lead) mbar_arrive_expect_tx(&bar.kfull[slot], kStageBytes);
                    if (boxes == 1) {                        // one box of both tiles
                        if (lead) tma_load_3d_at(dst, &map_c, &bar.kfull[slot], 0, row[0], 2 * c);
                    } else {                                 // a box a tile and page
#pragma unroll
                        for (int k = 0; k < kKeysB / 8; ++k) {
                            if (k >= boxes) break;
                            if (lead) {
                                tma_load_3d_at(dst + k * box * 128, &map_c, &bar.kfull[slot], 0, row[k], 2 * c);
                                tma_load_3d_at(dst + kTileBytes + k * box * 128, &map_c, &bar.kfull[slot], 0, row[k], 2 * c + 1);
                            }
                        }
                    }
                    if (++slot == L::kRing) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ----------------------------------- queries -----------------------------------
        if (elect_one()) {
            Item it;
            uint32_t ii = 0;
            for (bool have = first_item(p, bar.work, it); have; have = advance(p, it)) {
                const int rt = tile_of(p, it, g_of);
                if (rt < 0) continue;
                if (ii > 0 && !wait_for(bar, &bar.qempty, (ii - 1) & 1, p.err, -68)) break;
                const int row = it.b * p.rows_seq + rt * kRows;
                mbar_arrive_expect_tx(&bar.qfull, 9 * L::kQTile);
                tma_load_3d_at(smem + L::kOffQ, &map_qn, &bar.qfull, 0, row, 0);
                tma_load_2d_at(smem + L::kOffQ + 8 * L::kQTile, &map_qp, &bar.qfull, 0, row);
                ++ii;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------ scores ------------------------------------
        // The whole warp walks the loop, so that all it computes is uniform, and one lane issues.
        const bool lead = elect_one();
        const uint32_t id = idesc_bf16_f32(kKeysB, kRows, 0, 0), td = uniform(tmem) + kColS;
        const uint32_t base = (uniform(smem) >> 4) + kLeadK, qd = base + (L::kOffQ >> 4);
        Item it;
        uint32_t g = 0, ii = 0, slot = 0, phase = 0, rslot = 0, rphase = 0;
        bool ok = true;
        for (bool have = first_item(p, bar.work, it); have && ok; have = advance(p, it)) {
            if (tile_of(p, it, g_of) < 0) continue;
            if (!(ok = warp_wait(bar, &bar.qfull, ii & 1, p.err, -69))) break;
            const int nb = (int)uniform((uint32_t)it.nb);
            for (int j = 0; j < nb; ++j, ++g) {
                const uint32_t d = td + (g & 1) * kRows;
                if (g >= 2 && !(ok = warp_wait(bar, &bar.sempty[g & 1], ((g >> 1) - 1) & 1, p.err, -70))) break;
                if (!(ok = warp_wait(bar, &bar.rfull[rslot], rphase, p.err, -71))) break;
                tc_fence_after();
                const uint32_t rd = base + (L::kOffR >> 4) + rslot * (kTileBytes >> 4);
                if (lead) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) mma_ss(d, desc_of(rd + 2 * t), desc_of(qd + (8 * L::kQTile >> 4) + 2 * t), id, t > 0 ? 1u : 0u);
                    mma_commit(&bar.rempty[rslot]);
                }
                if (++rslot == L::kRopeRing) {
                    rslot = 0;
                    rphase ^= 1;
                }
#pragma unroll
                for (int c = 0; c < kStages; ++c) {
                    if (!(ok = warp_wait(bar, &bar.kfull[slot], phase, p.err, -72))) break;
                    tc_fence_after();
                    const uint32_t kd = base + slot * (kStageBytes >> 4);
                    if (lead) {
#pragma unroll
                        for (int t = 0; t < 8; ++t)          // tile 2 c + t / 4, 16 dims each
                            mma_ss(d, desc_of(kd + (((t >> 2) * kTileBytes + (t & 3) * 32) >> 4)),
                                   desc_of(qd + (((2 * c + (t >> 2)) * L::kQTile + (t & 3) * 32) >> 4)), id, 1u);
                        if (c == kStages - 1) mma_commit(&bar.sfull[g & 1]);
                    }
                    if (++slot == L::kRing) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
            }
            if (lead) mma_commit(&bar.qempty);
            ++ii;
        }
        if (lead) {
            mma_commit(&bar.drain);                          // every MMA done before tensor memory goes
            mbar_wait(&bar.drain, 0, kWait);
        }
        __syncwarp();
    } else {
        // ------------------------------------ output ------------------------------------
        const bool lead = elect_one();
        const uint32_t id = idesc_bf16_f32(128, kRows, 1, 0), td = uniform(tmem);
        const uint32_t base = uniform(smem) >> 4, pd = base + kLeadK + (L::kOffP >> 4);
        Item it;
        uint32_t g = 0, ii = 0, slot = 0;
        bool ok = true;
        for (bool have = first_item(p, bar.work, it); have && ok; have = advance(p, it)) {
            if (tile_of(p, it, g_of) < 0) continue;
            if (ii > 0 && !(ok = warp_wait(bar, &bar.ofree, (ii - 1) & 1, p.err, -73))) break;
            const int nb = (int)uniform((uint32_t)it.nb);
            for (int j = 0; j < nb; ++j, ++g) {
                if (!(ok = warp_wait(bar, &bar.pfull, g & 1, p.err, -74))) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kStages; ++c) {
                    const uint32_t vd = base + kLeadMn + slot * (kStageBytes >> 4);
                    if (lead) {
#pragma unroll
                        for (int t = 0; t < 4; ++t)          // 16 keys each
                            mma_ss(td + kRows * c, desc_of(vd + (t * 2048 >> 4)), desc_of(pd + 2 * t), id, t > 0 || j > 0 ? 1u : 0u);
                        mma_commit(&bar.kempty[slot]);
                    }
                    if (++slot == L::kRing) slot = 0;
                }
                if (lead) mma_commit(&bar.pdone);
            }
            ++ii;
        }
        if (lead) {
            mma_commit(&bar.drain);
            mbar_wait(&bar.drain, 0, kWait);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (*reinterpret_cast<volatile int *>(&bar.abort_flag)) {   // error path only: loads in flight land before the CTA leaves
        const uint64_t t0 = global_ns();
        do __nanosleep(1000);
        while (global_ns() - t0 < 200000ull);
    }
    // What follows on the stream waits for this kernel alone: it must not end before the one that finds the words, not
    // even where it read none of them (a padded batch without nodes).
    if (p.overlap_vis && threadIdx.x == 0) griddep_wait();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the pieces of the groups that a share's end cut, four warps a row (128 columns each). A NaN in a
// piece's lse reaches the row.
// A group that is cut is served where share c begins inside it and is the first to: CTA (c - 1, two rows).
// Where a group has many pieces (kSplit = 4), four times four warps take them in turn, and CTA (x, a row) looks
// for the x-th such share itself: most shares are none, and a CTA for each would cost more than the search.
template <int kSplit> struct Join {
    static constexpr int kRows = kSplit == 1 ? 2 : 1, kWarps = 4 * kSplit * kRows;
};
template <bool kBf16Out, int kSplit>
__global__ void __launch_bounds__(32 * Join<kSplit>::kWarps) merge_paged_rows_kernel(const PagedParams p) {
    constexpr int kWarps = Join<kSplit>::kWarps, kRows = Join<kSplit>::kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int c = blockIdx.x + 1;
    if constexpr (kSplit > 1) {
        __shared__ int counts[kWarps], cut;
        if (threadIdx.x == 0) cut = 0;
        for (int base = 1, seen = 0; base < p.shares; base += 32 * kWarps) {
            const int i = base + (int)threadIdx.x;
            const bool is = i < p.shares && p.cuts[i].pieces > 0;
            const uint32_t all = __ballot_sync(0xffffffffu, is);
            if (lane == 0) counts[warp] = __popc(all);
            __syncthreads();
            int rank = seen + __popc(all & ((1u << lane) - 1u));
            for (int w = 0; w < kWarps; ++w) {
                rank += w < warp ? counts[w] : 0;
                seen += counts[w];
            }
            if (is && rank == (int)blockIdx.x) cut = i;
            __syncthreads();
        }
        if ((c = cut) == 0) return;                           // fewer groups are cut
    }
    const PagedShare sh = p.cuts[c];
    const int part = warp / (4 * kRows), grow = blockIdx.y * kRows + (warp >> 2) % kRows;
    if (sh.pieces == 0 || grow >= sh.rows) return;            // (all warps of a row)
    const int g = grow / p.tile, row = grow % p.tile, col = 128 * (warp & 3) + 4 * lane;
    // piece k's place: share c - 1 + k's slot 2, but of share c - 1 the second item's where it did not begin here
    auto at = [&](int k) { return (int64_t)(2 * ((c - 1 + k) * p.group + g) + (k == 0 ? sh.second : 0)) * p.tile + row; };
    float M = -INFINITY;
    bool nan = false;
    for (int k = lane; k < sh.pieces; k += 32) {
        const float v = p.part_lse[at(k)];
        nan |= v != v;
        M = fmaxf(M, v);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __any_sync(0xffffffffu, nan);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float S = nan ? __uint_as_float(0x7fffffffu) : 0.f;
    if (M > -INFINITY)
        for (int base = 0; base < sh.pieces; base += 32) {
            const float v = base + lane < sh.pieces ? p.part_lse[at(base + lane)] : -INFINITY;
            const float wt = v == -INFINITY ? 0.f : __expf(v - M);
            float ws = wt;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
            S += ws;
            // the pieces that count (weight 0: no visible key), their loads independent
            uint32_t live = __ballot_sync(0xffffffffu, wt != 0.f && (kSplit == 1 || lane % kSplit == part));
            while (live) {
                float4 a[4];
                float wk[4];
                int n = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    wk[u] = 0.f;
                    if (!live) continue;                      // (uniform)
                    const int k = __ffs(live) - 1;
                    live &= live - 1;
                    wk[u] = __shfl_sync(0xffffffffu, wt, k);
                    a[u] = *reinterpret_cast<const float4 *>(p.part_o + at(base + k) * kDc + col);
                    n = u + 1;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u >= n) break;
                    acc = make_float4(fmaf(wk[u], a[u].x, acc.x), fmaf(wk[u], a[u].y, acc.y), fmaf(wk[u], a[u].z, acc.z),
                                      fmaf(wk[u], a[u].w, acc.w));
                }
            }
        }
    if constexpr (kSplit > 1) {
        __shared__ float4 sums[kSplit - 1][128];
        const int x = threadIdx.x & 127;
        if (part > 0) sums[part - 1][x] = acc;
        __syncthreads();
        if (part > 0) return;
#pragma unroll
        for (int k = 0; k < kSplit - 1; ++k)
            acc = make_float4(acc.x + sums[k][x].x, acc.y + sums[k][x].y, acc.z + sums[k][x].z, acc.w + sums[k][x].w);
    }
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const int64_t out = sh.row0 + grow;
    const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (kBf16Out)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + out * kDc + col) =
            make_uint2(q8::pack_bf16(v.x, v.y), q8::pack_bf16(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + out * kDc + col) = v;
    if (col == 0 && p.lse) p.lse[out] = S == 0.f ? -INFINITY : M + logf(S);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<EncodeTiledFn>(ptr);
    }
    return fn;
}

// Rows of 64 * blocks bf16 values, `stride` elements apart, as [blocks][rows][64]: a box lands as tiles of 128-byte
// swizzled rows.
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t stride, int blocks, int box_rows, int box_blocks) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)blocks};
    const cuuint64_t strides[2] = {(cuuint64_t)stride * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_blocks}, es[3] = {1, 1, 1};
    memset(m, 0, sizeof(*m));
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, blocks > 1 ? 3 : 2, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kRows, bool kBf16Out> cudaError_t launch(const PagedParams &p, cudaStream_t s) {
    using L = Layout<kRows>;
    const int64_t rows = (int64_t)p.B * p.rows_seq, slots = (int64_t)p.n_pages << p.shift;
    const int box = 1 << p.shift < kKeysB ? 1 << p.shift : kKeysB;
    CUtensorMap map_c, map_k, map_qn, map_qp;
    if (!make_map(&map_c, p.c_kv, slots, kDc, kDc / 64, box, box == kKeysB ? 2 : 1) || !make_map(&map_k, p.k_pe, slots, kDr, 1, box, 1) ||
        !make_map(&map_qn, p.q_nope, rows, p.q_nope_stride, kDc / 64, kRows, kDc / 64) ||
        !make_map(&map_qp, p.q_pe, rows, p.q_pe_stride, 1, kRows, 1))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(verify_paged_kernel<kRows, kBf16Out>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    // starts while the visibility kernel of the same call runs, and waits for it before it reads the bits
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.shares * p.group));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kSmem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = p.overlap_vis ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, verify_paged_kernel<kRows, kBf16Out>, map_c, map_k, map_qn, map_qp, p)) != cudaSuccess) return e;
    if (p.pieces) {
        const unsigned rows = (unsigned)(p.group * p.tile);
        if (p.deep)
            merge_paged_rows_kernel<kBf16Out, 4><<<dim3((unsigned)p.deep, rows), 32 * Join<4>::kWarps, 0, s>>>(p);
        else
            merge_paged_rows_kernel<kBf16Out, 1><<<dim3((unsigned)(p.shares - 1), rows / Join<1>::kRows), 32 * Join<1>::kWarps, 0, s>>>(p);
        e = cudaGetLastError();
    }
    return e;
}

template <int kRows> cudaError_t launch_rows(const PagedParams &p, cudaStream_t s) {
    return p.out_bf16 ? launch<kRows, true>(p, s) : launch<kRows, false>(p, s);
}

}  // namespace

cudaError_t launch_verify_paged(const PagedParams &p, cudaStream_t s) {
    return p.tile == 16 ? launch_rows<16>(p, s) : (p.tile == 32 ? launch_rows<32>(p, s) : launch_rows<64>(p, s));
}

}  // namespace kdt
