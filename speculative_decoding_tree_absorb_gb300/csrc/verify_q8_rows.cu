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
//    reference.
//  * The (row tile, key block) pairs of the batch are cut into equal contiguous shares, one
//    CTA an SM; tiles cut by a share boundary leave normalised pieces that a second kernel
//    joins by log-sum-exp.
//  * A group of codes marked NaN is stored as zeros and its key flagged: the flag makes the
//    key's visible scores NaN, so a row that sees it becomes NaN and a row that does not
//    see it is untouched (0 * NaN never enters a product).
//  * What bounds it: 64 rows a tile make the MMAs read shared memory for the whole of their
//    time (4 KB of A and 2 KB of B for 48 clocks each), and there is room for one block of
//    128 keys, so its stages follow one another: O^T's MMAs 1.7 k clocks, the last pair's
//    widening 2.5-3 k (its stores share shared memory with those MMAs), the last scores
//    0.6 k, softmax 1.2 k, hand-offs: 7.5 k clocks (3.9 us) a block. Measured: 64 single
//    tokens of 64 heads over 1-8 k keys 92 us (196 MB of cache: 2.1 TB/s, tensor pipe 23%);
//    3 sequences of 13 nodes and 16 heads over 5-32 k keys 70 us.
//  * Every wait is bounded; one that runs out records a status in the error word and the
//    kernel drains its MMAs, frees tensor memory and returns.
#include <float.h>
#include <math.h>

#include "kdt_internal.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace tc;

constexpr int kRowsT = kQ8Rows;                     // query rows of a tile (N)
constexpr int kKeysB = kQ8Keys;                     // keys of a block (M)
// Warps: 0 issues the MMAs, 1-3 copy the rope keys, 4-11 softmax, 12-27 converters (four for each
// pair of tiles). The launch gives each of the seven warpgroups 72 registers a thread; they trade.
constexpr int kSoftWarps = 8, kConvWarps = 16, kRopeWarps = 3, kSoft0 = 4, kConv0 = 12;
constexpr int kThreads = 32 * (kConv0 + kConvWarps);
constexpr int kRegsLaunch = 72, kRegsMma = 40, kRegsSoft = 120, kRegsConv = 56;
static_assert(kRegsMma + 2 * kRegsSoft + 4 * kRegsConv <= 7 * kRegsLaunch, "the warpgroups' shares exceed the launch's registers");
constexpr int kPairs = 4;                           // pairs of 64-dim tiles (128 latent dims each)
constexpr int kKTile = kKeysB * 128;                // [128 keys x 64 dims] bf16: 16 KB
constexpr int kQTile = kRowsT * 128;                // [64 rows x 64 dims] bf16: 8 KB
constexpr int kOffR = 8 * kKTile;                   // rope tile, then P^T
constexpr int kOffQ = kOffR + kKTile;               // nine Q tiles
constexpr int kSmem = kOffQ + 9 * kQTile + 1024;    // + alignment slack
constexpr uint32_t kColS = 256;                     // S^T columns; O^T tile q at 64 q
constexpr float kRaise = 20.f;                      // log2 units
// Minus the reference of a row that has seen no score yet but -inf: large enough that any other score
// votes for a rise (but one of -FLT_MAX itself), and finite, so that -inf stays -inf, of weight 0.
constexpr float kNoReference = FLT_MAX;
constexpr uint64_t kWait = 200000000ull;            // ns
constexpr int kAhead = 3;                           // blocks the L2 prefetch runs ahead

struct Bars {
    uint64_t kfull[kPairs];     // a pair of latent tiles converted 
    uint64_t kempty[kPairs];    // O^T's MMAs read it
    uint64_t rfull;             // rope tile stored (rope warps)
    uint64_t sfull;             // scores of the block in tensor memory
    uint64_t pfull;             // P^T stored, O^T rescaled if needed 
    uint64_t pdone;             // the block's O^T complete, P^T's space free
    uint64_t qfull;             // Q tiles of the item stored 
    uint64_t ofree;             // O^T of the item read out 
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    int work[4];                // this CTA's share: blocks, first sequence, tile, block
};

// One warp's part of an item's outputs on its way out: 32 dims of 8 rows in bf16, of 4 in float32.
union Stage {
    __nv_bfloat16 h[8][32];
    float f[4][32];
    uint4 all[32];
};

// Visibility words of a block's tree keys: up to 64 nodes (those of the tile's rows, from node i0
// on), kVisWords words each from word w0 on (128 keys touch at most five).
constexpr int kVisWords = 5;

struct Shared {
    Bars bar;
    alignas(16) float nm[kRowsT];   // minus the reference (read as float4)
    alignas(16) float zero[kRowsT];
    alignas(16) float m[kRowsT];    // the reference, log2 units
    alignas(16) float alpha[kRowsT];
    alignas(16) float inv[kRowsT];
    float red[4][kRowsT];       // per key quadrant
    uint32_t bad[2][kKeysB];    // keys with a NaN group, by block parity
    uint32_t vis[kRowsT * kVisWords];
    Stage stage[kSoftWarps];
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

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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

template <int kN> __device__ __forceinline__ void set_regs() {
    if constexpr (kN > kRegsLaunch) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
    if constexpr (kN < kRegsLaunch) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}

// 16 bytes to a shared-memory address (32-bit addressing: the tiles' offsets stay immediates).
__device__ __forceinline__ void sts(uint32_t addr, const uint4 &v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 16 bytes (the first `bytes` of them copied, the others zero) from global to shared memory.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
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
// [W c / C, W (c + 1) / C). One warp finds its share's first item {left, b, rt, kb}, and leaves for the
// merge where the share starts and which tile that is in.
__device__ __forceinline__ void find_share(const Q8Params &p, int64_t C, int64_t c, int lane, int *out) {
    int64_t W = 0;
    for (int b = lane; b < p.B; b += 32) W += (int64_t)p.tiles_seq * blocks_of(p, b);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) W += __shfl_xor_sync(0xffffffffu, W, off);
    const int64_t s0 = W * c / C, s1 = W * (c + 1) / C;
    if (lane == 0) {
        out[0] = (int)(s1 - s0);
        out[1] = out[2] = out[3] = 0;
        if (p.pieces) {
            p.shares[c].start = s0;
            p.shares[c].t0 = p.shares[c].t1 = s0;             // (an empty share behind the last position)
            if (c == C - 1) p.shares[C].start = W;
        }
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
            const int rt = (int)((s0 - at) / nb);
            out[1] = b;
            out[2] = rt;
            out[3] = (int)(s0 - at - (int64_t)rt * nb);
            if (p.pieces) {
                p.shares[c].t0 = at + (int64_t)rt * nb;
                p.shares[c].t1 = p.shares[c].t0 + nb;
                p.shares[c].row0 = (int64_t)b * p.rows_seq + (int64_t)rt * kRowsT;
                p.shares[c].rows = min(kRowsT, p.rows_seq - rt * kRowsT);
            }
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (__any_sync(0xffffffffu, hit)) break;
    }
    __syncwarp();
}

// Which of the 32 rows from row0 on see tree key t (t < 0: a prefix key, all of them; t >= T:
// behind the tree, none): bit r for row row0 + r, whose query is node (row0 + r) / H. Rows at or
// beyond rows_seq get any value.
__device__ __forceinline__ uint32_t seen_by(const Q8Params &p, const uint32_t *words, int i0, int w0, int t, int row0) {
    if (t < 0) return ~0u;
    if (t >= p.T) return 0u;
    uint32_t see = 0u;
    int i = row0 / p.H, left = p.H - (row0 - i * p.H);
    const uint32_t *word = words + (i - i0) * kVisWords + (t >> 5) - w0;
    for (int r = 0; r < 32 && i < p.T; ++i, word += kVisWords) {     // one node at a time: `left` rows of it
        const int n = min(left, 32 - r);
        if ((*word >> (t & 31)) & 1u) see |= (0xffffffffu >> (32 - n)) << r;
        r += n;
        left = p.H;
    }
    return see;
}

// Warms L2 with the queries of the item behind this one: they come from DRAM else, and their loads stand
// between two items (43 sequences of 2688 rows over 3 keys: 131 -> 109 us).
__device__ __forceinline__ void prefetch_next_q(const Q8Params &p, const Item &it) {
    if (it.left <= it.nb || p.q_nope_stride > 2 * kDc || p.q_pe_stride > 2 * kDc) return;   // (rows far apart: left alone)
    const bool wrap = it.rt + 1 == p.tiles_seq;
    const int rt = wrap ? 0 : it.rt + 1, live = min(kRowsT, p.rows_seq - rt * kRowsT);
    const int64_t row = (int64_t)(it.b + wrap) * p.rows_seq + rt * kRowsT;
    const __nv_bfloat16 *q = p.q_nope + row * p.q_nope_stride;
    for (int r = 0; r < live; r += 16) {
        const int n = min(16, live - r) - 1;
        prefetch_l2_bulk(q + r * p.q_nope_stride, (uint32_t)(n * p.q_nope_stride + kDc) * 2);
    }
    prefetch_l2_bulk(p.q_pe + row * p.q_pe_stride, (uint32_t)((live - 1) * p.q_pe_stride + kDr) * 2);
}

// One warp finds the words of a tree of at most 32 nodes (one word a node) from its parents, lane i
// node i's. It saves the launch of the visibility kernel (a short tree: 36 -> 31 us a call). A malformed
// entry ends its walks and is recorded, as there.
__device__ __forceinline__ uint32_t walk_tree(const Q8Params &p, int b, int lane) {
    const int par = lane < p.T ? __ldg(p.parent + (int64_t)b * p.T + lane) : -1;
    uint32_t m = 0u;
    int at = lane;
    bool on = lane < p.T;
    while (__any_sync(0xffffffffu, on)) {
        const int up = __shfl_sync(0xffffffffu, par, at);
        if (on) {
            m |= 1u << at;
            if (up < -1 || up >= at) record_error(p.err, (int32_t)((int64_t)b * p.T + at + 1));
            on = up >= 0 && up < at;
            at = on ? up : at;
        }
    }
    return m;
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
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0) tmem_alloc(&bar.tmem, 512);
    if (warp == 4) find_share(p, gridDim.x, blockIdx.x, lane, bar.work);
    if (threadIdx.x == 32) {
        for (int i = 0; i < kPairs; ++i) {
            mbar_init(&bar.kfull[i], kConvWarps / kPairs);
            mbar_init(&bar.kempty[i], 1);
        }
        mbar_init(&bar.rfull, kRopeWarps);
        mbar_init(&bar.sfull, 1);
        mbar_init(&bar.pfull, kSoftWarps);
        mbar_init(&bar.pdone, 1);
        mbar_init(&bar.qfull, kSoftWarps);
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

    if (warp >= kSoft0 && warp < kSoft0 + kSoftWarps) {
        // ------------------------- softmax, correction and epilogue -------------------------
        // key = lane of S^T; half = which 32 rows of the tile; srow: one row a thread of the first 64
        set_regs<kRegsSoft>();
        Item it = {bar.work[0], bar.work[1], bar.work[2], bar.work[3], 0, 0};
        bool have = fill(p, it);
        uint32_t g = 0, ii = 0;                              // blocks and items so far
        const int half = (warp - kSoft0) >> 2, key = 32 * (warp & 3) + lane;
        const int srow = (int)threadIdx.x - 32 * kSoft0;
        const uint32_t prow = smem + kOffR + key * 128;
        bool ok = true, vis_ready = false;
        uint32_t tree = 0u;                                  // of sequence tree_b, in the first softmax warp
        int tree_b = -1;
        // this thread's 32 scores of the block, scaled, plus off[row]; -inf where hidden
        auto scores = [&](const float *off, bool masked, uint32_t see, float (&x)[32]) {
            uint32_t raw[32];
            tmem_ld32(lane_addr(tmem + kColS, warp, 32 * half), raw);
            loaded(raw);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 o = reinterpret_cast<const float4 *>(off + 32 * half)[q];
                x[4 * q] = fmaf(__uint_as_float(raw[4 * q]), p.scale_log2, o.x);
                x[4 * q + 1] = fmaf(__uint_as_float(raw[4 * q + 1]), p.scale_log2, o.y);
                x[4 * q + 2] = fmaf(__uint_as_float(raw[4 * q + 2]), p.scale_log2, o.z);
                x[4 * q + 3] = fmaf(__uint_as_float(raw[4 * q + 3]), p.scale_log2, o.w);
            }
            if (sh.bad[g & 1][key]) {                        // NaN wherever it is seen
#pragma unroll
                for (int r = 0; r < 32; ++r) x[r] = __uint_as_float(0x7fffffffu);
            }
            if (masked) {
#pragma unroll
                for (int r = 0; r < 32; ++r) x[r] = (see >> r) & 1u ? x[r] : -INFINITY;
            }
        };
        // an item's rows of Q, in the order widening gives the dims: a warp takes 8 rows
        auto load_q = [&](const Item &q) {
            const int r0 = 8 * (warp - kSoft0), R0 = q.rt * kRowsT + r0, sub = lane & 7, kq = lane >> 3;
            const int64_t base = (int64_t)q.b * p.rows_seq + R0;
            // all loads first: their latency stands between two items
            uint4 v[8][2], w[2];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q_nope + (base + r) * p.q_nope_stride) + lane;
                const bool live = R0 + r < p.rows_seq;
                v[r][0] = live ? __ldg(src) : make_uint4(0u, 0u, 0u, 0u);      // 16-byte chunks of the row's 64
                v[r][1] = live ? __ldg(src + 32) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = R0 + 4 * h + kq < p.rows_seq
                           ? __ldg(reinterpret_cast<const uint4 *>(p.q_pe + (base + 4 * h + kq) * p.q_pe_stride) + sub)
                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sts(smem + kOffQ + (r0 + r) * 128 + (4 * h + (lane >> 3)) * kQTile + (((lane & 7) ^ ((r0 + r) & 7)) << 4),
                        q8::reorder8(v[r][h]));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r0 + 4 * h + kq;
                sts(smem + kOffQ + 8 * kQTile + r * 128 + ((sub ^ (r & 7)) << 4), w[h]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.qfull);
        };
        if (have) load_q(it);
        if (srow < kRowsT) sh.zero[srow] = 0.f;
        for (; have; have = advance(p, it), ++ii) {
            float l = 0.f;                                   // of row `lane` of the 32, over this warp's keys
            if (srow < kRowsT) {
                sh.m[srow] = -INFINITY;
                sh.nm[srow] = kNoReference;
            }
            barrier_or<1, 256>(false);
            bool fail = false;
            for (int j = 0; j < it.nb; ++j, ++g) {
                // which rows see this thread's key, when the block holds tree keys, or rows behind them
                const int key0 = (it.kb + j) * kKeysB;
                const bool masked = key0 + kKeysB > it.P;
                uint32_t see = ~0u;
                if (masked) {
                    if (!vis_ready) {
                        griddep_wait();
                        vis_ready = true;
                    }
                    const int i0 = it.rt * kRowsT / p.H, w0 = max(key0 - it.P, 0) >> 5;
                    if (p.parent) {
                        if (srow < 32) {
                            if (it.b != tree_b) tree = walk_tree(p, it.b, lane);
                            tree_b = it.b;
                            if (lane >= i0) sh.vis[(lane - i0) * kVisWords] = tree;
                        }
                    } else                               // (from L2: written while this kernel ran)
                    for (int e = srow; e < kRowsT * kVisWords; e += 32 * kSoftWarps) {
                        const int i = i0 + e / kVisWords, wd = w0 + e % kVisWords;
                        sh.vis[e] = i < p.T && wd < p.W ? __ldcg(p.vis + ((int64_t)it.b * p.T + i) * p.W + wd) : 0u;
                    }
                    barrier_or<1, 256>(false);
                    see = seen_by(p, sh.vis, i0, w0, key0 + key - it.P, it.rt * kRowsT + 32 * half);
                }
                ok = ok && warp_wait(bar, &bar.sfull, g & 1, p.err, -41);
                float x[32];                                 // score - reference
                // minus the reference, kNoReference for a row without one; an item's first block goes straight
                // to the maxima
                const float *off = j > 0 ? sh.nm : sh.zero;
                bool raised = false;
                if (j == 0 && (fail = barrier_or<1, 256>(!ok))) break;
                if (ok) tc_fence_after();
#pragma unroll 1
                for (;;) {
                    if (ok) scores(off, masked, see, x);
                    if (off == sh.nm) {
                        if (raised) break;
                        float top = -INFINITY;
#pragma unroll
                        for (int r = 0; r < 32; r += 2) top = fmax3(top, x[r], x[r + 1]);
                        if (!barrier_or<1, 256>(!ok || top > kRaise)) break;
                        if ((fail = barrier_or<1, 256>(!ok))) break;
                        off = sh.zero;                       // some row's reference has to rise: once more for
                        continue;                            // the scores themselves
                    }
                    // the block's maxima, quadrant by quadrant
                    sh.red[warp & 3][32 * half + lane] =
                        transpose_reduce(x, lane, [](float a, float b) { return fmaxf(a, b); });
                    barrier_or<1, 256>(false);
                    if (srow < kRowsT) {
                        const int r = srow;
                        const float to = fmaxf(fmaxf(sh.red[0][r], sh.red[1][r]), fmaxf(sh.red[2][r], sh.red[3][r]));
                        const float m = sh.m[r];
                        float a = 1.f;
                        if (to > m + kRaise) {
                            a = m == -INFINITY ? 1.f : ex2(m - to);
                            sh.m[r] = to;
                            sh.nm[r] = -to;
                        }
                        sh.alpha[r] = a;
                    }
                    barrier_or<1, 256>(false);
                    if (j > 0) {                             // O^T (complete: the block before waited) and l
#pragma unroll 1
                        for (int q = 0; q < kPairs; ++q) {
                            uint32_t o[32];
                            const uint32_t addr = lane_addr(tmem, warp, kRowsT * q + 32 * half);
                            tmem_ld32(addr, o);
                            loaded(o);
#pragma unroll
                            for (int r = 0; r < 32; ++r)
                                o[r] = __float_as_uint(__uint_as_float(o[r]) * sh.alpha[32 * half + r]);
                            tmem_st32(addr, o);
                        }
                        tmem_wait_st();
                        l *= sh.alpha[32 * half + lane];
                    }
                    raised = true;
                    off = sh.nm;
                }
                if (fail) break;
                // p = 2^(score - m) to this key's row of P^T
                tc_fence_before();
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t o[4];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int r = 8 * u + 2 * v;
                        x[r] = ex2(x[r]);
                        x[r + 1] = ex2(x[r + 1]);
                        o[v] = q8::pack_bf16(x[r], x[r + 1]);
                    }
                    sts(prow + (((4 * half + u) ^ (key & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.pfull);
                // the sums while the tensor cores work on P^T (a running sum a thread and row would take 32
                // registers)
                l += transpose_reduce(x, lane, [](float a, float b) { return a + b; });
                if (j + 1 == it.nb) {                        // the next item's Q: this one's scores are done
                    Item nx = it;
                    if (advance(p, nx)) load_q(nx);
                }
                ok = warp_wait(bar, &bar.pdone, g & 1, p.err, -42);
                sh.bad[g & 1][key] = 0u;                     // every warp has read it: pdone follows all of pfull
            }
            if (fail) break;
            // l over the keys, then out = O / l and lse = ln2 (m + log2 l)
            sh.red[warp & 3][32 * half + lane] = l;
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
            Stage &stage = sh.stage[warp - kSoft0];
            const int rows = min(32, p.rows_seq - it.rt * kRowsT - 32 * half);   // of this warp's 32 (may be <= 0)
            // A thread has one dim of 32 rows; 512 bytes of shared memory a warp turn them into 16-byte pieces of
            // rows, with widening's order of the dims undone on the way in (an exchange by shuffles took
            // 5.6 k clocks an item, stores of single values 11 k)
            const int dim = (lane & ~3) | ((lane & 1) << 1) | ((lane >> 1) & 1);
            // 16 rows at a time, a small loop: the code of an item's end is mostly fetched anew
#pragma unroll 1
            for (int e = 0; e < 2 * kPairs; ++e) {
                const int r0 = 16 * (e & 1);
                uint32_t o[16];
                tmem_ld16(lane_addr(tmem, warp, kRowsT * (e >> 1) + 32 * half + r0), o);
                loaded(o);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 iv = *reinterpret_cast<const float4 *>(sh.inv + 32 * half + r0 + 4 * m);
                    o[4 * m] = __float_as_uint(__uint_as_float(o[4 * m]) * iv.x);
                    o[4 * m + 1] = __float_as_uint(__uint_as_float(o[4 * m + 1]) * iv.y);
                    o[4 * m + 2] = __float_as_uint(__uint_as_float(o[4 * m + 2]) * iv.z);
                    o[4 * m + 3] = __float_as_uint(__uint_as_float(o[4 * m + 3]) * iv.w);
                }
                const int64_t at = (first + 32 * half + r0) * kDc + 128 * (e >> 1) + 32 * (warp & 3);
                if (whole && kBf16Out) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at + (lane >> 2) * kDc + 8 * (lane & 3);
#pragma unroll
                    for (int g8 = 0; g8 < 16; g8 += 8) {
#pragma unroll
                        for (int r = 0; r < 8; ++r) stage.h[r][dim] = __float2bfloat16_rn(__uint_as_float(o[g8 + r]));
                        __syncwarp();
                        if (r0 + g8 + (lane >> 2) < rows) *reinterpret_cast<uint4 *>(dst + g8 * kDc) = stage.all[lane];
                        __syncwarp();
                    }
                } else {
                    float *dst = (whole ? static_cast<float *>(p.out) : p.part_o) + at + (lane >> 3) * kDc + 4 * (lane & 7);
#pragma unroll
                    for (int g4 = 0; g4 < 16; g4 += 4) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) stage.f[r][dim] = __uint_as_float(o[g4 + r]);
                        __syncwarp();
                        if (r0 + g4 + (lane >> 3) < rows)
                            *reinterpret_cast<uint4 *>(dst + g4 * kDc) = stage.all[lane];
                        __syncwarp();
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ofree);
        }
    } else if (warp >= kConv0) {
        // --------------------------------- converters ---------------------------------
        // Four warps a pair of latent tiles, 32 keys each, so that a pair is converted as soon as
        // O^T's MMAs have released it, whatever the others do, in one pass: wait, widen, store, fence,
        // arrive, then all loads for the next block. (With every warp taking a share of every pair the
        // pairs followed one another, each as long as that whole chain: 9.0 k clocks a block.) Four
        // keys at a time: 8 lanes a key, 8 codes of each tile a lane (one 16-byte chunk of bf16, so
        // eight lanes' stores cover all banks).
        set_regs<kRegsConv>();
        Item it = {bar.work[0], bar.work[1], bar.work[2], bar.work[3], 0, 0};
        const int pair = (warp - kConv0) >> 2, k0 = 32 * ((warp - kConv0) & 3), sub = lane & 7, kq = lane >> 3;
        // shared-memory place of key k0 + kq (key k0 + kq + 4 t follows at + 512 t), and this lane's
        // swizzled chunk for even and odd t (which flip bit 2 of the key)
        const uint32_t krow0 = smem + 2 * pair * kKTile + (k0 + kq) * 128 + ((sub ^ kq) << 4), krow1 = krow0 ^ 64;
        const uint32_t pick = sub >> 2 ? 0x7632u : 0x5410u;  // the lane's group of a tile's two
        uint2 a[8], b[8];      // codes of key k0 + kq + 4 t in the pair's first and second tile
        uint32_t sc;           // the four scale bytes of key k0 + lane
        int j = 0;
        auto load = [&]() {    // block j of item it, which then moves on
            const int key0 = (it.kb + j) * kKeysB + k0, left = it.P + p.T - key0;
            const int64_t row = (int64_t)it.b * p.L + key0;
            const uint8_t *cp = p.c_q8 + (row + kq) * kDc + 128 * pair + 8 * sub;
            sc = lane < left ? __ldg(reinterpret_cast<const uint32_t *>(p.c_scale + (row + lane) * (kDc / KDT_Q8_GROUP)) + pair)
                             : 0x7f7f7f7fu;
            if (left >= 32) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    a[t] = __ldg(reinterpret_cast<const uint2 *>(cp + 4 * t * kDc));
                    b[t] = __ldg(reinterpret_cast<const uint2 *>(cp + 4 * t * kDc + 64));
                }
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    a[t] = b[t] = make_uint2(0u, 0u);
                    if (kq + 4 * t < left) {
                        a[t] = __ldg(reinterpret_cast<const uint2 *>(cp + 4 * t * kDc));
                        b[t] = __ldg(reinterpret_cast<const uint2 *>(cp + 4 * t * kDc + 64));
                    }
                }
            }
            if (++j == it.nb) {
                j = 0;
                advance(p, it);
            }
        };
        const uint32_t G = (uint32_t)bar.work[0];            // blocks of the share
        if (fill(p, it)) load();
        for (uint32_t g = 0; g < G; ++g) {
            // before the wait: a lane turns the scale bytes of its key into factors, and gets those of
            // its eight keys (the first tile's in the low half)
            const uint32_t b0 = sc & 255u, b1 = (sc >> 8) & 255u, b2 = (sc >> 16) & 255u, b3 = sc >> 24;
            const bool plain = !__any_sync(0xffffffffu, sc & 0x80808080u);         // mostly: no scale above 1, no NaN
            const bool nan = !plain && (b0 == (uint32_t)q8::kNaN || b1 == (uint32_t)q8::kNaN || b2 == (uint32_t)q8::kNaN ||
                                        b3 == (uint32_t)q8::kNaN);
            uint32_t f[8];
            {
                uint32_t fa, fb;
                if (plain) {
                    fa = q8::low_factors(b0, b1);
                    fb = q8::low_factors(b2, b3);
                } else {
                    fa = q8::factor(b0) | (q8::factor(b1) << 16);
                    fb = q8::factor(b2) | (q8::factor(b3) << 16);
                }
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    f[t] = __byte_perm(__shfl_sync(0xffffffffu, fa, 4 * t + kq), __shfl_sync(0xffffffffu, fb, 4 * t + kq), pick);
            }
            // the pair's space: read by O^T's MMAs of the block before
            if (g > 0 && !warp_wait(bar, &bar.kempty[pair], (g - 1) & 1, p.err, -45)) break;
            if (nan) sh.bad[g & 1][k0 + lane] = 1u;
            // two keys a lane at a time: their products, their stores
#pragma unroll
            for (int t0 = 0; t0 < 8; t0 += 2) {
                uint4 v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = t0 + (k >> 1);
                    v[k] = q8::widen8(k & 1 ? b[t] : a[t], __byte_perm(f[t], 0u, k & 1 ? 0x3232u : 0x1010u));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) sts((k >> 1 ? krow1 : krow0) + 512 * (t0 + (k >> 1)) + (k & 1) * kKTile, v[k]);
            }
            // some scale above 2^7: a second product
            if (!plain && __any_sync(0xffffffffu, max(max(b0, b1), max(b2, b3)) > q8::kHighByte)) {
                const uint32_t ha = q8::factor_high(b0) | (q8::factor_high(b1) << 16);
                const uint32_t hb = q8::factor_high(b2) | (q8::factor_high(b3) << 16);
#pragma unroll 1
                for (int t = 0; t < 16; ++t) {
                    const uint32_t f = __byte_perm(__shfl_sync(0xffffffffu, t < 8 ? ha : hb, 4 * (t & 7) + kq), 0u,
                                                   sub >> 2 ? 0x3232u : 0x1010u);
                    const uint32_t dst = ((t & 1) ? krow1 : krow0) + 512 * (t & 7) + (t >> 3) * kKTile;
                    uint4 v = lds(dst);
                    v.x = q8::mul_bf16x2(v.x, f);
                    v.y = q8::mul_bf16x2(v.y, f);
                    v.z = q8::mul_bf16x2(v.z, f);
                    v.w = q8::mul_bf16x2(v.w, f);
                    sts(dst, v);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.kfull[pair]);
            if (g + 1 < G) load();
        }
    } else {
        set_regs<kRegsMma>();
        if (warp > 0) {
        // ---------------- rope keys: 16-byte asynchronous copies, zeros behind the last row ----------------
        Item it = {bar.work[0], bar.work[1], bar.work[2], bar.work[3], 0, 0};
        bool ok = true;
        uint32_t g = 0;
        for (bool have = fill(p, it); have && ok; have = advance(p, it)) {
            for (int j = 0; j < it.nb; ++j, ++g) {
                // its space held P^T of the block before
                if (g > 0 && !(ok = warp_wait(bar, &bar.pdone, (g - 1) & 1, p.err, -46))) break;
                const int key0 = (it.kb + j) * kKeysB, left = it.P + p.T - key0;
                const __nv_bfloat16 *src = p.k_pe + ((int64_t)it.b * p.L + key0) * kDr;
                for (int c = 32 * (warp - 1) + lane; c < kKeysB * 8; c += 32 * kRopeWarps) {
                    const int key = c >> 3;                  // a row behind the last is not read (0 bytes)
                    cp_async16(smem + kOffR + key * 128 + (((c & 7) ^ (key & 7)) << 4), key < left ? src + 8 * c : src,
                               key < left ? 16u : 0u);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.rfull);
            }
        }
        } else if (elect_one()) {
        // -------------------------------- MMA issuer --------------------------------
        Item it = {bar.work[0], bar.work[1], bar.work[2], bar.work[3], 0, 0};
        bool have = fill(p, it);
        uint32_t g = 0, ii = 0;                              // blocks and items so far
        const uint32_t id_s = idesc_bf16_f32(kKeysB, kRowsT, 0, 0), id_o = idesc_bf16_f32(kKeysB, kRowsT, 1, 1);
        // Descriptors differ only in their low words (address and leading stride); each use adds a
        // constant to a base the compiler cannot see through, or it would keep all of them live.
        const uint64_t d0 = sdesc_sw128(0, 0, 1024);
        const uint32_t dhi = (uint32_t)(d0 >> 32);
        const uint32_t base = smem >> 4, lbo_k = (16u >> 4) << 16, lbo_mn = ((uint32_t)kKTile >> 4) << 16;
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
                if (j == 0) prefetch_next_q(p, it);
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

// Joins the pieces of the tiles that a share boundary cut. CTA (c - 1, y) serves boundary c (where
// share c begins) when it is the first inside its tile, rows kMergeRows y .. of it, two warps a row
// (256 columns each: with many pieces the loads of one row are a chain, and more of them in flight
// is what counts). The shares meeting the tile, c - 1 and on, each left a normalised state (o, lse):
// o = sum_k e^(lse_k - M) o_k / sum_k e^(lse_k - M). A NaN in a piece's lse reaches the row. The
// shares' bounds are read, not computed again: the 64-bit divisions for them took 30 us.
constexpr int kMergeRows = 4;

template <bool kBf16Out>
__global__ void __launch_bounds__(64 * kMergeRows) merge_q8_rows_kernel(const Q8Params p) {
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = p.ctas, c = blockIdx.x + 1;
    const Q8Share sh = p.shares[c];
    const int64_t before = p.shares[c - 1].start;
    if (sh.start == sh.t0 || before > sh.t0) return;          // between two tiles, or not the first inside this one
    const int row = blockIdx.y * kMergeRows + (warp >> 1), col = 256 * (warp & 1) + 4 * lane;
    if (row >= sh.rows) return;
    // share k's slot: 2k when it starts in the tile (which is its first item then), else 2k + 1; -1: it does
    // not meet the tile, or is empty
    auto slot = [&](int k) {
        if (k >= C) return -1;
        const int64_t a = p.shares[k].start, e = p.shares[k + 1].start;
        return a >= sh.t1 || a == e ? -1 : (a >= sh.t0 ? 2 * k : 2 * k + 1);
    };
    // two passes over the shares, 32 at a time: the largest lse, then the weighted sums
    float M = -INFINITY;
    bool nan = false;
    for (int base = c - 1; base < C && p.shares[base].start < sh.t1; base += 32) {
        const int sl = slot(base + lane);
        const float v = sl >= 0 ? p.part_lse[(int64_t)sl * kRowsT + row] : -INFINITY;
        nan |= v != v;
        M = fmaxf(M, v);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    nan = __any_sync(0xffffffffu, nan);
    float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    float S = nan ? __uint_as_float(0x7fffffffu) : 0.f;
    if (M > -INFINITY)
        for (int base = c - 1; base < C && p.shares[base].start < sh.t1; base += 32) {
            const int sl = slot(base + lane);
            const float v = sl >= 0 ? p.part_lse[(int64_t)sl * kRowsT + row] : -INFINITY;
            const float wt = v == -INFINITY ? 0.f : __expf(v - M);
            float ws = wt;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
            S += ws;
            // the pieces that count (weight 0: no visible key, no such share), their loads independent
            uint32_t live = __ballot_sync(0xffffffffu, wt != 0.f);
            while (live) {
                float4 a[4], d[4];
                float wk[4];
                int n = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    wk[u] = 0.f;
                    if (!live) continue;                      // (uniform)
                    const int k = __ffs(live) - 1;
                    live &= live - 1;
                    wk[u] = __shfl_sync(0xffffffffu, wt, k);
                    const float4 *src =
                        reinterpret_cast<const float4 *>(p.part_o + ((int64_t)__shfl_sync(0xffffffffu, sl, k) * kRowsT + row) * kDc + col);
                    a[u] = src[0];
                    d[u] = src[32];
                    n = u + 1;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u >= n) break;
                    acc[0] = make_float4(fmaf(wk[u], a[u].x, acc[0].x), fmaf(wk[u], a[u].y, acc[0].y), fmaf(wk[u], a[u].z, acc[0].z),
                                         fmaf(wk[u], a[u].w, acc[0].w));
                    acc[1] = make_float4(fmaf(wk[u], d[u].x, acc[1].x), fmaf(wk[u], d[u].y, acc[1].y), fmaf(wk[u], d[u].z, acc[1].z),
                                         fmaf(wk[u], d[u].w, acc[1].w));
                }
            }
        }
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const int64_t grow = sh.row0 + row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 v = make_float4(acc[h].x * inv, acc[h].y * inv, acc[h].z * inv, acc[h].w * inv);
        if (kBf16Out)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + grow * kDc + col + 128 * h) =
                make_uint2(q8::pack_bf16(v.x, v.y), q8::pack_bf16(v.z, v.w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + grow * kDc + col + 128 * h) = v;
    }
    if (col == 0 && p.lse) p.lse[grow] = S == 0.f ? -INFINITY : M + logf(S);
}

// The same for few tiles cut into many pieces (one short batch over a long cache): CTA (tile, row),
// its eight warps take every eighth piece with all 512 columns, and meet in shared memory.
template <bool kBf16Out>
__global__ void __launch_bounds__(256) merge_q8_deep_kernel(const Q8Params p) {
    griddep_wait();
    __shared__ float part[8][kDc];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, C = p.ctas;
    const int b = blockIdx.x / p.tiles_seq, rt = blockIdx.x % p.tiles_seq, row = blockIdx.y;
    const int64_t grow = (int64_t)b * p.rows_seq + (int64_t)rt * kRowsT + row;
    if (rt * kRowsT + row >= p.rows_seq) return;
    // the first share that starts inside the tile
    int c = -1;
    for (int base = 1; base < C && c < 0; base += 32) {
        const int k = base + lane;
        const bool in = k < C && p.shares[k].row0 == grow - row && p.shares[k].start > p.shares[k].t0 &&
                        p.shares[k].start < p.shares[k].t1;
        const uint32_t m = __ballot_sync(0xffffffffu, in);
        if (m) c = base + __ffs(m) - 1;
    }
    if (c < 0) return;                                        // not cut
    const int64_t t0 = p.shares[c].t0, t1 = p.shares[c].t1;
    auto slot = [&](int k) {
        if (k >= C) return -1;
        const int64_t a = p.shares[k].start, e = p.shares[k + 1].start;
        return a >= t1 || a == e ? -1 : (a >= t0 ? 2 * k : 2 * k + 1);
    };
    // the share before may be empty: the tile's first piece is the last non-empty one's
    int first = c - 1;
    while (first > 0 && p.shares[first].start == p.shares[first + 1].start) --first;
    float M = -INFINITY;
    bool nan = false;
    for (int base = first; base < C && p.shares[base].start < t1; base += 32) {
        const int sl = slot(base + lane);
        const float v = sl >= 0 ? p.part_lse[(int64_t)sl * kRowsT + row] : -INFINITY;
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
        for (int base = first; base < C && p.shares[base].start < t1; base += 32) {
            const int sl = slot(base + lane);
            const float v = sl >= 0 ? p.part_lse[(int64_t)sl * kRowsT + row] : -INFINITY;
            const float wt = v == -INFINITY ? 0.f : __expf(v - M);
            float ws = wt;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
            S += ws;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float wk = __shfl_sync(0xffffffffu, wt, warp + 8 * u);
                const int sk = __shfl_sync(0xffffffffu, sl, warp + 8 * u);
                if (wk != 0.f) {
                    const float4 *src = reinterpret_cast<const float4 *>(p.part_o + ((int64_t)sk * kRowsT + row) * kDc) + lane;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float4 d = src[32 * q];
                        acc[q] = make_float4(fmaf(wk, d.x, acc[q].x), fmaf(wk, d.y, acc[q].y), fmaf(wk, d.z, acc[q].z), fmaf(wk, d.w, acc[q].w));
                    }
                }
            }
        }
#pragma unroll
    for (int q = 0; q < 4; ++q) reinterpret_cast<float4 *>(part[warp])[32 * q + lane] = acc[q];
    __syncthreads();
    const float inv = S == 0.f ? 0.f : 1.f / S;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 x = reinterpret_cast<const float2 *>(part[k])[threadIdx.x];
        v.x += x.x;
        v.y += x.y;
    }
    v.x *= inv;
    v.y *= inv;
    if (kBf16Out)
        reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + grow * kDc)[threadIdx.x] = q8::pack_bf16(v.x, v.y);
    else
        reinterpret_cast<float2 *>(static_cast<float *>(p.out) + grow * kDc)[threadIdx.x] = v;
    if (threadIdx.x == 0 && p.lse) p.lse[grow] = S == 0.f ? -INFINITY : M + logf(S);
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
    if (p.pieces) {
        cudaLaunchConfig_t mc = {};
        // sixteen or more pieces a tile: their loads are what takes the time. A call, a CTA a row / the other join, by
        // pieces a tile: 152 42 / 56 us, 76 36 / 44, 64 31 / 39, 38 38 / 40, 17 50 / 52, 13 68 / 66, 8 46 / 42, 4 48 / 38
        const int64_t tiles = (int64_t)p.B * p.tiles_seq;
        const bool deep = tiles * 16 <= p.ctas;
        mc.gridDim = deep ? dim3((unsigned)tiles, kRowsT) : dim3((unsigned)(p.ctas - 1), kRowsT / kMergeRows);
        mc.blockDim = dim3(deep ? 256 : 64 * kMergeRows);
        mc.stream = s;
        mc.attrs = pdl;
        mc.numAttrs = 1;
        e = cudaLaunchKernelEx(&mc, deep ? merge_q8_deep_kernel<kBf16Out> : merge_q8_rows_kernel<kBf16Out>, p);
    }
    return e;
}

}  // namespace

cudaError_t launch_verify_q8_rows(const Q8Params &p, cudaStream_t s) {
    return p.out_bf16 ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace kdt
