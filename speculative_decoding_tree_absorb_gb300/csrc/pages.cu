// A paged latent cache: pages given to and taken from requests (kdt_page_assign) and new rows
// written to their slots (kdt_latent_write_paged). See include/kdt.h for the contracts.
#include <cmath>

#include "latent_rows.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"

namespace kdt {
namespace {

using namespace rows;

// ------------------------------------------------------------------------ pages --
// Request b needs ceil(new_len / page) pages and holds held[b]. In terms of one stack: all
// surplus pages go on top of it, the first given uppermost, then the missing ones come off the
// top. So the k-th page taken is the k-th given, or past those the stack's (k - given)-th from
// the top, and only pages given but not taken are written to the stack: nothing that another
// thread reads is written, and the order of threads does not show.
//
//  * One cluster does it all. Every CTA scans the B requests for itself (gives and takes before
//    each, in shared memory), then the cluster's threads share the pages, each found by a binary
//    search over the scanned counts, then the rows' slots, read through the new table.
//  * State that every CTA reads (held, n_free) is written behind a cluster barrier.
//  * Latency bounds it: a launch, the requests' lengths, a page's search and its read, the table again for the
//    rows. So a thread has four pages and a lane 16 rows in flight at once. 8 requests of 64 new rows, and back:
//    11 us a call, of it 5 - 7 on the device; 256 prompts of 2001 rows in pages of 16, 32256 pages and 512256
//    slots: 20 us, of which the slots take 12 (a row at a time 25); their return 8 (one CTA 29).
constexpr int kAssignThreads = 1024;
constexpr int kAssignCluster = 8;
constexpr int kMaxAssign = 16384;                   // requests: their scans lie in shared memory
// Dynamic shared memory that a launch is given unasked: 48 KB less the kernel's static variables (below 1 KB).
constexpr size_t kFreeSmem = 47 * 1024;
constexpr int kRowsALane = 16;                      // rows whose page a lane looks up at once
constexpr int kPagesAThread = 4;
constexpr int kRowsACta = 16384, kPagesACta = 4096; // slots, table entries that one CTA takes before another joins

struct AssignParams {
    int32_t *table, *held, *free_pages, *n_free;
    const int32_t *new_len, *start;
    int32_t *slots, *err;
    int64_t table_stride;
    int B, W, T, n_pages, shift;
};

__device__ __forceinline__ int2 warp_scan2(int2 v, int lane) {      // inclusive
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, v.x, off), y = __shfl_up_sync(0xffffffffu, v.y, off);
        if (lane >= off) v = make_int2(v.x + x, v.y + y);
    }
    return v;
}

// The last b with first[b] <= k.
__device__ __forceinline__ int owner_of(const int *first, int B, int k) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kAssignThreads) page_assign_kernel(const AssignParams p) {
    extern __shared__ int dyn[];
    int *gives = dyn, *takes = dyn + p.B;           // before request b
    __shared__ int2 warp_sum[32];
    __shared__ int s_taken, s_refused;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank, size;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    const int n_free = min(max(*p.n_free, 0), p.n_pages);
    if (tid == 0) {
        s_taken = 0;
        s_refused = INT32_MAX;
    }
    // pages request b asks for, -1 when it cannot be served whatever is free
    auto wants = [&](int b, int &have) {
        have = p.held[b];
        const int len = p.new_len[b];
        const int need = (int)(((uint32_t)max(len, 0) + (1u << p.shift) - 1) >> p.shift);
        return len < 0 || need > p.W || have < 0 || have > p.W ? -1 : need;
    };
    // -- gives and takes before each request
    const int per = (p.B + kAssignThreads - 1) / kAssignThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    int2 mine = make_int2(0, 0);
    for (int b = b0; b < b1; ++b) {
        int have;
        const int need = wants(b, have);
        gives[b] = mine.x;
        takes[b] = mine.y;
        if (need >= 0) mine = make_int2(mine.x + max(have - need, 0), mine.y + max(need - have, 0));
    }
    int2 incl = warp_scan2(mine, lane);
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int2 v = warp_sum[lane];
        const int2 s = warp_scan2(v, lane);
        warp_sum[lane] = make_int2(s.x - v.x, s.y - v.y);
        if (lane == 31) incl = s;                   // (kept for the totals below)
    }
    __shared__ int2 s_total;
    if (tid == 31) s_total = incl;
    __syncthreads();
    const int given = s_total.x;
    const int64_t room = (int64_t)given + n_free;
    const int2 self = warp_scan2(mine, lane);
    const int2 base = make_int2(warp_sum[warp].x + self.x - mine.x, warp_sum[warp].y + self.y - mine.y);
    int taken = 0, refused = INT32_MAX;
    for (int b = b0; b < b1; ++b) {
        gives[b] += base.x;
        takes[b] += base.y;
        int have;
        const int need = wants(b, have), end = takes[b] + max(need - have, 0);
        if (need < 0 || (need > have && end > room)) refused = min(refused, b);
        else if (need > have) taken = max(taken, end);
    }
    if (taken) atomicMax(&s_taken, taken);
    if (refused != INT32_MAX) atomicMin(&s_refused, refused);
    __syncthreads();
    taken = s_taken;
    auto served = [&](int b, int &need, int &have) {
        need = wants(b, have);
        return need >= 0 && !(need > have && takes[b] + need - have > room);
    };
    // -- pages: those taken to their tables, those given and not taken to the stack
    // (nothing read here is written here: a thread reads several before it writes)
    const uint32_t step = size * kAssignThreads, all = (uint32_t)max(taken, given);     // (below 2^31: k is free to pass it)
    for (uint32_t k0 = rank * kAssignThreads + tid; k0 < all; k0 += kPagesAThread * step) {
        int32_t page[kPagesAThread];
#pragma unroll
        for (int i = 0; i < kPagesAThread; ++i) {
            const int64_t k = k0 + i * step;
            page[i] = 0;
            if (k < given) {
                const int b = owner_of(gives, p.B, (int)k);
                int need, have;
                served(b, need, have);
                page[i] = p.table[b * p.table_stride + need + (k - gives[b])];
            } else if (k < all)
                page[i] = p.free_pages[n_free - 1 - (k - given)];
        }
#pragma unroll
        for (int i = 0; i < kPagesAThread; ++i) {
            const int64_t k = k0 + i * step;
            if (k < taken) {
                const int b = owner_of(takes, p.B, (int)k);
                int need, have;
                if (served(b, need, have) && need > have) p.table[b * p.table_stride + have + (k - takes[b])] = page[i];
            } else if (k < given && room - 1 - k < p.n_pages)
                p.free_pages[room - 1 - k] = page[i];
        }
    }
    // -- every row's slot
    if (p.slots) {
        if (size > 1) tc::cluster_sync();
        else __syncthreads();
        // a run of rows of one request is shared by as many lanes, up to 32, as it has rows
        const uint32_t T = (uint32_t)p.T;
        uint32_t lanes = 1;
        while (lanes < 32 && lanes < T) lanes *= 2;
        const uint32_t chunks = (T + lanes * kRowsALane - 1) / (lanes * kRowsALane), units = (uint32_t)p.B * chunks;
        const uint32_t abreast = 32 / lanes, stride = size * (kAssignThreads / 32) * abreast;
        for (uint32_t u = (rank * (kAssignThreads / 32) + warp) * abreast + lane / lanes; u < units; u += stride) {
            const uint32_t b = u / chunks, t0 = (u - b * chunks) * lanes * kRowsALane + (lane & (lanes - 1));
            int need, have;
            // modulo 2^32: a row before the first lies beyond every length
            const uint32_t row0 = (uint32_t)p.start[b] + t0, len = served((int)b, need, have) ? (uint32_t)p.new_len[b] : 0u;
            const uint32_t mask = (1u << p.shift) - 1u;
            const int32_t *pages = p.table + (int64_t)b * p.table_stride;
            int32_t *slots = p.slots + (int64_t)b * p.T + t0;
            int32_t page[kRowsALane];
#pragma unroll
            for (int i = 0; i < kRowsALane; ++i) {
                const uint32_t row = row0 + i * lanes;
                page[i] = t0 + i * lanes < T && row < len ? __ldcg(pages + (row >> p.shift)) : -1;
            }
#pragma unroll
            for (int i = 0; i < kRowsALane; ++i) {
                const int32_t slot = (int32_t)(((uint32_t)page[i] << p.shift) + ((row0 + i * lanes) & mask));
                if (t0 + i * lanes < T) slots[i * lanes] = (uint32_t)page[i] < (uint32_t)p.n_pages ? slot : -1;
            }
        }
    }
    // -- what every CTA has read
    if (size > 1) tc::cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        for (int b = tid; b < p.B; b += kAssignThreads) {
            int need, have;
            if (served(b, need, have)) p.held[b] = need;
        }
        if (tid == 0) {
            *p.n_free = (int32_t)min(room - taken, (int64_t)p.n_pages);
            if (p.err) *p.err = s_refused == INT32_MAX ? 0 : s_refused + 1;
        }
    }
}

// --------------------------------------------------------------- rows to their slots --
// One warp a row, as for the 8-bit cache (same norm, same rotation); a lane's pieces of the
// latent go out as 16 (bf16 input) or 8 bytes, so every store of a warp is contiguous. Bound by a launch (64
// rows 4.2 us, replayed) or by loads' latency: prompts in float32, 64 MB read and 28 written, 14.5 - 16 us, 5.7 - 6.4
// TB/s; the same rows in bf16, 61 MB in all, 12.5 us.
constexpr int kWarps = 8, kWriters = 4;             // warps a CTA, CTAs an SM when there are rows enough

struct WriteParams {
    const void *c, *k, *gamma;
    int64_t c_stride, k_stride;
    const int32_t *pos, *slots;
    __nv_bfloat16 *c_kv, *k_pe;
    int rows, n_slots;
    float eps;
};

template <typename E>
__global__ void __launch_bounds__(32 * kWarps, kWriters) latent_write_paged_kernel(const WriteParams p,
                                                                                   const __grid_constant__ TurnFreqs fr) {
    using R = Row<E>;
    const int lane = threadIdx.x & 31;
    const uint32_t step = gridDim.x * kWarps;
    const uint64_t freq = fr.f[lane];
    for (uint32_t n = blockIdx.x * kWarps + (threadIdx.x >> 5); n < (uint32_t)p.rows; n += step) {
        const int32_t slot = p.slots[n];
        if (slot < 0 || slot >= p.n_slots) continue;
        R c;
        c.template load<true>(static_cast<const E *>(p.c) + (int64_t)n * p.c_stride, lane);
        const E *k = static_cast<const E *>(p.k) + (int64_t)n * p.k_stride;
        float k0 = to_f32(k[lane]), k1 = to_f32(k[lane + kHalf]);
        const int32_t pos = p.pos ? p.pos[n] : 0;
        float y[16];
        c.get(y);
        if (p.gamma) rms_norm(y, static_cast<const E *>(p.gamma), p.eps, lane);
        __nv_bfloat16 *dst = p.c_kv + (int64_t)slot * kDc;
#pragma unroll
        for (int q = 0; q < R::kPieces; ++q) {
            uint32_t w[R::kPer / 2];
#pragma unroll
            for (int t = 0; t < R::kPer / 2; ++t) w[t] = q8::pack_bf16(y[R::kPer * q + 2 * t], y[R::kPer * q + 2 * t + 1]);
            if constexpr (R::kPer == 4)
                reinterpret_cast<uint2 *>(dst)[32 * q + lane] = make_uint2(w[0], w[1]);
            else
                reinterpret_cast<uint4 *>(dst)[32 * q + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (p.pos) rotate(k0, k1, pos, freq);
        __nv_bfloat16 *kd = p.k_pe + (int64_t)slot * kDr;
        kd[lane] = __float2bfloat16_rn(k0);
        kd[lane + kHalf] = __float2bfloat16_rn(k1);
    }
}

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

int page_shift(int page_size) {
    for (int s = 3; s <= 10; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

}  // namespace kdt

using namespace kdt;

extern "C" {

kdt_status kdt_page_assign(const kdt_page_args *a, cudaStream_t stream) {
    if (!a) return KDT_ERR_NULL_ARG;
    const int shift = page_shift(a->page_size);
    if (a->B < 0 || a->B > kMaxAssign || a->W < 1 || a->n_pages < 0 || a->T < 0 || shift < 0) return KDT_ERR_BAD_SHAPE;
    const int64_t stride = a->table_row_stride ? a->table_row_stride : a->W;
    if (stride < a->W || (int64_t)a->B * a->W > INT32_MAX || (int64_t)a->B * a->T > INT32_MAX ||
        (int64_t)a->n_pages << shift > INT32_MAX)
        return KDT_ERR_BAD_SHAPE;
    if (a->B == 0) return clear_error(a->err, stream);
    if (!a->table || !a->held || !a->free_pages || !a->n_free || !a->new_len) return KDT_ERR_NULL_ARG;
    if (a->T > 0 && (!a->slots || !a->start)) return KDT_ERR_NULL_ARG;
    for (const void *q : {(const void *)a->table, (const void *)a->held, (const void *)a->free_pages, (const void *)a->n_free,
                          (const void *)a->new_len, (const void *)a->start, (const void *)a->slots, (const void *)a->err})
        if (!aligned(q, 4)) return KDT_ERR_BAD_SHAPE;
    const kdt_status st =
        check_on_current_device({a->table, a->held, a->free_pages, a->n_free, a->new_len, a->start, a->slots, a->err});
    if (st != KDT_OK) return st;
    const AssignParams p = {a->table, a->held, a->free_pages, a->n_free, a->new_len, a->start, a->T > 0 ? a->slots : nullptr,
                            a->err,   stride,  a->B,          a->W,      a->T,       a->n_pages, shift};
    int S = 1;
    while (S < kAssignCluster &&
           ((int64_t)a->B * a->T > (int64_t)S * kRowsACta || (int64_t)a->B * a->W > (int64_t)S * kPagesACta))
        S <<= 1;
    const size_t smem = (size_t)a->B * 2 * sizeof(int);
    if (smem > kFreeSmem &&
        cudaFuncSetAttribute(page_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kMaxAssign * 2 * sizeof(int))) !=
            cudaSuccess)
        return KDT_ERR_CUDA;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)S;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S);
    cfg.blockDim = dim3(kAssignThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, page_assign_kernel, p) == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

kdt_status kdt_latent_write_paged(const kdt_latent_write_paged_args *a, cudaStream_t stream) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->rows < 0 || a->n_slots < 0) return KDT_ERR_BAD_SHAPE;
    if (a->D_c != kDc || a->D_r != kDr) return KDT_ERR_UNSUPPORTED;
    if (a->dtype != KDT_F32 && a->dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    const int esz = a->dtype == KDT_F32 ? 4 : 2;
    const int64_t cs = a->c_row_stride ? a->c_row_stride : kDc, ks = a->k_row_stride ? a->k_row_stride : kDr;
    if (cs < kDc || (cs * esz) % 16 || ks < kDr) return KDT_ERR_BAD_SHAPE;
    if (a->gamma && !(a->eps >= 0.f && a->eps < INFINITY)) return KDT_ERR_BAD_SHAPE;
    if (a->pos && !(a->base > 0.0 && a->base <= 1e300)) return KDT_ERR_BAD_SHAPE;
    if (a->rows == 0) return KDT_OK;
    if (!a->c || !a->k || !a->slots || !a->c_kv || !a->k_pe) return KDT_ERR_NULL_ARG;
    if (!aligned(a->c, 16) || !aligned(a->gamma, 16) || !aligned(a->k, esz) || !aligned(a->c_kv, 16) ||
        !aligned(a->k_pe, 16) || !aligned(a->pos, 4) || !aligned(a->slots, 4))
        return KDT_ERR_BAD_SHAPE;
    const kdt_status st = check_on_current_device({a->c, a->k, a->gamma, a->pos, a->slots, a->c_kv, a->k_pe});
    if (st != KDT_OK) return st;
    const TurnFreqs fr = a->pos ? turn_freqs(a->base) : TurnFreqs{};
    const WriteParams p = {a->c,     a->k, a->gamma, cs, ks, a->pos, a->slots, static_cast<__nv_bfloat16 *>(a->c_kv),
                           static_cast<__nv_bfloat16 *>(a->k_pe), a->rows, a->n_slots, a->eps};
    const int64_t ctas = ((int64_t)a->rows + kWarps - 1) / kWarps, most = (int64_t)sm_count() * kWriters;
    const int grid = (int)(ctas < most ? ctas : most);
    if (a->dtype == KDT_F32)
        latent_write_paged_kernel<float><<<grid, 32 * kWarps, 0, stream>>>(p, fr);
    else
        latent_write_paged_kernel<__nv_bfloat16><<<grid, 32 * kWarps, 0, stream>>>(p, fr);
    return cudaGetLastError() == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
