// C ABI of the attention over a paged latent cache: argument checks, plan and launches. See
// include/kdt.h for the contract.
#include <math.h>

#include "kdt_internal.cuh"

namespace kdt {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct PagedPlan {
    int ctas = 0, launches = 0, shares = 0;
    int tile = 0, group = 0, least = 1;    // rows of a tile, tiles side by side, least blocks of a share
    bool vis = false;                      // the visibility kernel finds the words first
    bool pieces = false;                   // a second kernel joins the pieces of what the split cut
    int deep = 0;                          // the groups, where a row can have more than a few
    size_t vis_off = 0, po_off = 0, pl_off = 0, cuts_off = 0, ws_bytes = 0;
};

constexpr int kMostGroup = 8;              // row tiles that walk the same keys side by side
// Key blocks that a share has at least, unless it is a whole group: of one block each, or three or four, one
// sequence of 13 nodes of 128 heads over 400 keys takes 33, 37, 39 us for 33, a batch of 64 single tokens over 200
// 24, 26, 24 for 24. (Two whole sequences of one block in one share took 30 us, a share each 20.)
constexpr int kLeastBlocks = 2;
// Shares a group from which several warps take a row's pieces in turn (us, L2 flushed, several warps / one): single
// tokens of 64 heads over 8192 keys, 12.7 shares a group 55.9 / 54.3, 15.2 52.1 / 50.3, 19 47.7 / 48.2, 38 38.0 / 42.1;
// of 128 heads 10.9 52.3 / 50.3, 19 42.1 / 42.1; 13 nodes of 32 heads over 4000 10.5 40.0 / 38.0, 21 31.6 / 31.8; of 16
// heads over 2000 8 29.8 / 29.8, 15.2 27.7 / 28.3. With 3 - 8 pieces a row the several lose up to 29 %.
constexpr int kDeep = 16;

kdt_status check_args(const kdt_verify_paged_args *a) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->B < 0 || a->B > 65535 || a->T < 1 || a->T > kMaxT || a->H < 1 || a->H > 1024) return KDT_ERR_BAD_SHAPE;
    if (a->D_c != kDc || a->D_r != kDr) return KDT_ERR_UNSUPPORTED;
    if (a->out_dtype != KDT_F32 && a->out_dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    const int shift = page_shift(a->page_size);
    if (a->num_splits < 0 || shift < 0 || a->n_pages < 1 || (int64_t)a->n_pages << shift > kMaxKv || a->table_width < 1)
        return KDT_ERR_BAD_SHAPE;
    if (a->table_row_stride && a->table_row_stride < a->table_width) return KDT_ERR_BAD_SHAPE;
    if (a->max_kv_len < a->T || a->max_kv_len > kMaxKv || (int64_t)a->max_kv_len > (int64_t)a->table_width << shift)
        return KDT_ERR_BAD_SHAPE;
    if ((int64_t)a->B * a->T * a->H > INT32_MAX) return KDT_ERR_BAD_SHAPE;
    if ((a->q_nope_row_stride && (a->q_nope_row_stride < kDc || a->q_nope_row_stride % 8)) ||
        (a->q_pe_row_stride && (a->q_pe_row_stride < kDr || a->q_pe_row_stride % 8)))
        return KDT_ERR_BAD_SHAPE;
    if (!(a->scale == a->scale) || isinf(a->scale)) return KDT_ERR_BAD_SHAPE;
    if (a->B == 0) return KDT_OK;
    if (!a->q_nope || !a->q_pe || !a->c_kv || !a->k_pe || !a->table || !a->prefix_len || !a->out) return KDT_ERR_NULL_ARG;
    if (a->parent && a->vis) return KDT_ERR_NULL_ARG;
    if (!a->parent && !a->vis && a->T > 1) return KDT_ERR_NULL_ARG;
    for (const void *p : {a->q_nope, a->q_pe, a->c_kv, a->k_pe, (const void *)a->out})
        if (!aligned(p, 16)) return KDT_ERR_BAD_SHAPE;
    for (const void *p : {(const void *)a->table, (const void *)a->prefix_len, (const void *)a->n_rows, (const void *)a->parent,
                          (const void *)a->vis, (const void *)a->lse, (const void *)a->err})
        if (!aligned(p, 4)) return KDT_ERR_BAD_SHAPE;
    return KDT_OK;
}

// Pure function of host-side fields.
kdt_status make_plan(const kdt_verify_paged_args *a, PagedPlan *out) {
    const kdt_status st = check_args(a);
    if (st != KDT_OK) return st;
    PagedPlan p;
    if (a->B == 0) {
        *out = p;
        return KDT_OK;
    }
    const int rows_seq = a->T * a->H;
    p.tile = rows_seq <= 16 ? 16 : (rows_seq <= 32 ? 32 : 64);
    const int tiles = (rows_seq + p.tile - 1) / p.tile, sms = sm_count();
    // side by side: all of a sequence's row tiles, or of more than 8 the number from 5 to 8 that leaves the fewest idle
    p.group = tiles;
    if (tiles > kMostGroup) {
        int best = INT32_MAX;
        for (int g = kMostGroup; g >= 5; --g) {
            const int used = (tiles + g - 1) / g * g;
            if (used < best) {
                best = used;
                p.group = g;
            }
        }
    }
    const int nblk = (a->max_kv_len + kPagedKeys - 1) / kPagedKeys;
    const int64_t groups = (int64_t)a->B * ((tiles + p.group - 1) / p.group), pairs = groups * nblk;
    int64_t C = sms / p.group > 0 ? sms / p.group : 1;
    if (a->num_splits > 0 && a->num_splits < C) C = a->num_splits;
    if (C > pairs) C = pairs;
    if (pairs / C > INT32_MAX / 2) return KDT_ERR_BAD_SHAPE;
    p.shares = (int)C;
    p.least = a->num_splits > 0 ? 1 : kLeastBlocks;
    p.ctas = p.shares * p.group;
    p.pieces = p.shares > 1 && nblk > 1;                      // a group of one block is never cut
    p.deep = p.shares >= kDeep * groups ? (int)groups : 0;
    size_t off = 0;
    p.vis = a->parent && a->T > 32;                           // the kernel walks a short tree itself
    if (p.vis) off = align_up(off + (size_t)a->B * a->T * ((a->T + 31) / 32) * sizeof(uint32_t));
    if (p.pieces) {
        const size_t rows = (size_t)2 * p.ctas * p.tile;
        p.po_off = off;
        off = align_up(off + rows * kDc * sizeof(float));
        p.pl_off = off;
        off = align_up(off + rows * sizeof(float));
        p.cuts_off = off;
        off = align_up(off + (size_t)p.shares * sizeof(PagedShare));
    }
    p.ws_bytes = off;
    p.launches = (p.vis ? 1 : 0) + 1 + (p.pieces ? 1 : 0);
    *out = p;
    return KDT_OK;
}

}  // namespace
}  // namespace kdt

using namespace kdt;

extern "C" {

size_t kdt_verify_attn_paged_workspace_size(const kdt_verify_paged_args *a) {
    PagedPlan p;
    return make_plan(a, &p) == KDT_OK ? p.ws_bytes : 0;
}

kdt_status kdt_verify_attn_paged_plan(const kdt_verify_paged_args *a, kdt_plan *out) {
    if (!out) return KDT_ERR_NULL_ARG;
    PagedPlan p;
    const kdt_status st = make_plan(a, &p);
    if (st != KDT_OK) return st;
    out->impl = KDT_IMPL_TCGEN05;
    out->num_splits = p.shares;
    out->num_launches = p.launches;
    out->ctas = p.ctas;
    out->workspace_bytes = p.ws_bytes;
    return KDT_OK;
}

kdt_status kdt_verify_attn_paged(const kdt_verify_paged_args *a, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    PagedPlan p;
    kdt_status st = make_plan(a, &p);
    if (st != KDT_OK) return st;
    if (a->B == 0) return clear_error(a->err, stream);
    if (p.ws_bytes > 0 && (!workspace || ws_bytes < p.ws_bytes || !aligned(workspace, kAlign))) return KDT_ERR_WORKSPACE;
    if ((st = check_on_current_device({a->q_nope, a->q_pe, a->c_kv, a->k_pe, a->table, a->prefix_len, a->n_rows, a->parent,
                                       a->vis, a->out, a->lse, a->err, p.ws_bytes ? workspace : nullptr})) != KDT_OK)
        return st;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const uint32_t *vis = a->vis;
    if (p.vis) {
        uint32_t *bits = reinterpret_cast<uint32_t *>(ws + p.vis_off);
        if (launch_build_visibility(a->parent, a->B, a->T, bits, a->err, stream) != cudaSuccess) return KDT_ERR_CUDA;
        vis = bits;
    } else if (a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t), stream) != cudaSuccess) {
        return KDT_ERR_CUDA;
    }
    PagedParams q = {};
    q.B = a->B;
    q.T = a->T;
    q.H = a->H;
    q.W = (a->T + 31) / 32;
    q.rows_seq = a->T * a->H;
    q.max_kv = a->max_kv_len;
    q.q_nope = static_cast<const __nv_bfloat16 *>(a->q_nope);
    q.q_pe = static_cast<const __nv_bfloat16 *>(a->q_pe);
    q.q_nope_stride = a->q_nope_row_stride ? a->q_nope_row_stride : kDc;
    q.q_pe_stride = a->q_pe_row_stride ? a->q_pe_row_stride : kDr;
    q.c_kv = static_cast<const __nv_bfloat16 *>(a->c_kv);
    q.k_pe = static_cast<const __nv_bfloat16 *>(a->k_pe);
    q.n_pages = a->n_pages;
    q.shift = page_shift(a->page_size);
    q.table = a->table;
    q.table_stride = a->table_row_stride ? a->table_row_stride : a->table_width;
    q.prefix_len = a->prefix_len;
    q.n_rows = a->n_rows;
    q.vis = vis;
    q.parent = p.vis ? nullptr : a->parent;
    q.scale_log2 = a->scale * 1.4426950408889634f;
    q.out = a->out;
    q.out_bf16 = a->out_dtype == KDT_BF16;
    q.lse = a->lse;
    q.err = a->err;
    q.tile = p.tile;
    q.group = p.group;
    q.shares = p.shares;
    q.least = p.least;
    q.pieces = p.pieces;
    q.deep = p.deep;
    q.overlap_vis = p.vis;
    q.part_o = reinterpret_cast<float *>(ws + p.po_off);
    q.part_lse = reinterpret_cast<float *>(ws + p.pl_off);
    q.cuts = reinterpret_cast<PagedShare *>(ws + p.cuts_off);
    return launch_verify_paged(q, stream) == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
