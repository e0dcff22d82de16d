// C ABI of the attention over the 8-bit latent cache: argument checks, plan (work split,
// workspace layout) and launches. See include/kdt.h for the contract.
#include <math.h>

#include "kdt_internal.cuh"

namespace kdt {
namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Q8Plan {
    int impl = KDT_IMPL_Q8_ROWS;
    int ctas = 0, launches = 0;
    int tiles_seq = 0;
    bool vis = false;                      // the visibility kernel finds the words first
    bool pieces = false;                   // a second kernel joins the pieces of what the split cut
    int splits = 0;                        // CTAs, or 4-CTA clusters, the work is shared among
    size_t vis_off = 0, po_off = 0, pl_off = 0, sched_off = 0, ws_bytes = 0;
};

// Which kernel, by estimates in us. The rows kernel takes a pair (64 rows of a sequence, 128 keys) in 3.7
// on one SM and 4.5 more for a tile's queries and output; a cluster takes (256 rows, 128 keys) in 2.05 on
// 4 SMs and 10 more for a unit of rows, and its set-up, schedule and drain are longer. Measured, rows
// kernel / clusters: 8 sequences of 8 k keys, 128 rows 47 / 84, 384 rows 95 / 113, 512 rows 119 / 117, 4096
// rows 793 / 536; 43 of 2688 rows, 3 keys 105 / 205, 300 keys 199 / 269, 1000 keys 406 / 403; 2 of 4096 rows,
// 2000 keys 79 / 84.
bool rows_cheaper(int64_t tiles, int64_t units, int nblk) {
    return 10.0 + tiles * (3.7 * nblk + 4.5) / sm_count() < 45.0 + units * (2.05 * nblk + 10.0) / tc_q8_max_clusters();
}

kdt_status check_args(const kdt_verify_q8_args *a) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->B < 0 || a->B > 65535 || a->T < 1 || a->T > kMaxT || a->H < 1 || a->H > 1024) return KDT_ERR_BAD_SHAPE;
    if (a->D_c != kDc || a->D_r != kDr) return KDT_ERR_UNSUPPORTED;
    if (a->out_dtype != KDT_F32 && a->out_dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    if (a->impl != KDT_IMPL_AUTO && a->impl != KDT_IMPL_TCGEN05 && a->impl != KDT_IMPL_Q8_ROWS)
        return KDT_ERR_UNSUPPORTED;
    if (a->num_splits < 0) return KDT_ERR_BAD_SHAPE;
    if (a->B == 0) return KDT_OK;
    if (!a->q_nope || !a->q_pe || !a->c_q8 || !a->c_scale || !a->k_pe || !a->prefix_len || !a->out)
        return KDT_ERR_NULL_ARG;
    if ((a->parent == nullptr) == (a->vis == nullptr)) return KDT_ERR_NULL_ARG;
    if (a->max_kv_len < a->T || a->max_kv_len > kMaxKv || (int64_t)a->max_kv_len > a->kv_row_stride)
        return KDT_ERR_BAD_SHAPE;
    for (const void *p : {a->q_nope, a->q_pe, (const void *)a->c_q8, (const void *)a->c_scale, a->k_pe,
                          (const void *)a->out})
        if (!aligned(p, 16)) return KDT_ERR_BAD_SHAPE;
    for (const void *p : {(const void *)a->prefix_len, (const void *)a->parent, (const void *)a->vis,
                          (const void *)a->lse, (const void *)a->err})
        if (!aligned(p, 4)) return KDT_ERR_BAD_SHAPE;
    if (!(a->scale == a->scale) || isinf(a->scale)) return KDT_ERR_BAD_SHAPE;
    if ((a->q_nope_row_stride && (a->q_nope_row_stride < kDc || a->q_nope_row_stride % 8)) ||
        (a->q_pe_row_stride && (a->q_pe_row_stride < kDr || a->q_pe_row_stride % 8)))
        return KDT_ERR_BAD_SHAPE;
    return KDT_OK;
}

// Pure function of host-side fields.
kdt_status make_plan(const kdt_verify_q8_args *a, Q8Plan *out) {
    const kdt_status st = check_args(a);
    if (st != KDT_OK) return st;
    Q8Plan p;
    if (a->B == 0) {
        *out = p;
        return KDT_OK;
    }
    const int rows_seq = a->T * a->H;
    p.tiles_seq = (rows_seq + kQ8Rows - 1) / kQ8Rows;
    const int units_seq = (rows_seq + tc_rows_per_unit() - 1) / tc_rows_per_unit();
    const int nblk = (a->max_kv_len + kQ8Keys - 1) / kQ8Keys;
    p.impl = a->impl != KDT_IMPL_AUTO ? a->impl
             : rows_cheaper((int64_t)a->B * p.tiles_seq, (int64_t)a->B * units_seq, nblk) ? KDT_IMPL_Q8_ROWS
                                                                                                  : KDT_IMPL_TCGEN05;
    const bool tc = p.impl == KDT_IMPL_TCGEN05;
    int piece_rows;
    if (tc) {
        if ((int64_t)a->B * rows_seq > INT32_MAX || a->kv_row_stride > INT32_MAX) return KDT_ERR_BAD_SHAPE;
        const int resident = tc_q8_max_clusters();
        p.splits = a->num_splits > 0 && a->num_splits < resident ? a->num_splits : resident;
        p.ctas = 4 * p.splits;
        piece_rows = tc_rows_per_unit();
    } else {
        const int64_t tiles = (int64_t)p.tiles_seq * a->B, pairs = tiles * nblk;
        if (tiles > INT32_MAX) return KDT_ERR_BAD_SHAPE;
        int64_t C = a->num_splits > 0 ? a->num_splits : sm_count();
        if (C > pairs) C = pairs;
        if (pairs / C > INT32_MAX / 2) return KDT_ERR_BAD_SHAPE;
        p.ctas = p.splits = (int)C;
        piece_rows = kQ8Rows;
    }
    // a tile of one block is never cut
    p.pieces = p.splits > 1 && (tc || nblk > 1);
    size_t off = 0;
    p.vis = a->parent && (tc || a->T > 32);                   // the rows kernel walks a short tree itself
    if (p.vis) off = align_up(off + (size_t)a->B * a->T * ((a->T + 31) / 32) * sizeof(uint32_t));
    if (p.pieces) {
        const size_t prow = (size_t)2 * p.splits * piece_rows;
        p.po_off = off;
        off = align_up(off + prow * kDc * sizeof(float));
        p.pl_off = off;
        off = align_up(off + prow * sizeof(float));
        p.sched_off = off;
        off = align_up(off + (tc ? kTcSchedWords * sizeof(int64_t) : (size_t)(p.splits + 1) * sizeof(Q8Share)));
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

size_t kdt_verify_attn_q8_workspace_size(const kdt_verify_q8_args *a) {
    Q8Plan p;
    return make_plan(a, &p) == KDT_OK ? p.ws_bytes : 0;
}

kdt_status kdt_verify_attn_q8_plan(const kdt_verify_q8_args *a, kdt_plan *out) {
    if (!out) return KDT_ERR_NULL_ARG;
    Q8Plan p;
    const kdt_status st = make_plan(a, &p);
    if (st != KDT_OK) return st;
    out->impl = p.impl;
    out->num_splits = p.splits;
    out->num_launches = p.launches;
    out->ctas = p.ctas;
    out->workspace_bytes = p.ws_bytes;
    return KDT_OK;
}

kdt_status kdt_verify_attn_q8(const kdt_verify_q8_args *a, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    Q8Plan p;
    kdt_status st = make_plan(a, &p);
    if (st != KDT_OK) return st;
    if (a->B == 0) return clear_error(a->err, stream);
    if (p.ws_bytes > 0 && (!workspace || ws_bytes < p.ws_bytes || !aligned(workspace, kAlign))) return KDT_ERR_WORKSPACE;
    if ((st = check_on_current_device({a->q_nope, a->q_pe, a->c_q8, a->c_scale, a->k_pe, a->prefix_len, a->parent,
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
    if (p.impl == KDT_IMPL_TCGEN05) {
        VerifyParams v;
        v.B = a->B;
        v.T = a->T;
        v.H = a->H;
        v.W = (a->T + 31) / 32;
        v.L = a->kv_row_stride;
        v.max_kv = a->max_kv_len;
        v.q_nope = a->q_nope;
        v.q_pe = a->q_pe;
        v.q_nope_stride = a->q_nope_row_stride ? a->q_nope_row_stride : kDc;
        v.q_pe_stride = a->q_pe_row_stride ? a->q_pe_row_stride : kDr;
        v.c_kv = a->c_q8;
        v.c_scale = a->c_scale;
        v.k_pe = a->k_pe;
        v.prefix_len = a->prefix_len;
        v.vis = vis;
        v.scale_log2 = a->scale * 1.4426950408889634f;
        v.out = static_cast<float *>(a->out);
        v.out_bf16 = a->out_dtype == KDT_BF16;
        v.lse = a->lse;
        v.part_o = reinterpret_cast<float *>(ws + p.po_off);
        v.part_lse = reinterpret_cast<float *>(ws + p.pl_off);
        v.tc_sched = p.pieces ? reinterpret_cast<int64_t *>(ws + p.sched_off) : nullptr;
        v.rows_total = (int64_t)a->B * a->T * a->H;
        v.tc_clusters = p.splits;
        v.num_splits = p.splits;
        v.blocks_per_split = 0;
        v.err = a->err;
        v.overlap_vis = p.vis;
        return launch_verify_tc_q8(v, stream) == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
    }
    Q8Params q = {};
    q.B = a->B;
    q.T = a->T;
    q.H = a->H;
    q.W = (a->T + 31) / 32;
    q.rows_seq = a->T * a->H;
    q.tiles_seq = p.tiles_seq;
    q.L = a->kv_row_stride;
    q.q_nope = static_cast<const __nv_bfloat16 *>(a->q_nope);
    q.q_pe = static_cast<const __nv_bfloat16 *>(a->q_pe);
    q.q_nope_stride = a->q_nope_row_stride ? a->q_nope_row_stride : kDc;
    q.q_pe_stride = a->q_pe_row_stride ? a->q_pe_row_stride : kDr;
    q.c_q8 = a->c_q8;
    q.c_scale = a->c_scale;
    q.k_pe = static_cast<const __nv_bfloat16 *>(a->k_pe);
    q.prefix_len = a->prefix_len;
    q.vis = vis;
    q.parent = p.vis ? nullptr : a->parent;
    q.scale_log2 = a->scale * 1.4426950408889634f;
    q.out = a->out;
    q.out_bf16 = a->out_dtype == KDT_BF16;
    q.lse = a->lse;
    q.part_o = reinterpret_cast<float *>(ws + p.po_off);
    q.part_lse = reinterpret_cast<float *>(ws + p.pl_off);
    q.err = a->err;
    q.ctas = p.ctas;
    q.pieces = p.pieces;
    q.shares = reinterpret_cast<Q8Share *>(ws + p.sched_off);
    q.overlap_vis = p.vis;
    return launch_verify_q8_rows(q, stream) == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
