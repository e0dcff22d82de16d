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
    size_t vis_off = 0, po_off = 0, pl_off = 0, ws_bytes = 0;
};

kdt_status check_args(const kdt_verify_q8_args *a) {
    if (!a) return KDT_ERR_NULL_ARG;
    if (a->B < 0 || a->B > 65535 || a->T < 1 || a->T > kMaxT || a->H < 1 || a->H > 1024) return KDT_ERR_BAD_SHAPE;
    if (a->D_c != kDc || a->D_r != kDr) return KDT_ERR_UNSUPPORTED;
    if (a->out_dtype != KDT_F32 && a->out_dtype != KDT_BF16) return KDT_ERR_UNSUPPORTED;
    if (a->impl != KDT_IMPL_AUTO && a->impl != KDT_IMPL_Q8_ROWS) return KDT_ERR_UNSUPPORTED;
    if (a->num_splits < 0) return KDT_ERR_BAD_SHAPE;
    if (a->B == 0) return KDT_OK;
    if (!a->q_nope || !a->q_pe || !a->c_q8 || !a->c_scale || !a->k_pe || !a->prefix_len || !a->out)
        return KDT_ERR_NULL_ARG;
    if ((a->parent == nullptr) == (a->vis == nullptr)) return KDT_ERR_NULL_ARG;
    if (a->max_kv_len < a->T || (int64_t)a->max_kv_len > a->kv_row_stride) return KDT_ERR_BAD_SHAPE;
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
    const int64_t tiles = (int64_t)p.tiles_seq * a->B;
    const int64_t pairs = tiles * ((a->max_kv_len + kQ8Keys - 1) / kQ8Keys);
    if (tiles > INT32_MAX || pairs / sm_count() > INT32_MAX / 2) return KDT_ERR_BAD_SHAPE;
    int64_t C = a->num_splits > 0 ? a->num_splits : sm_count();
    if (C > pairs) C = pairs;
    if (pairs / C > INT32_MAX / 2) return KDT_ERR_BAD_SHAPE;
    p.ctas = (int)C;
    size_t off = 0;
    if (a->parent) off = align_up(off + (size_t)a->B * a->T * ((a->T + 31) / 32) * sizeof(uint32_t));
    if (p.ctas > 1) {
        const size_t prow = (size_t)2 * p.ctas * kQ8Rows;
        p.po_off = off;
        off = align_up(off + prow * kDc * sizeof(float));
        p.pl_off = off;
        off = align_up(off + prow * sizeof(float));
    }
    p.ws_bytes = off;
    p.launches = (a->parent ? 1 : 0) + 1 + (p.ctas > 1 ? 1 : 0);
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
    out->num_splits = p.ctas;
    out->num_launches = p.launches;
    out->ctas = p.ctas;
    out->workspace_bytes = p.ws_bytes;
    return KDT_OK;
}

kdt_status kdt_verify_attn_q8(const kdt_verify_q8_args *a, void *workspace, size_t ws_bytes, cudaStream_t stream) {
    Q8Plan p;
    kdt_status st = make_plan(a, &p);
    if (st != KDT_OK) return st;
    if (a->B == 0) return KDT_OK;
    if (p.ws_bytes > 0 && (!workspace || ws_bytes < p.ws_bytes || !aligned(workspace, kAlign))) return KDT_ERR_WORKSPACE;
    if ((st = check_on_current_device({a->q_nope, a->q_pe, a->c_q8, a->c_scale, a->k_pe, a->prefix_len, a->parent,
                                       a->vis, a->out, a->lse, a->err, p.ws_bytes ? workspace : nullptr})) != KDT_OK)
        return st;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
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
    q.scale_log2 = a->scale * 1.4426950408889634f;
    q.out = a->out;
    q.out_bf16 = a->out_dtype == KDT_BF16;
    q.lse = a->lse;
    q.part_o = reinterpret_cast<float *>(ws + p.po_off);
    q.part_lse = reinterpret_cast<float *>(ws + p.pl_off);
    q.err = a->err;
    q.ctas = p.ctas;
    if (a->parent) {
        uint32_t *vis = reinterpret_cast<uint32_t *>(ws + p.vis_off);
        if (launch_build_visibility(a->parent, a->B, a->T, vis, a->err, stream) != cudaSuccess) return KDT_ERR_CUDA;
        q.vis = vis;
        q.overlap_vis = true;
    } else {
        q.vis = a->vis;
        if (a->err && cudaMemsetAsync(a->err, 0, sizeof(int32_t), stream) != cudaSuccess) return KDT_ERR_CUDA;
    }
    return launch_verify_q8_rows(q, stream) == cudaSuccess ? KDT_OK : KDT_ERR_CUDA;
}

}  // extern "C"
