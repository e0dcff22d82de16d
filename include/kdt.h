/*
 * kdt.h -- C ABI of libkdt.so: DDTree tree-verify MLA-absorb attention with
 * visibility masking, for NVIDIA GB300 (sm_103a).
 *
 * The method (page "The Verify-Attn Kernel: A Single File Write That Completed a
 * Critical Piece of the DDTree Engine", section "The Design Journey: From Concept
 * to CUDA"; page "The Moment of Truth: Validating a Custom CUDA Attention Kernel
 * for Speculative Decoding", sections "Context" and "The Design Journey: From
 * Theory to Silicon"): for every sequence b, draft-tree query i and head h,
 *
 *   s_j = scale * ( q_nope[b,i,h,:512] . c_kv[b,j,:512] + q_pe[b,i,h,:64] . k_pe[b,j,:64] )
 *
 * over the visible keys j -- the shared prefix j < prefix_len[b], plus tree node i
 * itself and its ancestors (node t at cache row prefix_len[b] + t) -- then
 *
 *   out[b,i,h,:] = sum_j softmax(s)_j * c_kv[b,j,:]      (the latent; the w_vc
 *                                                          up-projection stays outside)
 *   lse[b,i,h]   = ln sum_j exp(s_j)                      (natural log, scaled scores)
 *
 * The per-row lse is what merges this result with attention computed elsewhere
 * over other keys (section "Design Decisions and Trade-Offs" of the first page:
 * long prefix by another kernel, tree tail by this one, combined by log-sum-exp).
 *
 * Conventions for every entry point:
 *  - All tensor arguments are caller-owned DEVICE pointers, row-major and
 *    contiguous, 16-byte aligned, with no aliasing between inputs and outputs
 *    (kdt_verify_attn_host alone takes host tensors).
 *  - Calls are asynchronous on `stream` (0 = legacy default stream). Argument
 *    checks run on the host before any launch and never synchronise. A launch
 *    failure is returned as KDT_ERR_CUDA; faults inside a kernel surface at the
 *    caller's next synchronisation.
 *  - The library allocates no memory: scratch space is the caller's `workspace`
 *    (kdt_verify_attn_noalloc, at the end, uses a fixed array inside the library
 *    instead; kdt_verify_attn_host creates and releases its events). Its global
 *    state: that fixed device array (KDT_NOALLOC_SCRATCH_BYTES on every GPU that
 *    loads the library) and per-device caches of the SM count, of how many
 *    tensor-core clusters are resident at once, and of the array's device address.
 *    Concurrent calls are safe given distinct workspaces.
 *  - One GPU per call: kdt_verify_attn's tensors (and its workspace) must be device
 *    memory of the device current on the calling thread -- not host, managed or
 *    another GPU's memory reached through unified addressing -- else the call
 *    returns KDT_ERR_NOT_DEVICE before any launch. The tensor-core kernel loads key
 *    tiles with cluster-multicast TMA, which this library issues only over the
 *    memory of the GPU the call runs on.
 *  - Errors found in the DATA on the device (a malformed tree) are reported
 *    through a caller-provided device word `err` (0 = ok, else 1 + the flat index
 *    b*T + i of the first offending parent entry), never by a trap.
 */
#ifndef KDT_H
#define KDT_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDT_OK = 0,
    KDT_ERR_NULL_ARG = 1,     /* a required pointer is NULL, or both/neither of parent and vis */
    KDT_ERR_BAD_SHAPE = 2,    /* sizes out of range or inconsistent (B, T, H, strides, kv bounds) */
    KDT_ERR_UNSUPPORTED = 3,  /* valid but not implemented here (D_c != 512, D_r != 64, impl) */
    KDT_ERR_WORKSPACE = 4,    /* workspace NULL or smaller than kdt_verify_attn_workspace_size() */
    KDT_ERR_CUDA = 5,         /* a CUDA runtime call or kernel launch failed */
    KDT_ERR_NOT_DEVICE = 6    /* a tensor is not device memory of the current device */
} kdt_status;

/* Static, never-NULL English name of a status. */
const char *kdt_status_str(kdt_status s);

/* Library version: major * 10000 + minor * 100 + patch. */
int kdt_version(void);

typedef enum { KDT_F32 = 0, KDT_BF16 = 1 } kdt_dtype;

/* Kernel family. AUTO picks by shape and dtype: small problems -- B*T*H * max_kv_len at
 * most 2^18 for bf16 inputs, 2^19 for fp32 -- go to SIMT_SMALL, the SIMT kernel on 16-row
 * tiles with one 64-key block per split, spread over many CTAs (the tensor-core kernel's
 * pipeline has a fixed latency of tens of microseconds); otherwise bf16 inputs use the
 * tcgen05 tensor-core kernel and fp32 inputs the SIMT kernel on 64-row tiles (which
 * computes in fp32; the tensor path would round inputs). kdt_verify_attn_plan reports the
 * choice. Both SIMT forms are valid for both dtypes. */
typedef enum {
    KDT_IMPL_AUTO = 0,
    KDT_IMPL_SIMT = 1,
    KDT_IMPL_TCGEN05 = 2,
    KDT_IMPL_SIMT_SMALL = 3,
    KDT_IMPL_Q8_ROWS = 4    /* kdt_verify_attn_q8 only: tensor cores with the keys on the M side */
} kdt_impl;

/*
 * kdt_build_visibility -- draft-tree parent array -> packed ancestor bits.
 *
 * The mask comes from the tree (page "The Moment of Truth ...", section
 * "Context"): tree key t is visible to query i iff t == i or t is an ancestor of i
 * ("The Verify-Attn Kernel ...", sections "The Design Journey" and "Assumptions
 * and the Path Forward").
 *
 *   parent  device int32 [B,T]; parent[b,0] is normally -1 (the root). Requires
 *           -1 <= parent[b,i] < i (topological order; several roots allowed).
 *   vis     device uint32 [B,T,W], W = ceil(T/32): bit (t % 32) of word t / 32 of
 *           vis[b,i] is set iff t == i or t is an ancestor of i. Bits >= T are 0.
 *   err     device int32, may be NULL. Zeroed, then set to 1 + (b*T + i) of the
 *           first parent entry outside [-1, i); rows reached through such an entry
 *           stop at it. If NULL, malformed entries are silently cut the same way.
 * Errors: KDT_ERR_NULL_ARG (parent or vis NULL), KDT_ERR_BAD_SHAPE (B < 0, T < 1,
 * T > 4096), KDT_ERR_CUDA.
 */
kdt_status kdt_build_visibility(const int32_t *parent, int B, int T, uint32_t *vis, int32_t *err,
                                cudaStream_t stream);

/* Arguments of kdt_verify_attn. Sizes: B >= 0 sequences, 1 <= T <= 4096 tree
 * queries per sequence, 1 <= H <= 1024 heads. */
typedef struct {
    int B, T, H;
    int D_c;                /* latent width, must be 512 */
    int D_r;                /* rope width, must be 64 */
    kdt_dtype dtype;        /* element type of q_nope, q_pe, c_kv, k_pe (all the same) */
    const void *q_nope;     /* [B,T,H,512] absorbed query (q_nope . w_kc done by the caller) */
    const void *q_pe;       /* [B,T,H,64] rotated rope query */
    const void *c_kv;       /* [B,L,512] latent cache; row j of sequence b at c_kv + (b*L + j)*512 */
    const void *k_pe;       /* [B,L,64]  rope keys, same row indexing */
    int64_t kv_row_stride;  /* L: rows per sequence in c_kv/k_pe, >= max_kv_len */
    const int32_t *prefix_len; /* device [B]: shared-prefix length; tree node t at row prefix_len[b]+t */
    int max_kv_len;         /* host bound: >= max_b prefix_len[b] + T (sizes the grid, no
                               sync); below 2^31 - 256 */
    const int32_t *parent;  /* device [B,T] parent array, or NULL */
    const uint32_t *vis;    /* device [B,T,ceil(T/32)] packed visibility bits, or NULL */
    float scale;            /* score scale, e.g. 1/sqrt(192) */
    float *out;             /* device fp32 [B,T,H,512] */
    float *lse;             /* device fp32 [B,T,H], or NULL */
    int32_t *err;           /* device int32 error word, or NULL: 0, or with `parent` 1 + the
                               index b*T + i of the first malformed entry, or a negative
                               code if an internal wait for a copy or pipeline stage gave up */
    int impl;               /* kdt_impl */
    int num_splits;         /* 0 = choose automatically. SIMT_SMALL: KV splits per 16-row
                               tile (at most 32), merged by log-sum-exp. SIMT (64-row tiles):
                               the number of CTAs its (64-row tile, 128-key block) pairs are
                               cut into equal contiguous shares for (at most one per pair;
                               automatic: one per SM). Tensor-core kernel: the number of
                               persistent 4-CTA clusters its (256-row unit, 128-key block)
                               work is cut into equal shares for (at most those resident at
                               once). With either share split, the tiles or units a share
                               boundary cuts are merged by log-sum-exp. */
    int64_t q_nope_row_stride; /* elements between consecutive (b,i,h) rows of q_nope; 0 = 512
                                  (contiguous). Lets the kernels read a combined [.., 512 + 64]
                                  query buffer where it lies (stride 576, q_pe = q_nope + 512)
                                  instead of a split copy. Else >= 512, a multiple of 8. */
    int64_t q_pe_row_stride;   /* the same for q_pe; 0 = 64, else >= 64, a multiple of 8 */
} kdt_verify_args;

/*
 * kdt_verify_attn -- tree-verify MLA-absorb attention (the definition at the top).
 *
 * Exactly one of `parent` and `vis` must be non-NULL. With `parent`, the bits are
 * first built into the workspace as by kdt_build_visibility (and `err` reports a
 * malformed tree). With `vis`, the caller's bits are used as given: they need not
 * come from a tree, and a row whose visible set is empty (no prefix, no bit set)
 * gets out = 0 and lse = -inf.
 * Rows of c_kv/k_pe at or beyond prefix_len[b] + T never affect the result, whatever
 * they hold (NaN included); rows below max_kv_len may be read (the one-pass small-shape
 * kernel copies a sequence's first max_kv_len rows before it knows prefix_len[b]).
 * Inputs are all fp32 or all bf16; out and lse are fp32.
 * `workspace` must hold kdt_verify_attn_workspace_size(a) bytes (256-byte aligned;
 * may be NULL when that size is 0). Its contents need no initialisation.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (including prefix bound violations
 * detectable on the host: max_kv_len > kv_row_stride, max_kv_len < T),
 * KDT_ERR_UNSUPPORTED (D_c != 512, D_r != 64, unknown impl, TCGEN05 with fp32),
 * KDT_ERR_WORKSPACE, KDT_ERR_NOT_DEVICE (a tensor or the workspace is not device
 * memory of the current device), KDT_ERR_CUDA. prefix_len values are device data: the
 * caller guarantees prefix_len[b] + T <= max_kv_len.
 */
kdt_status kdt_verify_attn(const kdt_verify_args *a, void *workspace, size_t ws_bytes,
                           cudaStream_t stream);

/* Bytes of workspace kdt_verify_attn needs for these arguments (0 possible).
 * Depends only on host-side fields (sizes, dtype, impl, num_splits, which of
 * parent/vis is given). Returns 0 for arguments kdt_verify_attn would reject. */
size_t kdt_verify_attn_workspace_size(const kdt_verify_args *a);

/* What kdt_verify_attn will launch for these arguments. */
typedef struct {
    int impl;               /* the kdt_impl chosen (never KDT_IMPL_AUTO) */
    int num_splits;         /* splits, CTAs or clusters actually used (see kdt_verify_args) */
    int num_launches;       /* kernels launched per call */
    int ctas;               /* CTAs of the main attention kernel */
    size_t workspace_bytes;
} kdt_plan;

kdt_status kdt_verify_attn_plan(const kdt_verify_args *a, kdt_plan *plan);

/*
 * kdt_verify_attn_host -- kdt_verify_attn on HOST buffers, the copies pipelined with
 * the compute.
 *
 * Same arguments and results as kdt_verify_attn, except that q_nope, q_pe, c_kv,
 * k_pe, prefix_len, parent (or vis), out and lse are HOST pointers; `err`, when
 * given, stays a DEVICE word with the same meaning (flat index over the whole
 * batch). Host rows must be contiguous (both row strides 0) and every host tensor
 * 16-byte aligned. For the copies to overlap the host buffers must be page-locked
 * (cudaHostAlloc, cudaHostRegister, a pinned torch tensor); pageable buffers give
 * the same results with the copies serialised.
 *
 * The B sequences are cut into n_chunks chunks of B / n_chunks whole sequences
 * (n_chunks must divide B; 0 = 4, else 2, else 1). Every chunk's inputs are copied
 * into `dev_buf` on stream_in (one copy per tensor); chunk c's attention (with its
 * visibility bits when parent is given) runs on `stream` once its inputs landed; its
 * out and lse are copied back on stream_out right behind it. So the copy of chunk c+1
 * in, the compute of chunk c and the copy of chunk c-1 out overlap, and the host link
 * sets the pace. The chunks' results are those of kdt_verify_attn called on each
 * chunk: they agree with one call over the whole batch within the path's tolerance
 * (the work split differs), not bit for bit.
 *
 *   dev_buf     device scratch of kdt_verify_attn_host_buffer_size(a, n_chunks)
 *               bytes, 256-byte aligned, no initialisation needed: every chunk's
 *               inputs and outputs, one error word per chunk, one verify workspace.
 *   stream      carries the compute; the call is complete -- out and lse written
 *               on the host -- once `stream` reaches the point after the call
 *               (synchronise it, or an event recorded on it, before reading out).
 *               The copies in wait for the work queued on `stream` before the call.
 *   stream_in, stream_out
 *               two more streams, distinct from each other and from `stream`. They
 *               should be non-blocking (cudaStreamNonBlocking) and `stream` not the
 *               legacy default stream with blocking streams, or the copies and the
 *               compute serialise (the results are the same).
 * The library creates two events per chunk plus two per call and releases them
 * before it returns (CUDA frees an event destroyed while pending once it completes).
 * Errors: those of kdt_verify_attn; KDT_ERR_BAD_SHAPE also for an n_chunks that
 * does not divide B, a nonzero row stride, or two equal streams; KDT_ERR_WORKSPACE
 * for a missing, short or misaligned dev_buf; KDT_ERR_NOT_DEVICE when dev_buf or
 * `err` is not device memory of the current device.
 */
kdt_status kdt_verify_attn_host(const kdt_verify_args *a, int n_chunks, void *dev_buf, size_t dev_bytes,
                                cudaStream_t stream, cudaStream_t stream_in, cudaStream_t stream_out);

/* Bytes of dev_buf kdt_verify_attn_host needs for these (host-pointer) arguments and
 * chunk count; 0 for arguments it would reject (and for B = 0). */
size_t kdt_verify_attn_host_buffer_size(const kdt_verify_args *a, int n_chunks);

/*
 * kdt_merge_attn_states -- combine two attention results over DISJOINT key sets
 * (e.g. a long prefix done elsewhere and the tree tail done here; section "Design
 * Decisions and Trade-Offs" of "The Verify-Attn Kernel ..."):
 *   M = max(lse_a, lse_b), w = exp(lse - M),
 *   o = (w_a o_a + w_b o_b) / (w_a + w_b),  lse = M + ln(w_a + w_b);
 * both -inf gives o = 0, lse = -inf.
 *   o_a, o_b, o    device fp32 [rows, D]; lse_a, lse_b, lse  device fp32 [rows].
 *   D a multiple of 4, 4 <= D <= 4096. `o`/`lse` may alias o_a/lse_a (in place).
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_CUDA.
 */
kdt_status kdt_merge_attn_states(const float *o_a, const float *lse_a, const float *o_b,
                                 const float *lse_b, int64_t rows, int D, float *o, float *lse,
                                 cudaStream_t stream);

/*
 * kdt_vc_up_proj -- per-head value up-projection of the latent attention output. The
 * verify kernel stops at the latent, and each head's value weights are applied by a
 * separate GEMM after it (page "The Verify-Attn Kernel ...", section "Design Decisions
 * and Trade-Offs"):
 *
 *   v[r, h, n] = sum_{d < D_c} o[r, h, d] * w_vc[h, d, n]        r < R, h < H, n < D_v
 *
 *   o      device fp32 [R, H, D_c]: e.g. kdt_verify_attn's `out` with R = B*T rows
 *   w_vc   device [H, D_c, D_v] in w_dtype (bf16)
 *   v      device fp32 [R, H, D_v], written whole; must not overlap o or w_vc
 *   err    device int32, may be NULL: zeroed, then a negative code if an internal
 *          pipeline wait expired (the kernel then returns early; v is incomplete)
 * Sizes: D_c = 512, D_v 64 or 128, 1 <= H <= 1024, R >= 0, R*H <= 2^31.
 * Arithmetic: each o element is split into two bf16 parts whose sum is o to within
 * 2^-16 |o|; both are multiplied by the bf16 weights on the tensor cores with fp32
 * accumulation, so the result meets the fp32 path's bound (1e-4 absolute + 1e-4
 * relative) against the exact product.
 * Errors: KDT_ERR_BAD_SHAPE (sizes, 16-byte alignment of o, w_vc and v),
 * KDT_ERR_UNSUPPORTED (D_c, D_v, w_dtype other than KDT_BF16), KDT_ERR_NULL_ARG,
 * KDT_ERR_NOT_DEVICE (a tensor not in device memory of the current device; its weights
 * and rows are read through TMA tensor maps), KDT_ERR_CUDA.
 */
kdt_status kdt_vc_up_proj(const float *o, const void *w_vc, kdt_dtype w_dtype, int R, int H, int D_c, int D_v,
                          float *v, int32_t *err, cudaStream_t stream);

/*
 * kdt_verify_attn_noalloc -- kdt_verify_attn without a caller workspace.
 *
 * The method's pages have no counterpart to this entry point; it exists for
 * callers that cannot allocate device memory when they call the library: a
 * serving engine that reserved nearly all HBM for its KV-cache pool at start-up
 * (a later cudaMalloc fails, or would fragment the pool), a plugin inside a host
 * framework whose allocator it may not call, or a latency-critical loop that cannot
 * afford the implicit device synchronisation of cudaMalloc/cudaFree.
 *
 * Same arguments, results and errors as kdt_verify_attn, but the scratch space
 * (packed visibility bits built from `parent`, split-KV partials) lives in a fixed
 * device array of KDT_NOALLOC_SCRATCH_BYTES inside libkdt.so, present on every GPU
 * that loads the library until the process exits. Nothing is allocated: no
 * cudaMalloc, no cudaFree, no allocating library routine.
 *  - Size limit: 64 MiB, enough for the partial states of the tensor-core path and of
 *    the 64-row SIMT path on any GPU they support. If the call needs more scratch, a
 *    SIMT_SMALL call's automatic split count (num_splits == 0) is lowered until the
 *    partials fit;
 *    if the call still does not fit, or an explicit num_splits does not fit, it
 *    returns KDT_ERR_WORKSPACE and launches nothing.
 *  - Set-up: the first call made on a device (with that device current) looks up
 *    the array's device address with cudaGetSymbolAddress and keeps it for that
 *    device; make that first call before any stream capture on that device. A
 *    cudaDeviceReset destroys the array with the context: the kept address then
 *    dangles, so do not call this entry point again in a process after resetting
 *    a device it was used on.
 *  - Sharing: every call on a device uses the same array and it keeps the last
 *    call's contents. The kernels overwrite every scratch byte they read, so no
 *    clearing is needed, but calls whose work overlaps on the GPU (other streams,
 *    other host threads) race on the array: order them on one stream or serialise
 *    them.
 */
#define KDT_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

kdt_status kdt_verify_attn_noalloc(const kdt_verify_args *a, cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * The steps next to verify in a DDTree step: rotary embedding of the tree's rope
 * parts before it, the greedy accept walk and the cache compaction after it.
 * ------------------------------------------------------------------------------ */

/*
 * kdt_tree_build -- best-first draft tree on the device (page "The Architecture of an
 * Inference Engine ...", section "The Context": the tree builder constructs the draft
 * tree on the GPU instead of with a per-request CPU heap).
 * For every depth d = 1..D ahead of the root the drafter gives K candidates,
 * cand_tok[b,d-1,:] with log-probabilities cand_lp[b,d-1,:], the same below every node of
 * depth d-1. A node's score is the float32 sum of the log-probabilities on its path (the
 * root's is 0). The tree grows N times by the best node not yet in it whose parent is:
 * higher score, then lower depth, then lower parent index, then lower candidate rank
 * (a depth's candidates ranked by log-probability, highest first, ties by position; NaN
 * counts as -inf). Nodes are numbered in the order they join, the root 0, so the output
 * is in topological order and feeds kdt_build_visibility / kdt_verify_attn directly.
 *   cand_tok  device int32 [B,D,K];  cand_lp  device float32 [B,D,K]
 *   root_tok  device int32 [B] or NULL: tok[b,0] (else -1)
 *   parent, tok  device int32 [B,N+1] out; depth (int32) and score (float32) [B,N+1]
 *            out, each may be NULL
 * Sizes: 1 <= D <= 64, 1 <= K <= 32, 1 <= N <= 4095 and N <= K + K^2 + ... + K^D.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_CUDA.
 */
kdt_status kdt_tree_build(const int32_t *cand_tok, const float *cand_lp, int B, int D, int K, int N,
                          const int32_t *root_tok, int32_t *parent, int32_t *tok, int32_t *depth, float *score,
                          cudaStream_t stream);

/* Arguments of kdt_rope_neox. */
typedef struct {
    int B, T, H;            /* sequences, tree nodes per sequence (1..4096), heads (1..1024) */
    int D_r;                /* rope width: even, 2..256 */
    kdt_dtype dtype;        /* element type of q and k_pe */
    void *q;                /* device, or NULL: the rope part of query row (b,i,h) is the D_r
                               elements at q + ((b*T + i)*H + h) * q_row_stride; rotated in place.
                               Point it at the rope slice of a combined [.., D_c + D_r] query
                               buffer to rotate that buffer where it lies. */
    int64_t q_row_stride;   /* elements between consecutive (b,i,h) rows, >= D_r */
    void *k_pe;             /* device [B, L, D_r], or NULL: rows prefix_len[b] + i (the tree's
                               new key rows) rotated in place; rows outside [0, L) are skipped */
    int64_t kv_row_stride;  /* L, >= T (used with k_pe) */
    const int32_t *prefix_len; /* device [B] (used with k_pe) */
    const int32_t *pos;     /* device [B,T]: rotary position of tree node i (normally
                               prefix_len[b] + depth(i), the root at depth 0) */
    double base;            /* angle base (theta), > 0, e.g. 10000 */
} kdt_rope_args;

/*
 * kdt_rope_neox -- NeoX rotary embedding in place (page "The Query-Split Kernel: A
 * Pivotal Edit ...", sections "The Reasoning Chain" -- rope applied in place on the rope
 * portion of the query buffer -- and "Input Knowledge" -- NeoX variant, float64 angles).
 * For a vector x of width d at position p and j < d/2: a_j = p * base^(-2j/d) in float64,
 * c_j and s_j its cosine and sine rounded to float32, then in float32
 *   (x_j, x_{j+d/2}) <- (x_j c_j - x_{j+d/2} s_j,  x_{j+d/2} c_j + x_j s_j),
 * each product and sum rounded to nearest on its own (no fused multiply-add), the
 * results rounded to nearest (even) to the element type. Every head of node (b,i) and
 * its key row use pos[b,i].
 * Errors: KDT_ERR_NULL_ARG (pos NULL, both q and k_pe NULL, k_pe without prefix_len),
 * KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED (dtype), KDT_ERR_CUDA.
 */
kdt_status kdt_rope_neox(const kdt_rope_args *a, cudaStream_t stream);

/*
 * kdt_tree_accept -- greedy walk of a verified draft tree (page "The Moment of Truth
 * ...", section "Context": the accept kernel walks the tree greedily to decide which
 * draft tokens are accepted). Node 0 is the root; from it, move to the child c of the
 * current node with tok[c] == target[current] (the lowest index if several), until no
 * child matches.
 *   parent   device int32 [B,T], -1 <= parent[b,i] < i (as for kdt_build_visibility)
 *   tok      device int32 [B,T]: node i's draft token (tok[b,0] unused)
 *   target   device int32 [B,T]: the target model's greedy next token after node i
 *   acc_nodes device int32 [B,T] out: the accepted path (node indices from the root),
 *            then -1
 *   n_acc    device int32 [B] out: path length, >= 1 (the root always stays)
 *   bonus    device int32 [B] out: target[last node of the path], the token the
 *            target model adds after the accepted ones
 *   err      device int32, may be NULL: zeroed, then 1 + (b*T + i) of the first parent
 *            entry outside [-1, i); such entries are skipped.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (B < 0, T < 1, T > 4096), KDT_ERR_CUDA.
 */
kdt_status kdt_tree_accept(const int32_t *parent, const int32_t *tok, const int32_t *target, int B, int T,
                           int32_t *acc_nodes, int32_t *n_acc, int32_t *bonus, int32_t *err,
                           cudaStream_t stream);

/*
 * kdt_kv_compact -- drop the unaccepted branches from the cache (page "The Architecture
 * of an Inference Engine ...", sections "The Context" and "Input Knowledge Required").
 * The tree's rows sit at cache rows prefix_len[b] + t; the k-th node of the accepted
 * path moves to row prefix_len[b] + k of both c_kv [B,L,D_c] and k_pe [B,L,D_r], in
 * place. With update_prefix != 0, prefix_len[b] += n_acc[b] afterwards. Rows past the
 * new length keep what they held. Path entries that are not increasing tree indices, or
 * that point past row L, are not copied.
 * D_c and D_r times the element size must be multiples of 16 bytes; c_kv and k_pe
 * 16-byte aligned. Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED,
 * KDT_ERR_CUDA.
 */
kdt_status kdt_kv_compact(void *c_kv, void *k_pe, kdt_dtype dtype, int D_c, int D_r, int B, int T,
                          int64_t kv_row_stride, int32_t *prefix_len, const int32_t *acc_nodes,
                          const int32_t *n_acc, int update_prefix, cudaStream_t stream);

/* ------------------------------------------------------------------------------
 * The 8-bit latent cache: the same step on a cache of a little over half the bytes.
 *
 * Row j of sequence b (656 bytes instead of bf16's 1152) is
 *   c_q8     uint8 [B,L,512]  e4m3 codes (1 sign, 4 exponent, 3 mantissa bits) of the latent
 *   c_scale  uint8 [B,L,16]   one power of two for each 32 consecutive codes (E8M0: byte s
 *                             stands for 2^(s-127))
 *   k_pe     bf16  [B,L,64]   rotated rope key, kept in 16 bits
 * and stands for c[d] = e4m3(c_q8[d]) * 2^(c_scale[d/32] - 127). Scale bytes lie in
 * [27, 227] (2^-100 .. 2^100), or are 255: a group that held an infinity or NaN, which
 * reads as NaN. Within that range every value is a bf16 number exactly, so the attention
 * below loses nothing against one over the bf16 cache of the same values. The codes 0x7f
 * and 0xff (e4m3's NaN) are never written and are not valid in a cache.
 * Rows are contiguous; all three bases are 16-byte aligned.
 * ------------------------------------------------------------------------------ */
#define KDT_Q8_GROUP 32

/* Arguments of kdt_latent_write_q8. */
typedef struct {
    int B, T;               /* sequences, new rows per sequence (tree nodes, or a prompt chunk): T >= 1 */
    int D_c, D_r;           /* must be 512 and 64 */
    kdt_dtype dtype;        /* element type of c, k and gamma */
    const void *c;          /* latent of row (b,i): the 512 elements at c + (b*T + i) * c_row_stride */
    int64_t c_row_stride;   /* elements, 0 = 512; else >= 512 and a multiple of 16 bytes */
    const void *k;          /* its rope key, not yet rotated: 64 elements at k + (b*T + i) * k_row_stride */
    int64_t k_row_stride;   /* elements, 0 = 64; else >= 64 */
    const void *gamma;      /* [512] weight of the latent's RMS norm, or NULL: no norm */
    float eps;              /* the norm's epsilon, >= 0 (used with gamma) */
    const int32_t *pos;     /* device [B,T] rotary positions, or NULL: k is written as it is */
    double base;            /* angle base (theta), > 0 (used with pos) */
    const int32_t *prefix_len; /* device [B]: row (b,i) goes to cache row prefix_len[b] + i */
    const int32_t *n_rows;  /* device [B]: sequence b has rows i < n_rows[b] only (a padded batch), or NULL: T */
    uint8_t *c_q8;          /* the cache */
    uint8_t *c_scale;
    void *k_pe;
    int64_t kv_row_stride;  /* L: cache rows per sequence, >= 1 */
} kdt_latent_write_args;

/*
 * kdt_latent_write_q8 -- norm, rotate, quantise and store new rows in one pass.
 * For every row x = c[b,i,:]:  y_d = x_d * r * gamma_d with r = 1 / sqrt(mean x^2 + eps)
 * (y = x without gamma), in float32. For each group of 32: a = max |y_d|, e = the least
 * integer with a <= 448 * 2^e, clamped to [-100, 100] (a = 0 gives -100); the scale byte
 * is e + 127 and the codes are e4m3 (round to nearest even, at most 448) of y_d * 2^-e.
 * If a is infinite or NaN the byte is 255 and the codes are 0.
 * k_pe[row] is k rotated as by kdt_rope_neox (position pos[b,i], width 64), the angle
 * taken exactly modulo a full turn and its cosine and sine in float32, rounded once to bf16.
 * Cache rows outside [0, L), and rows of sequences beyond n_rows, are left as they were.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (sizes, strides, alignment, B*T > 2^31 - 1),
 * KDT_ERR_UNSUPPORTED (D_c, D_r, dtype), KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_latent_write_q8(const kdt_latent_write_args *a, cudaStream_t stream);

/*
 * kdt_latent_read_q8 -- cache rows back in 16 or 32 bits, e.g. to move a sequence to the
 * bf16 cache kdt_verify_attn reads, or to expand a stretch of keys and values.
 *   c_q8, c_scale, k_pe, L (kv_row_stride)  the cache, B sequences
 *   start    device int32 [B]: first cache row of sequence b, or NULL: 0
 *   n_rows   device int32 [B]: rows of sequence b to read (of the R), or NULL: R
 *   c        device [B,R,512], k device [B,R,64], both of `dtype` (KDT_F32 or KDT_BF16);
 *            either may be NULL. Row (b,i) gets cache row start[b] + i exactly (every
 *            stored value is a bf16 number); a cache row outside [0, L) reads as zeros;
 *            rows i >= n_rows[b] of c and k are left as they were.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (also alignment, B*R > 2^31 - 1),
 * KDT_ERR_UNSUPPORTED, KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_latent_read_q8(const uint8_t *c_q8, const uint8_t *c_scale, const void *k_pe, int64_t kv_row_stride,
                              int B, int R, const int32_t *start, const int32_t *n_rows, kdt_dtype dtype, void *c,
                              void *k, cudaStream_t stream);

/*
 * kdt_kv_compact_q8 -- kdt_kv_compact for the 8-bit cache: the codes, scales and rope keys
 * of the accepted path's rows move to rows prefix_len[b] + k, in place; the same rules.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_kv_compact_q8(uint8_t *c_q8, uint8_t *c_scale, void *k_pe, int B, int T, int64_t kv_row_stride,
                             int32_t *prefix_len, const int32_t *acc_nodes, const int32_t *n_acc, int update_prefix,
                             cudaStream_t stream);

/* Arguments of kdt_verify_attn_q8. Sizes as for kdt_verify_attn. */
typedef struct {
    int B, T, H;
    int D_c, D_r;           /* must be 512 and 64 */
    const void *q_nope;     /* bf16 [B,T,H,512] absorbed query */
    int64_t q_nope_row_stride; /* elements between (b,i,h) rows; 0 = 512, else >= 512 and a multiple of 8 */
    const void *q_pe;       /* bf16 [B,T,H,64] rotated rope query */
    int64_t q_pe_row_stride;   /* 0 = 64, else >= 64 and a multiple of 8 */
    const uint8_t *c_q8;    /* the cache */
    const uint8_t *c_scale;
    const void *k_pe;
    int64_t kv_row_stride;  /* L: rows per sequence, >= max_kv_len */
    const int32_t *prefix_len; /* device [B]; tree node t at row prefix_len[b] + t */
    int max_kv_len;         /* host bound: >= max_b prefix_len[b] + T; below 2^31 - 256 */
    const int32_t *parent;  /* device [B,T] parent array, or NULL */
    const uint32_t *vis;    /* device [B,T,ceil(T/32)] packed visibility bits, or NULL */
    float scale;
    void *out;              /* [B,T,H,512] of out_dtype */
    kdt_dtype out_dtype;    /* KDT_F32 or KDT_BF16 */
    float *lse;             /* device fp32 [B,T,H], or NULL */
    int32_t *err;           /* device int32 error word, or NULL (as for kdt_verify_attn) */
    int impl;               /* KDT_IMPL_AUTO (the cheaper one for these sizes), KDT_IMPL_TCGEN05 (256 rows
                               at a time on 4-CTA clusters) or KDT_IMPL_Q8_ROWS (64 rows on one SM) */
    int num_splits;         /* 0 = automatic; else the CTAs the (64-row tile, 128-key block) pairs are cut
                               into equal shares for (at most one per pair), or the clusters (at most
                               those resident at once) */
} kdt_verify_q8_args;

/*
 * kdt_verify_attn_q8 -- kdt_verify_attn over the 8-bit latent cache: the same scores, mask,
 * softmax, latent output and log-sum-exp, over the values the cache stands for. T = 1 is
 * plain decoding. Products run on the tensor cores in bf16 (exact for the cache's values)
 * with float32 sums; scores, softmax statistics and the output's sums are float32, the
 * weights are rounded to bf16 for the second product, and the output once to out_dtype.
 * Exactly one of `parent` and `vis` is given; a row that sees no key gets out = 0 and
 * lse = -inf. A row that sees a NaN group, or a k_pe that makes its score NaN or +inf, gets
 * NaN (a score of -inf has weight 0); a row from which such a key is hidden is not affected
 * by it, and rows of the cache at or beyond prefix_len[b] + T are never read. prefix_len
 * values are device data: the caller guarantees 0 <= prefix_len[b] <= max_kv_len - T.
 * `workspace` must hold kdt_verify_attn_q8_workspace_size(a) bytes (256-byte aligned);
 * its contents need no initialisation. Calls that may run at the same time, captured ones
 * included, need workspaces of their own.
 * Errors: those of kdt_verify_attn, for the same reasons.
 */
kdt_status kdt_verify_attn_q8(const kdt_verify_q8_args *a, void *workspace, size_t ws_bytes, cudaStream_t stream);

/* Bytes of workspace kdt_verify_attn_q8 needs for these arguments (host-side fields only);
 * 0 for arguments it would reject. */
size_t kdt_verify_attn_q8_workspace_size(const kdt_verify_q8_args *a);

/* What kdt_verify_attn_q8 will launch for these arguments. */
kdt_status kdt_verify_attn_q8_plan(const kdt_verify_q8_args *a, kdt_plan *plan);

/* ------------------------------------------------------------------------------
 * A paged latent cache: rows of many requests in pages that requests get and give
 * back as their lengths change, instead of one block of L rows each.
 *
 *   c_kv  bf16 [n_pages, page_size, 512], k_pe bf16 [n_pages, page_size, 64]; page_size a power
 *         of two from 8 to 1024, n_pages * page_size below 2^31 - 256. Row `slot` of the cache is
 *         row slot % page_size of page slot / page_size.
 *   table int32 [B, W], row stride table_row_stride (0 = W): row j of sequence b lies in page
 *         table[b, j / page_size]. Entries behind the pages a call needs are never read as
 *         pages, whatever they hold. The attention only reads: there sequences may share pages
 *         (kdt_page_assign knows one holder of a page).
 * ------------------------------------------------------------------------------ */

/* Arguments of kdt_page_assign. All arrays on the device. */
typedef struct {
    int B;                  /* requests, at most 16384 */
    int W;                  /* entries of a table row: the most pages a request can hold */
    int32_t *table;         /* [B, W], updated */
    int64_t table_row_stride; /* 0 = W */
    int32_t *held;          /* [B]: pages request b holds, updated */
    int32_t *free_pages;    /* [n_pages] a stack: the first *n_free entries are the free pages, updated */
    int32_t *n_free;        /* [1], updated */
    int n_pages;
    int page_size;
    const int32_t *new_len; /* [B]: rows request b is to have room for (0 gives all its pages back) */
    const int32_t *start;   /* [B] first row whose slot is asked for (used with T > 0) */
    int T;                  /* rows a request whose slots are asked for, or 0 */
    int32_t *slots;         /* [B, T] out: cache row of row start[b] + i, or -1 at or beyond new_len[b] */
    int32_t *err;           /* device int32, or NULL: 0, else 1 + the first request that was refused */
} kdt_page_args;

/*
 * kdt_page_assign -- every request to ceil(new_len / page_size) pages, and where its rows go.
 * As if every surplus page were first put on the stack (requests in order, a request's pages in
 * table order, the first one given ending uppermost) and then every missing page taken off it in
 * the same order: a call that grows lengths and one that shrinks them back leave all state as it
 * was. Entries of `table` behind a request's pages and of `free_pages` at or beyond *n_free keep
 * what they held.
 * A request that asks for more than W pages, has a negative length or a `held` outside [0, W], or
 * comes when the pages free (those given back by all requests in this call included) no longer
 * cover what it and the requests before it miss, is refused: it keeps what it has, its slots are
 * -1, and `err` names the first such.
 * Slots feed kdt_latent_write_paged; a call for decoding has start = the lengths before and T = 1.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (sizes, page size, alignment, B*W or B*T > 2^31 - 1),
 * KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_page_assign(const kdt_page_args *a, cudaStream_t stream);

/* Arguments of kdt_latent_write_paged. */
typedef struct {
    int rows;               /* new rows, of all sequences */
    int D_c, D_r;           /* must be 512 and 64 */
    kdt_dtype dtype;        /* element type of c, k and gamma */
    const void *c;          /* latent of row n: the 512 elements at c + n * c_row_stride */
    int64_t c_row_stride;   /* elements, 0 = 512; else >= 512 and a multiple of 16 bytes */
    const void *k;          /* its rope key, not yet rotated: 64 elements at k + n * k_row_stride */
    int64_t k_row_stride;   /* elements, 0 = 64; else >= 64 */
    const void *gamma;      /* [512] weight of the latent's RMS norm, or NULL: no norm */
    float eps;              /* the norm's epsilon, >= 0 (used with gamma) */
    const int32_t *pos;     /* device [rows] rotary positions, or NULL: k is written as it is */
    double base;            /* angle base (theta), > 0 (used with pos) */
    const int32_t *slots;   /* device [rows]: cache row of row n; one outside [0, n_slots) is not written */
    void *c_kv;             /* bf16 [n_slots, 512] */
    void *k_pe;             /* bf16 [n_slots, 64] */
    int n_slots;            /* n_pages * page_size */
} kdt_latent_write_paged_args;

/*
 * kdt_latent_write_paged -- norm, rotate and store new rows at their slots in one pass: the norm
 * and rotation of kdt_latent_write_q8 in float32, each value rounded once to bf16. Slots of
 * different rows must differ (of two rows with one slot, either or a mixture of both is kept).
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE (sizes, strides, alignment), KDT_ERR_UNSUPPORTED
 * (D_c, D_r, dtype), KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_latent_write_paged(const kdt_latent_write_paged_args *a, cudaStream_t stream);

/*
 * kdt_kv_compact_paged -- kdt_kv_compact for a paged cache: the k-th node of the accepted path
 * moves from row prefix_len[b] + acc_nodes[b,k] of its sequence to row prefix_len[b] + k; the same
 * rules, with W * page_size in the place of L. Rows whose page is outside [0, n_pages) are not
 * copied. dtype, D_c and D_r as for kdt_kv_compact.
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED, KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_kv_compact_paged(void *c_kv, void *k_pe, kdt_dtype dtype, int D_c, int D_r, int n_pages, int page_size,
                                const int32_t *table, int W, int64_t table_row_stride, int B, int T, int32_t *prefix_len,
                                const int32_t *acc_nodes, const int32_t *n_acc, int update_prefix, cudaStream_t stream);

/* Arguments of kdt_verify_attn_paged. Sizes as for kdt_verify_attn, B*T*H below 2^31. */
typedef struct {
    int B, T, H;
    int D_c, D_r;           /* must be 512 and 64 */
    const void *q_nope;     /* bf16 [B,T,H,512] absorbed query */
    int64_t q_nope_row_stride; /* elements between (b,i,h) rows; 0 = 512, else >= 512 and a multiple of 8 */
    const void *q_pe;       /* bf16 [B,T,H,64] rotated rope query */
    int64_t q_pe_row_stride;   /* 0 = 64, else >= 64 and a multiple of 8 */
    const void *c_kv;       /* the cache */
    const void *k_pe;
    int n_pages, page_size;
    const int32_t *table;   /* device [B, table_width] */
    int table_width;
    int64_t table_row_stride; /* 0 = table_width */
    const int32_t *prefix_len; /* device [B]; tree node t at row prefix_len[b] + t */
    const int32_t *n_rows;  /* device [B]: sequence b has tree nodes i < n_rows[b] only (a padded batch; 0: it is
                               not there), or NULL: T. Rows of out and lse behind them are left as they were. */
    int max_kv_len;         /* host bound: >= max_b prefix_len[b] + T, <= table_width * page_size */
    const int32_t *parent;  /* device [B,T] parent array, or NULL. Entries of a padded batch's missing nodes may be
                               read, and reported when malformed: -1 is safe there */
    const uint32_t *vis;    /* device [B,T,ceil(T/32)] packed visibility bits, or NULL. With T = 1 both may be
                               NULL: the row sees its prefix and itself */
    float scale;
    void *out;              /* [B,T,H,512] of out_dtype */
    kdt_dtype out_dtype;    /* KDT_F32 or KDT_BF16 */
    float *lse;             /* device fp32 [B,T,H], or NULL */
    int32_t *err;           /* device int32 error word, or NULL: 0, or 1 + the index b*T + i of the first malformed
                               parent entry, or 1 + B*T + b for a sequence b one of whose pages is outside
                               [0, n_pages) (the lowest of these), or a negative code if an internal wait gave up */
    int num_splits;         /* 0 = automatic; else the shares that the work is cut into (at most one for each
                               block of keys, and one an SM) */
} kdt_verify_paged_args;

/*
 * kdt_verify_attn_paged -- kdt_verify_attn over a paged latent cache: the same scores, mask,
 * softmax, latent output and log-sum-exp, key j of sequence b read from the page the table names.
 * T = 1 is plain decoding: one new token a sequence, whose row has been written before the call.
 * Products run on the tensor cores in bf16 with float32 sums; scores, softmax statistics and the
 * output's sums are float32, the weights are rounded to bf16 for the second product, and the output
 * once to out_dtype. The work is split over the keys and joined by log-sum-exp. Meant for few rows a
 * sequence (T*H up to some 500): from there on kdt_verify_attn over a contiguous cache is faster, up
 * to 1.5 times at 4096 rows.
 * A row that sees no key gets out = 0 and lse = -inf. A row that sees a key whose score is NaN or
 * +inf gets NaN (a score of -inf has weight 0), and infinite or NaN latents reach the rows that see
 * them; a row from which such a key is hidden is not affected by it. Cache rows at or beyond
 * prefix_len[b] + n_rows[b] never affect the result, and their pages are never looked up. Rows of a
 * page outside [0, n_pages) read as zeros. prefix_len values are device data: the caller guarantees
 * 0 <= prefix_len[b] <= max_kv_len - n_rows[b]; others are brought into that range.
 * `workspace` must hold kdt_verify_attn_paged_workspace_size(a) bytes (256-byte aligned); its
 * contents need no initialisation. Calls that may run at the same time, captured ones included,
 * need workspaces of their own.
 * Errors: those of kdt_verify_attn, for the same reasons.
 */
kdt_status kdt_verify_attn_paged(const kdt_verify_paged_args *a, void *workspace, size_t ws_bytes, cudaStream_t stream);

/* Bytes of workspace kdt_verify_attn_paged needs for these arguments (host-side fields only);
 * 0 for arguments it would reject. */
size_t kdt_verify_attn_paged_workspace_size(const kdt_verify_paged_args *a);

/* What kdt_verify_attn_paged will launch for these arguments. */
kdt_status kdt_verify_attn_paged_plan(const kdt_verify_paged_args *a, kdt_plan *plan);

/* ------------------------------------------------------------------------------
 * Sampled acceptance, beside the greedy kdt_tree_accept.
 * ------------------------------------------------------------------------------ */

/*
 * kdt_tree_sample -- verify a drafted tree against the target's probabilities from given
 * random numbers. The emitted tokens (the accepted drafts and the bonus token) are
 * distributed as samples of the target, whatever was drafted.
 * At node i of sequence b, with l the V logits of (b,i): w_j = e^{(l_j - max l) / temperature},
 * held to 2^-44 of the largest, Z = sum_j w_j. From the root, the children c of the current
 * node are tried in index order: c is accepted, and becomes the current node, when
 *     u_node[b,c] * (Z - sum of the weights of the siblings tried before) < w_{tok[c]}
 * (a token that an earlier sibling drafted too counts once: the later one is never accepted).
 * When no child is accepted the bonus token is the least j with sum_{k <= j} w'_k >
 * u_bonus[b] * sum_k w'_k, where w' is w with the children's tokens set to 0.
 * A comparison that float32 sums leave in doubt, and every draw, is made in fixed point: the
 * result does not depend on how the work is split.
 *   parent   device int32 [B,T], -1 <= parent[b,i] < i;  tok device int32 [B,T] (tok[b,0] unused)
 *   logits   device, row (b,i) at logits + (b*T + i) * row_stride elements, V of them used, of
 *            dtype; row_stride 0 = V. -inf is a token that cannot be drawn.
 *   u_node   device float32 [B,T], u_bonus device float32 [B]: numbers in [0, 1)
 *   acc_nodes, n_acc, bonus  out, as kdt_tree_accept's: they feed kdt_kv_compact(_q8)
 *   logp     device float32 [B,T] out, or NULL: entry k < n_acc is the log-probability (natural,
 *            under the target at this temperature) of the token emitted after path node k, off by at
 *            most 2e-5 + 2^-23 of its size (the bonus token's: 3e-7 + 2^-23 of it); 0 behind
 *   err      device int32, or NULL: zeroed, then 1 + (b*T + i) of the first parent entry outside
 *            [-1, i) (skipped), child on the way whose token is outside [0, V) (never accepted), or
 *            node on the way whose logits have a NaN, a +inf or nothing but -inf (the walk ends
 *            there with bonus -1; also when a u of 1 or more leaves nothing to draw from).
 * Sizes: T <= 4096, V <= 524288, temperature in [1e-3, 1e3] (kdt_tree_accept is the greedy limit).
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED, KDT_ERR_NOT_DEVICE, KDT_ERR_CUDA.
 */
kdt_status kdt_tree_sample(const int32_t *parent, const int32_t *tok, const void *logits, kdt_dtype dtype, int B, int T,
                           int V, int64_t row_stride, double temperature, const float *u_node, const float *u_bonus,
                           int32_t *acc_nodes, int32_t *n_acc, int32_t *bonus, float *logp, int32_t *err,
                           cudaStream_t stream);

/* Arguments of kdt_sample. A setting is one number for all rows, or an array of one a row. */
typedef struct {
    int R, V;               /* rows, vocabulary (at most 524288) */
    const void *logits;     /* device, row r at logits + r * row_stride elements, V of them used */
    kdt_dtype dtype;
    int64_t row_stride;     /* 0 = V */
    const float *u;         /* device [R]: numbers in [0, 1) */
    const float *temperature; /* device [R], or NULL: temperature_all. In [1e-3, 1e3], or 0: greedy */
    double temperature_all;
    const int32_t *top_k;   /* device [R], or NULL: top_k_all. <= 0 or > V: all tokens */
    int top_k_all;
    const float *top_p;     /* device [R], or NULL: top_p_all. >= 1: all of them */
    double top_p_all;
    const float *min_p;     /* device [R], or NULL: min_p_all. <= 0: all of them; above 1 counts as 1 */
    double min_p_all;
    int32_t *token;         /* device [R] out */
    float *logp;            /* device [R] out, or NULL: natural log of the token's probability at this
                               temperature, before the filters (0 for a greedy row) */
    int32_t *err;           /* device int32, or NULL: 0, else 1 + the first row that has no token */
} kdt_sample_args;

/*
 * kdt_sample -- one token a row from given random numbers, under temperature, top-k, top-p and
 * min-p: the first token behind a prompt, a drafter's own tokens, plain decoding.
 * With l the row's logits: w_j = e^{(l_j - max l) / temperature}, held to 2^-44 of the largest. In
 * the order of falling logits (equal ones in index order) the row keeps
 *   the first top_k tokens; of those the least number whose weights reach top_p times the sum of
 *   the top_k's (at least one); and of those the ones with w >= min_p.
 * The token is the least j such that the kept weights up to and including j, in index order, sum
 * to more than u times the sum of all kept weights. temperature 0 gives the first token of the
 * largest logit. Sums are in fixed point: the result does not depend on how the work is split.
 * -inf is a token that cannot be drawn. A row whose logits have a NaN, a +inf or nothing but
 * -inf, or whose settings are not numbers in their ranges, gets token -1 and logp 0.
 * logp is off by at most 1e-6 + 2^-23 of its size.
 * Two kinds of rows are slower (160000 tokens on GB300): those whose top_k is above the number of tokens that
 * are not -inf, with more than 2048 that are (0.4 ms for 0.03; top_k at most that number, or 0, avoids it), and float32
 * rows with more than 2048 logits that agree in their upper 16 bits where a filter's border falls (2.5 ms for 0.1).
 * Errors: KDT_ERR_NULL_ARG, KDT_ERR_BAD_SHAPE, KDT_ERR_UNSUPPORTED (dtype), KDT_ERR_NOT_DEVICE,
 * KDT_ERR_CUDA.
 */
kdt_status kdt_sample(const kdt_sample_args *a, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDT_H */
