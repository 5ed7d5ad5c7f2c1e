/*
 * st_attn.h -- C ABI of the B200 (sm_100a) factorized sparse causal self-attention library.
 *
 * The method: "Sparse Transformers（稀疏 Transformer）深度解读报告" §2.1-§2.2 (factorized heads,
 * strided and fixed patterns), §3.1 (head integration, Eq.6-8), §3.4 (recompute in the
 * backward pass), §3.5 (block-sparse kernels: blocked computation, fused softmax, the upper
 * triangle never computed).  The block layout follows "长序列为何不必让每个 token 看见全部历史？
 * 滑动窗口、块稀疏与全局 token" §05 (only selected block pairs enter the kernel, boundary blocks
 * carry an element mask) and the attention arithmetic its §01-§02.
 *
 * Allowed sets (0-based positions, every set restricted to j <= i):
 *   strided  A1(i) = {max(0, i-l) .. i}          A2(i) = {j : (i-j) mod l == 0}
 *   fixed    A1(i) = {j : j/l == i/l}            A2(i) = {j : j mod l in [l-c-o, l-1-o]}
 * where o is the fixed pattern-2 head's sub-block offset (below).  A merged head attends to
 * A1 union A2 with one softmax.
 *
 * Arithmetic (per batch b, head h, row i):  S_ij = q_i.k_j / sqrt(d) for j in A(h, i);
 * P_ij = softmax_j(S_ij); O_i = sum_j P_ij v_j; lse_i = ln sum_j exp(S_ij) (natural log, fp32).
 * A row whose allowed set is empty (only the first l-c-o rows of a fixed pattern-2 head) gets
 * O_i = 0 and lse_i = -inf and passes no gradient.  No dropout.  bf16 I/O computes with bf16
 * tensor-core products and fp32 accumulation; fp32 I/O keeps the score product in three-term
 * bf16 split precision (error about 2^-16) and the rest in bf16 products, fp32 accumulation.
 *
 * Conventions for every call:
 *   - Tensors are contiguous row-major [batch, heads, n, width] (lse and the like
 *     [batch, heads, n]), in device memory owned by the caller, each 16-byte aligned; the row
 *     widths are the descriptor's d (Q, K) and dv (V, O), both 64 for the kernels.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy default stream) and
 *     return after enqueueing work; argument errors are reported before anything is enqueued.
 *   - No call allocates device memory except st_layout_upload (the layout's own tables).
 *   - Nothing throws across this boundary.  A device-side bounded wait that gives up sets the
 *     layout's device error word; st_layout_check reports it (ST_ERR_DEVICE_TIMEOUT).
 */
#ifndef ST_ATTN_H
#define ST_ATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define ST_API __attribute__((visibility("default")))
#else
#define ST_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *st_stream_t; /* same type as cudaStream_t */

typedef enum {
    ST_OK = 0,
    ST_ERR_INVALID_ARG = 1,     /* NULL pointer, bad enum, inconsistent or non-positive sizes */
    ST_ERR_UNSUPPORTED = 2,     /* valid for the method, not handled by the kernels (d != 64 ...) */
    ST_ERR_ALIGNMENT = 3,       /* a tensor pointer is not 16-byte aligned */
    ST_ERR_NOT_UPLOADED = 4,    /* st_layout_upload has not been called for this layout */
    ST_ERR_CUDA = 5,            /* a CUDA runtime or driver call failed */
    ST_ERR_OOM = 6,             /* host or device allocation failed */
    ST_ERR_DEVICE_TIMEOUT = 7,  /* a bounded device wait gave up (see st_layout_check) */
    ST_ERR_WORKSPACE = 8,       /* workspace NULL or smaller than the *_workspace_bytes figure */
    ST_ERR_INTERNAL = 9,
    ST_ERR_BAD_PAGE = 10        /* a block table named a page outside the cache (st_window_check) */
} st_status_t;

typedef enum { ST_STRIDED = 1, ST_FIXED = 2 } st_family_t;

/* Head integration ("Sparse Transformers 深度解读报告" §3.1):
 *   ST_PER_HEAD_ALTERNATING  heads alternate pattern head 1 (h even) and head 2 (h odd), Eq.8
 *   ST_MERGED                every head attends to A1 union A2, Eq.7
 *   ST_SINGLE_A1/_A2         every head uses head 1 (resp. head 2): one layer of Eq.6 */
typedef enum {
    ST_PER_HEAD_ALTERNATING = 1,
    ST_MERGED = 2,
    ST_SINGLE_A1 = 3,
    ST_SINGLE_A2 = 4
} st_head_mode_t;

/* Pattern-2 heads of the fixed family are numbered k = 0, 1, ... in head order (k = h/2 when
 * alternating, k = h otherwise) and look at the sub-block shifted by o_k = (k * step) mod l,
 * step = a2_offset_step, or c when a2_offset_step <= 0 (the page's advice that several heads
 * should attend different c-wide sub-blocks, §2.2).  Unused by the strided family. */
typedef struct {
    int32_t family;         /* st_family_t */
    int32_t head_mode;      /* st_head_mode_t */
    int32_t num_heads;      /* 1 .. 64 */
    int32_t a2_offset_step; /* <= 0: c */
} st_pattern_t;

/* ST_FP16 is taken by the window, norm-and-rotation and paged calls below; the factorized patterns'
 * calls (st_attn_*) refuse it with ST_ERR_INVALID_ARG. */
typedef enum { ST_BF16 = 1, ST_FP32 = 2, ST_FP16 = 3 } st_dtype_t;

/* Shapes of one call.  Q, K, dQ, dK are [batch, heads, n, d]; V, O, dO, dV are
 * [batch, heads, n, dv] ("Sparse Transformers 深度解读报告" §4.5: the models' per-head widths
 * are 32, 64 and 128, and the CIFAR-10 model halves its query-key projection, d = dv / 2).
 * Scores are scaled by 1/sqrt(d).  Widths with kernels: the forward (bf16) and the decode step
 * take (d, dv) = (32, 32), (64, 64), (128, 128) and (64, 128); the backward pass and the fp32
 * forward take (64, 64).  Other widths are valid arguments and return ST_ERR_UNSUPPORTED. */
typedef struct {
    int64_t batch, heads, n, d; /* heads must equal the layout's num_heads, n its n */
    int32_t dtype;              /* st_dtype_t: Q, K, V, O, dO, dQ, dK, dV all in this type */
    int32_t dv;                 /* width of the V, O, dO, dV rows; 0 means d; negative: invalid */
} st_desc_t;

/* Allowed-set kind of one head (st_layout_head_kind). */
typedef enum {
    ST_KIND_SA1 = 1, ST_KIND_SA2 = 2, ST_KIND_SU = 3,
    ST_KIND_FA1 = 4, ST_KIND_FA2 = 5, ST_KIND_FU = 6
} st_kind_t;

typedef struct st_layout st_layout_t; /* opaque; owns its host tables and its device copy */

/* Build the block layout of a pattern (host only, no CUDA call).
 *   n      sequence length, >= 1; the kernels further need n % 128 == 0 and n % l == 0
 *   l      stride / block length, >= 1
 *   c      fixed family: summary width, 1 <= c <= l (kernels: c a power of two <= 128 and
 *          every o_k + c <= l); strided family: ignored
 *   block  64 or 128: granularity of the natural-frame CSR that st_layout_export returns
 * The layout holds, per distinct head kind, the natural-frame CSR of active key blocks per
 * query block with deduplicated element masks of boundary blocks (the bit-exact contract), and
 * the execution-frame work lists the kernels run (128 x 128 tiles; the strided pattern-2 head
 * runs on the (n/l) x l grid view of the sequence, one column per tile row group, the fixed
 * pattern-2 head on its compacted summary keys).  Errors: ST_ERR_INVALID_ARG for invalid
 * values, ST_ERR_OOM.  *out is set only on ST_OK; release with st_layout_destroy. */
ST_API st_status_t st_layout_build(const st_pattern_t *pattern, int64_t n, int32_t l, int32_t c,
                            int32_t block, st_layout_t **out);

/* Copy the execution tables to the current CUDA device, asynchronously on `stream`.  Allocates
 * the layout's device buffers on first call (the only allocation in this library).  A layout
 * is bound to the device current at upload.  Errors: ST_ERR_UNSUPPORTED if the kernels cannot
 * run this layout (n % 128, n % l, c, heads > 64), ST_ERR_CUDA, ST_ERR_OOM. */
ST_API st_status_t st_layout_upload(st_layout_t *layout, st_stream_t stream);

/* Kind (st_kind_t) and fixed sub-block offset o of head `head` (host only).
 * Errors: ST_ERR_INVALID_ARG (NULL layout, head outside [0, num_heads)). */
ST_API st_status_t st_layout_head_kind(const st_layout_t *layout, int32_t head, int32_t *kind,
                                int32_t *offset);

/* Natural-frame CSR of head `head` (borrowed pointers, valid until st_layout_destroy):
 *   query block qb (rows qb*block .. +block-1) lists key blocks col_idx[row_ptr[qb] ..
 *   row_ptr[qb+1]-1] in increasing order; a key block is listed iff some (i, j) in the block pair
 *   is allowed.  mask_id[e] is -1 when every pair of the block is allowed, else the index of
 *   its element mask: masks + mask_id * (block*block/32) u32 words, bit (r*block + cc) set iff
 *   (qb*block + r, kb*block + cc) is allowed, words little-endian.  Rows or columns past n are
 *   never set.  Identical masks are stored once per head kind.  The CSR of a head kind is built
 *   on its first export (the kernels run the execution frames, not this view), so the first call
 *   can take time at long n; ST_ERR_OOM if it does not fit in host memory. */
ST_API st_status_t st_layout_export(const st_layout_t *layout, int32_t head, const int32_t **row_ptr,
                             const int32_t **col_idx, const int32_t **mask_id,
                             const uint32_t **masks, int32_t *n_qblk, int32_t *nnz,
                             int32_t *n_masks);

/* Per batch element figures of the execution plan (host only).  Errors: ST_ERR_INVALID_ARG
 * (NULL argument), ST_ERR_UNSUPPORTED (a layout the kernels cannot run has no plan). */
typedef struct {
    int64_t fwd_items;      /* forward work items (query tiles over all heads and passes) */
    int64_t exec_tiles;     /* active 128 x 128 tile pairs the kernels compute */
    int64_t bwd_items;      /* backward work items (key tiles over all heads and passes) */
    int64_t allowed_pairs;  /* sum over heads and rows of |A(h, i)| */
    int32_t passes;         /* 1, or 2 for merged strided heads (band part, then grid part) */
    int32_t split_passes;   /* passes with a key tile whose query run is split over several CTAs
                               (each adds one short summing launch to the backward pass) */
    int32_t dq_direct_heads; /* heads whose every query tile is read by one backward item: their
                                dQ is written by st_attn_bwd_main, not accumulated */
    int32_t reserved;       /* 0 */
} st_layout_info_t;
ST_API st_status_t st_layout_info(const st_layout_t *layout, st_layout_info_t *info);

/* Host enumeration of the keys row i of head `head` attends in the execution frames (the same
 * frame and interval rules the kernels use), increasing, written to keys[0 .. *count-1];
 * keys must hold n entries.  For tests of the execution plan against the set definitions.
 * Errors: ST_ERR_INVALID_ARG (NULL pointer, head or i out of range), ST_ERR_UNSUPPORTED (a
 * layout the kernels cannot run has no plan). */
ST_API st_status_t st_layout_exec_row(const st_layout_t *layout, int32_t head, int64_t i, int64_t *keys,
                               int64_t *count);

/* Synchronise `stream` and report (and clear) the layout's device error word:
 * ST_ERR_DEVICE_TIMEOUT if a kernel's bounded wait gave up since the last check. */
ST_API st_status_t st_layout_check(st_layout_t *layout, st_stream_t stream);

/* Diagnostic of the failure path: launches one warp on `stream` whose single bounded wait is on
 * an mbarrier that nothing completes, so it gives up after the kernels' wait limit (1 s) and
 * records the timeout in the layout's device error word, as a stalled kernel pipeline would.
 * The next st_layout_check then returns ST_ERR_DEVICE_TIMEOUT (and clears the word); the CUDA
 * context stays usable.  Lets a caller test its error handling without a real fault.
 * Errors: ST_ERR_INVALID_ARG (NULL layout, or the current device is not the layout's),
 * ST_ERR_NOT_UPLOADED, ST_ERR_CUDA (launch failed). */
ST_API st_status_t st_selftest_wait_timeout(st_layout_t *layout, st_stream_t stream);

/* Release the layout's host tables and device buffers (NULL is a no-op).  Work already enqueued
 * that uses the layout must have completed. */
ST_API void st_layout_destroy(st_layout_t *layout);

/* Workspace (device bytes, 256-byte aligned) the calls below need.  0 for a NULL argument or a
 * descriptor whose sizes are invalid (non-positive, or batch x heads x n above 2^40 rows). */
ST_API size_t st_attn_fwd_workspace_bytes(const st_desc_t *desc, const st_layout_t *layout);
ST_API size_t st_attn_bwd_workspace_bytes(const st_desc_t *desc, const st_layout_t *layout);

/* Forward pass.  q, k, v: inputs; o: output; lse: [batch, heads, n] fp32 output.
 * Launches the fused tcgen05 attention kernel (one pass, or two for merged strided heads whose
 * second pass merges by log-sum-exp into the first pass's O and lse).
 * The workspace (st_attn_fwd_workspace_bytes, never 0) starts with the work-unit counters of the
 * persistent kernel, zeroed on `stream` by every call: calls that run at the same time need
 * separate workspaces.  fp32 I/O adds the bf16 copies of q, k and v after them.
 * Errors (nothing enqueued): ST_ERR_INVALID_ARG (NULL pointer; descriptor sizes, heads or n not
 * the layout's; the current device is not the layout's), ST_ERR_UNSUPPORTED (row widths or a
 * layout the kernels do not handle), ST_ERR_ALIGNMENT, ST_ERR_NOT_UPLOADED, ST_ERR_WORKSPACE;
 * ST_ERR_CUDA if a launch fails. */
ST_API st_status_t st_attn_fwd(const void *q, const void *k, const void *v, const st_layout_t *layout,
                        void *o, float *lse, void *workspace, size_t workspace_bytes,
                        const st_desc_t *desc, st_stream_t stream);

/* Backward pass with recomputation ("Sparse Transformers 深度解读报告" §3.4): attention
 * probabilities are rebuilt from q, k and the saved lse.  o, dO: forward output and its
 * gradient; dq, dk, dv: outputs (every element written; keys no query reads get 0).
 * The workspace holds the fp32 dQ accumulator and the per-row D_i = dO_i . O_i.
 * Errors as for st_attn_fwd. */
ST_API st_status_t st_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                        const float *lse, const void *dO, const st_layout_t *layout, void *dq,
                        void *dk, void *dv, void *workspace, size_t workspace_bytes,
                        const st_desc_t *desc, st_stream_t stream);

/* The three phases st_attn_bwd runs, callable one by one on the same stream (in this order,
 * with the same workspace) to time or overlap them:
 *   st_attn_bwd_prepare  D_i = dO_i . O_i into the workspace, zero the fp32 dQ accumulator, and
 *                        zero dK/dV of heads whose keys are not all written by the main phase
 *   st_attn_bwd_main     the recomputing tcgen05 kernel: dK, dV written, dQ accumulated -- or,
 *                        for a head whose every query tile is read by a single key tile (the
 *                        fixed pattern's same-block head with l = 128), written to dq directly
 *   st_attn_bwd_finish   dQ accumulator -> dq (output dtype) for the other heads
 * Arguments as for st_attn_bwd; errors as for st_attn_bwd. */
ST_API st_status_t st_attn_bwd_prepare(const void *o, const void *dO, const st_layout_t *layout,
                                       void *dk, void *dv, void *workspace,
                                       size_t workspace_bytes, const st_desc_t *desc,
                                       st_stream_t stream);
ST_API st_status_t st_attn_bwd_main(const void *q, const void *k, const void *v, const float *lse,
                                    const void *dO, const st_layout_t *layout, void *dq, void *dk,
                                    void *dv,
                                    void *workspace, size_t workspace_bytes,
                                    const st_desc_t *desc, st_stream_t stream);
ST_API st_status_t st_attn_bwd_finish(const st_layout_t *layout, void *dq, void *workspace,
                                      size_t workspace_bytes, const st_desc_t *desc,
                                      st_stream_t stream);

/* Backward pass for callers that cannot allocate device memory (no counterpart in the paper:
 * this is a deployment convenience).  A plug-in inside a host application that owns every device
 * allocation, or code that must not pay cudaMalloc's implicit synchronisation, can call this
 * instead of st_attn_bwd: same arguments and results, but no workspace argument -- the scratch
 * (fp32 dQ accumulator and D_i) lives in a fixed array of ST_NOALLOC_SCRATCH_BYTES that is part of
 * the library's device image, held on every GPU that loads the library until the process exits.
 * Nothing is allocated (no cudaMalloc, cudaFree or allocating library call).
 *   - The first call on a device looks up the array's device address (once per device, with
 *     that device current); make that first call before any stream capture.  The address is
 *     tied to the device's context: after a cudaDeviceReset the next call looks it up again
 *     (that call too should come before any stream capture).
 *   - The limit: a call is accepted when st_attn_bwd_workspace_bytes(desc, layout) <=
 *     ST_NOALLOC_SCRATCH_BYTES; larger problems are rejected with ST_ERR_WORKSPACE before
 *     anything is enqueued.  The workspace grows with batch * heads * n and also holds the
 *     partial dK/dV of split key tiles and, for fp32 I/O, bf16 copies of the inputs, so the row
 *     count alone is only an upper bound: with bf16 I/O and no split key tiles, batch * heads * n
 *     up to about 129,000 rows.
 *   - All calls on a device share the array; each call re-initialises what it reads, but calls
 *     whose work overlaps on the GPU (other streams, other threads) race on it. */
#define ST_NOALLOC_SCRATCH_BYTES (32u << 20)
ST_API st_status_t st_attn_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                                       const float *lse, const void *dO,
                                       const st_layout_t *layout, void *dq, void *dk, void *dv,
                                       const st_desc_t *desc, st_stream_t stream);

/* Decode step ("长序列为何不必让每个 token 看见全部历史？…" §11: incremental inference brings one new
 * query row per step, Q_LEN = 1, against the key/value cache including the new position).
 * For every (batch, head): the query row q[b, h] at sequence position pos attends to its allowed
 * set A(h, pos) among the cache rows 0..pos -- by the set definitions exactly row pos of
 * st_attn_fwd on the full sequence.  Scores and the softmax are computed in fp32 ("Sparse
 * Transformers 深度解读报告" §3.6: query-key products in fp32 when sampling).
 *   q:        [batch, heads, 64] (desc->dtype)
 *   k_cache,
 *   v_cache:  [batch, heads, n, 64], n = the layout's n (the cache capacity); rows past pos are
 *             not read
 *   o:        [batch, heads, 64] output (desc->dtype);  lse: [batch, heads] fp32 output (natural
 *             log; -inf for a row with no allowed key, whose o is 0)
 *   workspace: st_attn_decode_workspace_bytes (a chunk counter per (batch, head), then the per-chunk
 *             partial results), 256-byte aligned; the call zeroes the counters (one memset on
 *             `stream`) and launches one kernel, whose last chunk of each row combines the row's
 *             chunks, so calls that share a workspace must not overlap on the GPU
 * desc is the full-sequence descriptor (its n is the cache capacity).  The layout need not be
 * uploaded: the kernels read only the per-head set kinds, passed by value.  Errors:
 * ST_ERR_INVALID_ARG (NULL pointers, pos outside [0, n), heads or n not the layout's),
 * ST_ERR_UNSUPPORTED (d != 64, more than 64 heads, a row with over 4,194,240 allowed keys),
 * ST_ERR_ALIGNMENT, ST_ERR_WORKSPACE,
 * ST_ERR_CUDA. */
ST_API size_t st_attn_decode_workspace_bytes(const st_desc_t *desc, const st_layout_t *layout);
ST_API st_status_t st_attn_decode(const void *q, const void *k_cache, const void *v_cache,
                                  const st_layout_t *layout, int64_t pos, void *o, float *lse,
                                  void *workspace, size_t workspace_bytes, const st_desc_t *desc,
                                  st_stream_t stream);

/* Host enumeration of the cache rows the decode step reads for head `head` at position pos,
 * increasing, written to keys[0 .. *count-1]; keys must hold pos + 1 entries.  For tests of the
 * decode step's key sets against the set definitions. */
ST_API st_status_t st_decode_row_keys(const st_layout_t *layout, int32_t head, int64_t pos,
                                      int64_t *keys, int64_t *count);

/* ================================================================================================
 * Operators of language models: attention with a sliding window and sinks, per-head norms with
 * the position rotation, and a paged key/value cache.  They share these conventions:
 *   - Tensors are given with element strides (st_strides_t); the innermost dimension is contiguous.
 *     Pointers are 16-byte aligned and every stride of a dimension longer than 1 is positive and a
 *     multiple of 16 bytes (ST_ERR_ALIGNMENT otherwise; a stride of 0 or below: ST_ERR_INVALID_ARG).
 *     Elements of one tensor do not overlap, and outputs do not overlap inputs or each other unless
 *     a call says so.
 *   - Each handle belongs to the device current at its upload; calls are made with that device
 *     current (ST_ERR_INVALID_ARG otherwise).
 *   - Nothing is allocated and nothing is kept between calls: a call may be captured into a CUDA
 *     graph.  Calls whose work overlaps on the GPU need separate workspaces.
 * ================================================================================================ */

/* Element strides of a [batch, heads, rows, width] tensor. */
typedef struct {
    int64_t batch, head, row;
} st_strides_t;

/* A sliding window with sinks.  A query at position p sees the keys j with
 *     j <= p  and  (window == 0  or  j > p - window  or  j < sinks):
 * the last `window` positions, its own included (0: the whole past), and the first `sinks`.
 * Query heads share key heads in groups: head h reads key head h / (heads / kv_heads). */
typedef struct st_window st_window_t;

/* heads, kv_heads >= 1 with heads % kv_heads == 0; window, sinks in 0 .. 2^30 (host only). */
ST_API st_status_t st_window_create(int32_t heads, int32_t kv_heads, int64_t window, int64_t sinks,
                                    st_window_t **out);
/* Bind the handle to the current device and allocate its error word (the only allocation). */
ST_API st_status_t st_window_upload(st_window_t *window, st_stream_t stream);
/* Synchronise `stream`, report and clear the handle's device error word: ST_ERR_DEVICE_TIMEOUT if
 * a bounded wait gave up, ST_ERR_BAD_PAGE if a block table named a page outside the cache.  The
 * error word is shared by every call made with the handle, on any stream. */
ST_API st_status_t st_window_check(st_window_t *window, st_stream_t stream);
/* Release the handle (NULL is a no-op).  Work that uses it must have completed, and captured graphs of
 * its calls hold the error word's address: they must not be replayed after this. */
ST_API void st_window_destroy(st_window_t *window);

/* Shapes of a window call.  q, o, dO, dq: [batch, heads, nq, d]; k, v, dk, dv: [batch, kv_heads,
 * nk, d]; lse: [batch, heads, nq] fp32, contiguous.  Query row i stands at position q_start + i of
 * the keys' sequence.  Scores are scaled by 1 / sqrt(d).  d: 64 or 128; dtype: ST_BF16 or ST_FP16;
 * nq, nk <= 2^30; q_start + nq <= 2^30 (others: ST_ERR_UNSUPPORTED). */
typedef struct {
    int64_t batch, nq, nk, d, q_start;
    int32_t dtype, reserved;
    st_strides_t q, k, v, o, dout, dq, dk, dv; /* the forward reads q, k, v, o only */
} st_window_desc_t;

/* Forward: O_i = sum_j softmax_j(q_i . k_j / sqrt d) v_j over the keys that row i sees, and
 * lse_i = ln sum_j exp(q_i . k_j / sqrt d).
 *   lens  device int32 [batch] or NULL: the sequence of batch element b has lens[b] positions
 *         (clamped to 0 .. nk; NULL: nk).  Rows at positions lens[b] and beyond are padding: O = 0
 *         and lse = -inf; keys there are not seen, whatever they hold (NaN included).
 * o and lse must not overlap each other or an input.
 * A row that sees a score of NaN or +inf gets NaN in O and lse.  A NaN or an infinity in a row before
 * lens[b] may reach O of other rows of its batch element and group too (0 times NaN is NaN).  A row whose
 * scores are all -inf gets O = 0 and lse = -inf.
 * 16-bit products with fp32 accumulation; the probabilities are rounded to the inputs' type for
 * the second product.
 * Errors: ST_ERR_INVALID_ARG (NULL pointer, sizes, q_start < 0, another device current, an output that
 * is another array),
 * ST_ERR_UNSUPPORTED, ST_ERR_ALIGNMENT, ST_ERR_NOT_UPLOADED, ST_ERR_CUDA. */
ST_API st_status_t st_window_fwd(const void *q, const void *k, const void *v, const int32_t *lens,
                                 const st_window_t *window, void *o, float *lse,
                                 const st_window_desc_t *desc, st_stream_t stream);

/* Backward with recomputation from q, k and the saved lse: dq, dk, dv (every element written;
 * padding rows and unseen keys get 0, whatever dO, O and lse hold there).  The sums run in a fixed
 * order: the same inputs give the same bits.  dS (and P) are rounded to the inputs' type for their
 * products; with ST_FP16 they are scaled by powers of two that keep them in range, per key head.  A NaN or
 * an infinity in a row before lens[b] (dO, O and lse included) may reach any gradient of its batch element
 * and group, those of unseen keys too.
 * dq, dk, dv and the workspace must not overlap each other or an input.
 * Errors as for the forward, and ST_ERR_WORKSPACE. */
ST_API size_t st_window_bwd_workspace_bytes(const st_window_desc_t *desc, const st_window_t *window);
ST_API st_status_t st_window_bwd(const void *q, const void *k, const void *v, const void *o,
                                 const float *lse, const void *dO, const int32_t *lens,
                                 const st_window_t *window, void *dq, void *dk, void *dv,
                                 void *workspace, size_t workspace_bytes, const st_window_desc_t *desc,
                                 st_stream_t stream);

/* ---- norms of queries and keys per head, with the position rotation -------------------------- */
typedef enum { ST_ROPE_NONE = 0, ST_ROPE_LINEAR = 1, ST_ROPE_NTK = 2, ST_ROPE_YARN = 3 } st_rope_scaling_t;

/* Rotation speeds (host only): turns[i] = 2^64 w_i / 2 pi, i < rot / 2, in units of 2^-64 turns per
 * position, with w_i = base^(-2i / rot), and the factor *mscale on cos and sin (1 except for YARN).  Scaling by
 * `factor` s >= 1 for contexts s times the `original` one:
 *   LINEAR  w_i / s (positions interpolated)
 *   NTK     base s^(rot / (rot - 2)): the slowest pair slows by s, the fastest keeps its speed
 *   YARN    by parts: r_i = original w_i / 2 pi turns over the original context, kept share
 *           t = clamp((r_i - 1) / (32 - 1), 0, 1), w_i (t + (1 - t) / s); mscale = 0.1 ln s + 1
 * Errors: ST_ERR_INVALID_ARG (NULL, rot odd or < 2 (NTK: < 4), base <= 1, factor < 1, original <= 0). */
ST_API st_status_t st_rope_turns(int32_t rot, double base, int32_t scaling, double factor, double original,
                                 uint64_t *turns, float *mscale);

/* Shapes of a norm-and-rotation call.  q and q_out: [batch, heads, n, d]; k and k_out: [batch,
 * kv_heads, n, d]; in the backward the *_out strides are those of the output gradients, and dq, dk
 * those of the input gradients.  d: a multiple of 16 up to 256; rot: a multiple of 16, 16 .. d;
 * dtype: ST_BF16, ST_FP16 or ST_FP32; wdtype: type of wq and wk (dtype or ST_FP32).
 * positions: int32, element (b, t) at b * pos_batch + t (pos_batch 0: shared by the batch). */
typedef struct {
    int64_t batch, heads, kv_heads, n, d, start, pos_batch;
    int32_t rot, interleaved, dtype, wdtype;
    float eps, mscale;
    st_strides_t q, k, q_out, k_out, dq, dk;
} st_rope_desc_t;

/* Per head row x of q or k: y = x / sqrt(mean(x^2) + eps) * w (wq, wk: [d] weights, or both NULL:
 * no norm), then the rotation of the first `rot` elements by the angle a_i = pos w_i:
 *   half layout (interleaved 0): pairs (i, i + rot/2);  interleaved: pairs (2i, 2i + 1)
 *   (y0, y1) -> mscale (y0 cos a - y1 sin a, y1 cos a + y0 sin a)
 * pos = positions[b, t], or start + t when positions is NULL.  Angles are products of 64-bit
 * integers modulo a turn, so far positions keep their accuracy.  fp32 arithmetic, rounded once.  turns:
 * device [rot / 2].
 * q_out may be q and k_out may be k (same strides); otherwise outputs overlap nothing.  Errors:
 * ST_ERR_INVALID_ARG (NULL pointer, sizes, an output that is another array), ST_ERR_UNSUPPORTED,
 * ST_ERR_ALIGNMENT, ST_ERR_CUDA. */
ST_API st_status_t st_qk_norm_rope(const void *q, const void *k, const void *wq, const void *wk,
                                   const uint64_t *turns, const int32_t *positions, void *q_out, void *k_out,
                                   const st_rope_desc_t *desc, st_stream_t stream);

/* Gradients: gq, gk of the outputs; dq, dk of the inputs (dq may be gq, dk may be gk, same strides);
 * dwq, dwk: [d] fp32 (NULL without weights), summed in a fixed order.  Other outputs and the workspace
 * overlap nothing. */
ST_API size_t st_qk_norm_rope_bwd_workspace_bytes(const st_rope_desc_t *desc);
ST_API st_status_t st_qk_norm_rope_bwd(const void *q, const void *k, const void *gq, const void *gk,
                                       const void *wq, const void *wk, const uint64_t *turns,
                                       const int32_t *positions, void *dq, void *dk, float *dwq, float *dwk,
                                       void *workspace, size_t workspace_bytes, const st_rope_desc_t *desc,
                                       st_stream_t stream);

/* ---- paged key/value cache -------------------------------------------------------------------
 * Keys and values live in pages of page_size positions: k_pages, v_pages [num_pages, kv_heads,
 * page_size, d] (strides: batch = page).  A request's block table lists its pages in order; the slot
 * of a position is page * page_size + its offset. */
typedef struct {
    int64_t num_pages, page_size;  /* num_pages * page_size <= 2^31 - 1 */
    st_strides_t k, v;
} st_pages_t;

/* One serving step's plan, on the device: block tables and slot maps from the requests' lengths.
 *   lens, new   [requests] int32: positions already cached, and new tokens of this step
 *   block_table [requests, max_pages] int32, row stride table_stride: the columns of newly taken
 *               pages are written, the others left as they were
 *   free_pages  [*] int32, free_count [1] int32: a stack of free pages; pages are taken from its top,
 *               free_pages[free_count - 1] first, request by request
 * Tokens are numbered request by request: request r has tokens offsets[r] .. offsets[r + 1] - 1
 * (new[r] of them; negative counts as 0).  A request is served unless lens[r] or new[r] is negative,
 * its positions need more than max_pages pages, its tokens pass `tokens`, or its pages and those
 * asked for by the requests before it (ones refused for that included) exceed free_count.
 *   lens_out   [requests]: lens + new of a served request, else lens
 *   free_left  [1]: free_count less the pages taken
 *   offsets    [requests + 1]
 *   slots, positions [tokens]: of each token; -1 for tokens of a request not served and for entries
 *              past the last token (and the slot of a token whose block table entry is negative)
 *   status     [requests]: 0 served, 1 not served
 * free_pages may be NULL where free_capacity is 0.  Inputs and outputs must not overlap (block_table
 * apart).  requests: 1 .. 8192; tokens: 1 .. 2^30; page_size: 1 .. 2^20; max_pages: 1 .. 2^24.  Slots are
 * 32-bit: a slot past 2^31 - 1 is given as -1.
 * Errors: ST_ERR_INVALID_ARG (NULL pointer, sizes, an output that is an input), ST_ERR_UNSUPPORTED
 * (requests > 8192), ST_ERR_CUDA. */
typedef struct {
    int64_t requests, tokens, max_pages, table_stride, page_size, free_capacity;
} st_plan_desc_t;
ST_API st_status_t st_paged_plan(const int32_t *lens, const int32_t *new_tokens, int32_t *block_table,
                                 const int32_t *free_pages, const int32_t *free_count, int32_t *lens_out,
                                 int32_t *free_left, int32_t *offsets, int32_t *slots, int32_t *positions,
                                 int32_t *status, const st_plan_desc_t *desc, st_stream_t stream);

/* New tokens into the cache, with their norm and rotation in the same pass: q [tokens, heads, d] ->
 * q_out, k [tokens, kv_heads, d] -> normed and rotated into its slot of k_pages, v -> v_pages.
 * desc is as for st_qk_norm_rope with batch = 1 and n = tokens (strides: row = token, head; k_out and
 * start unused); v: strides of the values.  positions, slots: [tokens] int32, as st_paged_plan gives
 * them.  A token whose slot is outside 0 .. num_pages * page_size - 1 is skipped: its q_out row and
 * the cache are left as they were.  q_out may be q (same strides); otherwise outputs overlap nothing.
 * Slots must be distinct: of two tokens with one slot either may
 * be stored, in part. */
ST_API st_status_t st_paged_append(const void *q, const void *k, const void *v, const void *wq, const void *wk,
                                   const uint64_t *turns, const int32_t *positions, const int32_t *slots,
                                   void *q_out, void *k_pages, void *v_pages, const st_strides_t *v_strides,
                                   const st_pages_t *pages, const st_rope_desc_t *desc, st_stream_t stream);

/* Attention of one new token per request over its pages.  q, o: [requests, heads, d] contiguous; lse:
 * [requests, heads] fp32; block_table as above; lens [requests] int32: keys in the cache, the new
 * token's included (clamped to 0 .. max_pages * page_size), so the query stands at lens - 1.  A request
 * of length 0 gets O = 0, lse = -inf.  A key whose page is outside 0 .. num_pages - 1 is not seen, and
 * the window's error word records it (ST_ERR_BAD_PAGE from st_window_check).  Cache rows that are
 * not seen are not used, whatever they hold; a score of NaN or +inf gives NaN in O and lse.  For the
 * second product the probabilities are rounded to the inputs' type; with ST_BF16 and heads / kv_heads <= 8
 * they keep 16 bits (two bf16 parts).  d: 64 or 128; dtype: ST_BF16 or ST_FP16; heads / kv_heads <= 64;
 * requests <= 8192; page_size a multiple of 16; max_pages * page_size <= 2^30.  o, lse and the workspace must not overlap each other or an input.  The
 * order of the sums depends on lens and on the device only: the same inputs give the same bits.
 * Errors: ST_ERR_INVALID_ARG, ST_ERR_UNSUPPORTED, ST_ERR_ALIGNMENT, ST_ERR_NOT_UPLOADED,
 * ST_ERR_WORKSPACE, ST_ERR_CUDA. */
typedef struct {
    int64_t requests, d, max_pages, table_stride;
    int32_t dtype, reserved;
    st_pages_t pages;
} st_paged_desc_t;
ST_API size_t st_paged_decode_workspace_bytes(const st_paged_desc_t *desc, const st_window_t *window);
ST_API st_status_t st_paged_decode(const void *q, const void *k_pages, const void *v_pages,
                                   const int32_t *block_table, const int32_t *lens, const st_window_t *window,
                                   void *o, float *lse, void *workspace, size_t workspace_bytes,
                                   const st_paged_desc_t *desc, st_stream_t stream);

/* Static description of a status code. */
ST_API const char *st_status_string(st_status_t status);

/* Library version string. */
ST_API const char *st_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ST_ATTN_H */
