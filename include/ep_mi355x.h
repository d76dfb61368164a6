/*
 * ep_mi355x.h: C ABI of the MI355X (gfx950) MoE expert-parallel hot path,
 * taken at one GPU's share: every expert is resident locally (a world of
 * one), so there are no peers and no collectives.
 *
 *   ep_layout    topk_idx -> per-expert counts, aligned exclusive offsets,
 *                a destination slot per (token, k), receive metadata
 *   ep_dispatch  permute-copy token rows (bf16, fp32, or fp8 e4m3 / fp4x2
 *                bytes with optional fp32 per-128-value scales) into the
 *                expert-major expand buffer
 *   ep_combine   gather each token's top-k expert-output rows (bf16 or fp32),
 *                weight them by the router weights, sum in binary32 in k
 *                order, store in the rows' type
 *
 * between them, the experts' own part: ep_moe_layer (a whole layer for a few
 * tokens), ep_expert_matvec (products with bf16, 8-bit or 4-bit weights),
 * ep_swiglu / ep_swiglu_backward (the activation, with an 8-bit checkpoint),
 * ep_expert_wgrad (the weight gradient), and the same path in 8-bit integers:
 * ep_quantize_rows, ep_swiglu_quantize and ep_quantized_matmul,
 *
 * before them: ep_router (a router's logits -> topk_idx, topk_weights,
 * per-expert counts, balance and z loss) and ep_router_backward,
 *
 * and around them: ep_layout_dispatch (layout + dispatch in one launch for a
 * one-tile batch), the non-expand mode (ep_dispatch_compact,
 * ep_combine_compact, ep_layout_dispatch_compact: one row per received
 * token), ep_zero_padding (zero the alignment rows), the CU-limited mode
 * (ep_set_workgroup_limit / ep_get_workgroup_limit) and the helpers
 * ep_layout_workspace_bytes, ep_layout_dispatch_workspace_bytes, ep_supported
 * and ep_last_error; ep_layout_noalloc
 * runs ep_layout on a fixed scratch array for callers that cannot allocate.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All array arguments are DEVICE pointers owned by the caller; the library
 *   never allocates, frees, copies to the host or synchronises. Every call
 *   only enqueues kernels on `stream` (a hipStream_t passed as void*; NULL
 *   is the default stream) and returns; results are ready when the stream
 *   reaches that point. Calls are stream-ordered and capturable.
 * - Arrays are dense and row-major with the shapes given below. Row pointers
 *   of x, expand_x, expert_out, out and the scale arrays must be 16-byte
 *   aligned; int32 / fp32 arrays 4-byte aligned.
 * - Return value: EP_OK (0) on success, a negative EP_E* code on error.
 *   Arguments are checked on the host before anything is enqueued; on an
 *   error nothing is launched and ep_last_error() returns a message (per
 *   calling thread). No entry point throws or aborts.
 * - Shapes (hidden, topk, dtype) select kernels compiled ahead of time with
 *   those values as template constants; a shape outside the compiled set is
 *   rejected with EP_EUNSUPPORTED before any work (capability gate).
 * - dtype numbering follows the MORI v2 EpDType enumeration ("MORI JIT v2",
 *   section 3.7): bf16 = 0, fp32 = 1, fp8 = 2, fp4x2 = 3.
 *
 * Sources: "DeepEP 整体架构分析" (DeepEP overall architecture), the EPHandle
 * structure and the dispatch / combine data-flow figure; "MORI JIT v2",
 * section 3.5 (invalid configurations are rejected before any work: token
 * bytes 16-byte aligned, topk within one wavefront, receive capacity covers
 * the worst case), section 3.7 (dtype is a transport attribute: dispatch
 * moves bytes, combine reduces and rejects byte dtypes), section 4 (no
 * compile, allocation or host synchronisation on the launch path; graph
 * capture), section 6 (every C entry point reports errors by return value
 * plus a last-error string).
 */
#ifndef EP_MI355X_H
#define EP_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define EP_OK 0
#define EP_EINVAL (-1)        /* an argument is out of range or misaligned        */
#define EP_EUNSUPPORTED (-2)  /* no compiled kernel for this (hidden, topk, dtype) */
#define EP_ECAPACITY (-3)     /* capacity_rows cannot hold the worst case          */
#define EP_EHIP (-4)          /* the HIP runtime reported an error on launch       */

/* Element types (MORI v2 EpDType numbering). */
#define EP_BF16 0
#define EP_FP32 1
#define EP_FP8_E4M3 2
#define EP_FP4X2 3

/* Scores of ep_router. */
#define EP_SOFTMAX 0
#define EP_SIGMOID 1

/* Largest num_sequences of ep_router. */
#define EP_MAX_SEQUENCES 65536

/* Largest in_features of ep_quantized_matmul: a sum of that many products of two 8-bit
 * integers is below 2^31. */
#define EP_MAX_QUANTIZED_WIDTH 131056

/* Largest expert count and top-k the layout kernels accept. */
#define EP_MAX_EXPERTS 1024
#define EP_MAX_TOPK 64

/* Largest num_tokens * topk of ep_moe_layer (128 tokens at top-8). */
#define EP_MOE_MAX_ENTRIES 1024

/*
 * Bytes of device workspace ep_layout needs for (num_tokens, topk,
 * num_experts): per-tile expert histograms and per-tile received-token
 * counts passed between its kernels when num_tokens*topk is above 2^14
 * (smaller inputs take one launch and need none: the result is 0), plus,
 * when there are many tiles per expert, their per-tile prefixes and totals.
 * Returns 0 for out-of-range arguments. The workspace is scratch: its
 * contents on entry do not matter and are overwritten; two ep_layout calls
 * in flight at once must not share one workspace.
 */
size_t ep_layout_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts);

/*
 * Workspace bytes that let ep_layout_dispatch walk a dispatch plan: the
 * layout's own workspace (ep_layout_workspace_bytes), rounded up to 256 bytes,
 * plus 8 bytes per (token, k) entry for the plan. ep_layout_dispatch needs
 * only ep_layout_workspace_bytes; given this much, a batch of more than one
 * layout tile also has the layout write the plan into the tail of the
 * workspace and dispatch follow it (measured on MI355X: prefill step 171.4
 * against 176.4 us, mori_default 47.9 against 49.7; with x evicted from the
 * last-level cache 193.5 against 232.1, 52.9 against 63.5). Results are
 * identical either way. Returns 0 for out-of-range arguments.
 */
size_t ep_layout_dispatch_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t num_experts);

/*
 * Routing layout (DeepEP overall architecture, EPHandle fields
 * num_unaligned_recv_tokens_perpert, psum_num_recv_tokens_per_expert,
 * dst_buffer_slot_idx, recv_src_metadata, num_recv_tokens,
 * num_expanded_tokens; in the dispatch data-flow figure the notify warps count
 * entries per expert and compute each entry's target slot).
 *
 * Inputs
 *   topk_idx          int32 [num_tokens, topk]: expert id of each (t, k);
 *                     an id outside [0, num_experts) masks the entry
 *                     (it gets no slot and is not counted).
 *   num_tokens        T >= 0
 *   topk              K in 1 .. EP_MAX_TOPK (compiled set, see EP_EUNSUPPORTED)
 *   num_experts       E in 1 .. EP_MAX_EXPERTS
 *   expert_alignment  A >= 1: every expert segment is padded to a multiple of A
 *   capacity_rows     rows of the expand buffer the caller will dispatch into;
 *                     must be >= T*K + E*(A-1) (the worst case), else
 *                     EP_ECAPACITY
 * Outputs (device, written in full unless noted)
 *   counts            int32 [E]: unmasked entries routed to each expert
 *   offsets           int32 [E+1]: offsets[0] = 0, offsets[e+1] = offsets[e]
 *                     + A*ceil(counts[e]/A); offsets[E] = num_expanded_tokens
 *   dst_slot          int32 [T, K]: expand row of (t, k), or -1 when masked.
 *                     Inside an expert segment rows are handed out in
 *                     token-major (t, then k) order starting at offsets[e];
 *                     the padding rows of a segment belong to nobody.
 *   recv_src_metadata int32 [T, K+2]: row i describes the i-th token (in
 *                     ascending t) with at least one unmasked entry:
 *                     [t, source rank (always 0 here), dst_slot[t, 0..K-1]].
 *                     Rows i >= *num_recv are left untouched.
 *   num_recv          int32 [1]: number of such tokens (stays on the device)
 *   workspace         device scratch of >= ep_layout_workspace_bytes(T, K, E)
 *   dispatch_plan     optional (NULL: not written), int32 [T*K, 2], 8-byte
 *                     aligned: the order in which ep_dispatch copies rows
 *                     fastest. The entries are cut into tiles of whole tokens,
 *                     floor(W / K) tokens each, where W = 1024 for E <= 256,
 *                     512 for E <= 512 and 256 above. Each tile's span
 *                     lists its unmasked entries by ascending slot as
 *                     (t*K + k, dst_slot[t, k]), then (-1, -1) once per
 *                     masked entry. This array is not part of the pages'
 *                     handle: it is a gfx950-specific write-order aid, and
 *                     every other output is the same with or without it.
 *                     Measured on MI355X (steps with ep_dispatch following
 *                     the plan against token-major): prefill with 470 MB of
 *                     rows 167.5 against 175.9 us with the rows cached,
 *                     190.9 against 231.5 us with them evicted; mori_default
 *                     (1024 tokens) 46.0 against 49.7 and 52.5 against
 *                     63.5 us. The layout pays 0.1-0.4 us for it.
 *   prefetch,         optional read-ahead (NULL and 0: none): device memory
 *   prefetch_bytes    the caller reads next, typically the token rows x
 *                     (and their scale rows) that ep_dispatch copies. The
 *                     layout leaves most compute units idle; workgroups
 *                     added to its launches read one 4-byte word of every
 *                     128-byte line of the first min(prefetch_bytes, 128 MiB)
 *                     bytes with ordinary loads, which brings those lines
 *                     into the last-level cache while the layout runs. It
 *                     reads only inside [prefetch, prefetch + prefetch_bytes),
 *                     writes nothing there and changes no result. Ignored
 *                     under a workgroup cap. The pointer must be 4-byte
 *                     aligned; NULL with nonzero bytes is EP_EINVAL.
 *                     Measured on MI355X (prefill step, 4096 tokens of
 *                     hidden 7168, 58.7 MB of rows): with the rows not in the
 *                     cache the step takes 177 us with the read-ahead against
 *                     191 us without; with the rows cached, 172 against 167
 *                     us (the reads then only add work). Worth asking for
 *                     when x was produced long before dispatch.
 * Results are a pure function of the inputs (no atomics whose order matters).
 */
int ep_layout(const int32_t *topk_idx, int32_t num_tokens, int32_t topk, int32_t num_experts,
              int32_t expert_alignment, int64_t capacity_rows, int32_t *counts,
              int32_t *offsets, int32_t *dst_slot, int32_t *recv_src_metadata,
              int32_t *num_recv, void *workspace, size_t workspace_bytes,
              int32_t *dispatch_plan, const void *prefetch, size_t prefetch_bytes,
              void *stream);

/*
 * Bytes of the library's fixed layout scratch, one copy per GPU (8 MiB):
 * the largest ep_layout_workspace_bytes() that ep_layout_noalloc accepts. It
 * covers batches of up to 4,176,896 (token, k) entries at 256 experts
 * (522,112 tokens at top-8), 1,046,016 at 512 and 261,632 at 1024; batches
 * of at most 2^14 entries need no scratch at all.
 */
#define EP_LAYOUT_SCRATCH_BYTES 8388608 /* 8 MiB */

/*
 * ep_layout without a workspace argument, for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc). Same arguments, outputs, checks and errors as
 * ep_layout; the workspace is instead a fixed device array of
 * EP_LAYOUT_SCRATCH_BYTES inside the library, one copy per GPU, kept until
 * the process ends. The call allocates nothing: on the first call on a GPU it
 * looks up that GPU's copy (with the GPU current), then only enqueues kernels.
 *
 * Extra rules:
 * - `stream` must belong to the current device (EP_EINVAL otherwise).
 * - ep_layout_workspace_bytes(num_tokens, topk, num_experts) must not exceed
 *   EP_LAYOUT_SCRATCH_BYTES (EP_EINVAL, with the sizes in the message).
 * - Every call on one GPU shares that GPU's scratch and nothing in it is
 *   cleared between calls (no word needs to start at zero): two calls in
 *   flight at once on one GPU (on different streams, or overlapping graph
 *   replays) race and may return wrong results. Calls on one stream are
 *   ordered and safe.
 * - The first call on a GPU fails with EP_EHIP if the runtime cannot resolve
 *   the scratch address; a failed lookup is retried on the next call.
 */
int ep_layout_noalloc(const int32_t *topk_idx, int32_t num_tokens, int32_t topk,
                      int32_t num_experts, int32_t expert_alignment, int64_t capacity_rows,
                      int32_t *counts, int32_t *offsets, int32_t *dst_slot,
                      int32_t *recv_src_metadata, int32_t *num_recv, int32_t *dispatch_plan,
                      const void *prefetch, size_t prefetch_bytes, void *stream);

/*
 * Dispatch in the expand layout (DeepEP overall architecture, dispatch copy
 * epilogue writing token data and scale factors; "MORI JIT v2", section 3.7:
 * the payload is moved as bytes whatever its dtype, fp8 / fp4x2 arrive
 * already quantised, and for fp4x2 hidden counts bytes).
 *
 * For every (t, k) with 0 <= dst_slot[t, k] < capacity_rows:
 *   expand_x[dst, :]        = x[t, :]            (bytes of one row)
 *   expand_scales[dst, :]   = x_scales[t, :]     (only if both are non-NULL)
 *   expand_weights[dst]     = topk_weights[t, k] (only if both are non-NULL)
 * Rows no entry points at (alignment padding) are not written. Entries
 * outside [0, capacity_rows) are skipped.
 *
 *   x               EP_BF16: bf16 [T, hidden]; EP_FP32: fp32 [T, hidden];
 *                   EP_FP8_E4M3: e4m3 bytes [T, hidden];
 *                   EP_FP4X2: packed e2m1 pairs, [T, hidden] bytes (2*hidden values)
 *   x_scales        fp32 [T, S] with S = values per row / 128, or NULL; only for
 *                   fp8 and fp4x2 (values per row a multiple of 128). The
 *                   scale rows are optional for both byte dtypes, fp8
 *                   included: the payload travels as bytes either way ("MORI
 *                   JIT v2" section 3.7; its HIP backend moves fp8 rows with
 *                   no scales), so fp8 with x_scales = NULL is accepted and
 *                   moves the rows alone, and the multiple-of-128 rule
 *                   applies only when scales are given. A stricter contract,
 *                   fp8 always with scales, is left to the caller.
 *   topk_weights    fp32 [T, K] or NULL
 *   dst_slot        int32 [T, K], as produced by ep_layout
 *   expand_x        [capacity_rows, hidden] of the same element type as x
 *   expand_scales   fp32 [capacity_rows, S], given exactly when x_scales is
 *   expand_weights  fp32 [capacity_rows] or NULL
 *   dispatch_plan   optional (NULL: token-major order): the plan ep_layout
 *                   wrote in the same call as dst_slot. It changes only the
 *                   order of the copies, never their result. Entries of the
 *                   plan outside [0, T*K) and slots outside
 *                   [0, capacity_rows) are skipped. A plan that does not
 *                   match dst_slot copies what the plan says.
 * Errors: EP_EINVAL for a NULL required pointer, misalignment, row bytes
 * not a multiple of 16, scales for bf16 / fp32 or only one scale pointer;
 * EP_EUNSUPPORTED for (hidden, topk, dtype) outside the compiled set.
 */
int ep_dispatch(const void *x, const float *x_scales, const float *topk_weights,
                const int32_t *dst_slot, int32_t num_tokens, int32_t hidden, int32_t topk,
                int32_t dtype, int64_t capacity_rows, void *expand_x, float *expand_scales,
                float *expand_weights, const int32_t *dispatch_plan, void *stream);

/*
 * Layout and dispatch in one call (the DeepEP overall-architecture page,
 * dispatch data-flow figure: the dispatch kernel's notify warps count per
 * expert and compute each token's target slot before the copy epilogue
 * moves the data). It produces everything ep_layout and ep_dispatch produce,
 * with the same arguments, meanings, checks and errors as those two calls
 * (the dispatch arguments take their slots from this layout). When T*K fits
 * one layout tile (the floor(W / K) tokens of ep_layout's dispatch_plan,
 * W = 1024, 512 or 256 by num_experts: a decode step, say) it runs as a
 * single launch: workgroup 0 ranks all entries and writes the layout's
 * outputs, and the copying workgroups find their entries' slots in their own
 * LDS (with expert_alignment 1 and no workgroup cap, by counting the entries
 * whose (expert id, entry index) is smaller; otherwise by ranking all entries
 * as workgroup 0 does). This saves a launch and the trip of dst_slot through
 * memory. Larger batches run the launches of ep_layout and ep_dispatch (no
 * read-ahead), walking a dispatch plan kept in the workspace when the
 * workspace holds ep_layout_dispatch_workspace_bytes, token-major otherwise. Results are identical either way.
 */
int ep_layout_dispatch(const int32_t *topk_idx, int32_t num_tokens, int32_t topk,
                       int32_t num_experts, int32_t expert_alignment, int64_t capacity_rows,
                       int32_t *counts, int32_t *offsets, int32_t *dst_slot,
                       int32_t *recv_src_metadata, int32_t *num_recv, void *workspace,
                       size_t workspace_bytes, const void *x, const float *x_scales,
                       const float *topk_weights, int32_t hidden, int32_t dtype, void *expand_x,
                       float *expand_scales, float *expand_weights, void *stream);

/*
 * Gather combine (DeepEP overall architecture, combine reduce epilogue
 * weighting expert outputs by topk_weights and adding a bias; "MORI JIT v2",
 * section 3.7: combine reduces bf16 or fp32 rows, writes the same type, and
 * rejects byte dtypes).
 *
 * For every token t and channel h:
 *   acc = +0.0f
 *   for k = 0 .. K-1 with 0 <= dst_slot[t, k] < capacity_rows:
 *       acc = acc + w[t, k] * float(expert_out[dst_slot[t, k], h])
 *   if bias: acc = acc + float(bias[t, h])
 *   out[t, h] = acc stored as dtype (bf16: round to nearest even)
 * Each product and each sum is rounded to binary32 on its own (no fused
 * multiply-add), in k order, so the result is a pure function of the inputs.
 * w[t, k] = topk_weights[t, k], or 1 when topk_weights is NULL.
 *
 *   expert_out      [capacity_rows, hidden] of dtype EP_BF16 or EP_FP32
 *   topk_weights    fp32 [T, K] or NULL
 *   bias            [T, hidden] of the same dtype, or NULL
 *   dst_slot        int32 [T, K]
 *   out             [T, hidden] of the same dtype; every row is written
 * Errors: EP_EINVAL for a byte dtype (fp8 / fp4x2), NULL or misaligned
 * pointers; EP_EUNSUPPORTED for (hidden, topk, dtype) outside the compiled set.
 */
int ep_combine(const void *expert_out, const float *topk_weights, const void *bias,
               const int32_t *dst_slot, int32_t num_tokens, int32_t hidden, int32_t topk,
               int32_t dtype, int64_t capacity_rows, void *out, void *stream);

/*
 * Non-expand dispatch (DeepEP overall architecture: EPHandle do_expand =
 * false; the dispatch copy epilogue writes recv_x, recv_topk_idx and
 * recv_topk_weights): one row per received token instead of one per
 * (token, k). In a world of one the received tokens are those with an
 * unmasked entry, in ascending order, as ep_layout lists them in
 * recv_src_metadata. For i < *num_recv, with t = recv_src_metadata[i][0]:
 *   recv_x[i]            = x[t]                      (bytes of one row)
 *   recv_scales[i]       = x_scales[t]               (only if both are non-NULL)
 *   recv_topk_idx[i][k]  = dst_slot[t][k] >= 0 ? topk_idx[t][k] : -1
 *   recv_topk_weights[i] = topk_weights[t]           (only if both are non-NULL)
 * Rows i >= *num_recv are not written. x, x_scales, dtype and hidden as for
 * ep_dispatch; recv_x [T, hidden], recv_scales [T, S], recv_topk_idx int32
 * [T, K], recv_topk_weights fp32 [T, K] (room for every token); topk_idx,
 * dst_slot, recv_src_metadata and num_recv as written by ep_layout.
 * Shapes are run-time values (no capability gate). Errors: EP_EINVAL.
 */
int ep_dispatch_compact(const void *x, const float *x_scales, const int32_t *topk_idx,
                        const float *topk_weights, const int32_t *dst_slot,
                        const int32_t *recv_src_metadata, const int32_t *num_recv,
                        int32_t num_tokens, int32_t hidden, int32_t topk, int32_t dtype,
                        void *recv_x, float *recv_scales, int32_t *recv_topk_idx,
                        float *recv_topk_weights, void *stream);

/*
 * Layout and non-expand dispatch in one call (the DeepEP overall-architecture
 * page: EPHandle do_expand = false, with the dispatch kernel's notify warps
 * computing the layout before its copy epilogue writes recv_x, recv_topk_idx
 * and recv_topk_weights). It produces everything ep_layout and
 * ep_dispatch_compact produce, with the same arguments, meanings, checks and
 * errors as those two calls (the dispatch reads this layout's dst_slot,
 * recv_src_metadata and num_recv). When T*K fits one layout tile (the
 * floor(W / K) tokens of ep_layout's dispatch_plan: a decode step, say) it
 * runs as a single launch in which every workgroup ranks the entries and the
 * received tokens itself and workgroup 0 writes the layout's outputs; larger
 * batches run the launches of ep_layout and ep_dispatch_compact. Results are
 * identical either way.
 */
int ep_layout_dispatch_compact(const int32_t *topk_idx, int32_t num_tokens, int32_t topk,
                               int32_t num_experts, int32_t expert_alignment,
                               int64_t capacity_rows, int32_t *counts, int32_t *offsets,
                               int32_t *dst_slot, int32_t *recv_src_metadata, int32_t *num_recv,
                               void *workspace, size_t workspace_bytes, const void *x,
                               const float *x_scales, const float *topk_weights, int32_t hidden,
                               int32_t dtype, void *recv_x, float *recv_scales,
                               int32_t *recv_topk_idx, float *recv_topk_weights, void *stream);

/*
 * Non-expand combine (DeepEP overall architecture: combine reduce epilogue
 * with bias, do_expand = false). The expert side returns one row per
 * received token with that token's experts already reduced, so in a world
 * of one combine only puts rows back in token order and adds the bias:
 *   out[t] = float(expert_out[i]) + float(bias[t])  for t = recv_src_metadata[i][0]
 *   out[t] = +0.0 + float(bias[t])                   for a token with no unmasked entry
 * in binary32, one rounded add per value, stored in the rows' type (bf16:
 * round to nearest even; fp32: as is); without a bias, the row's bits, or
 * +0. dtype EP_BF16 or EP_FP32 ("MORI JIT v2" section 3.7: combine takes bf16
 * or fp32 rows and writes the same type). expert_out [T, hidden] (rows
 * >= *num_recv are not read), bias [T, hidden] of the same type or NULL, out
 * [T, hidden] of the same type, every row written. Errors: EP_EINVAL (byte
 * dtypes and unknown dtypes rejected, NULL or misaligned pointers).
 */
int ep_combine_compact(const void *expert_out, const void *bias, const int32_t *dst_slot,
                       const int32_t *recv_src_metadata, const int32_t *num_recv,
                       int32_t num_tokens, int32_t hidden, int32_t topk, int32_t dtype, void *out,
                       void *stream);

/*
 * Optional clean-up of the expand layout: zero the alignment padding rows of
 * every expert segment, rows [offsets[e] + counts[e], offsets[e+1]), so a
 * consumer that walks whole aligned segments (DeepEP overall architecture,
 * EPHandle expert_alignment; the pages leave padding content open and
 * ep_dispatch does not write it) reads zeros there. Real rows are untouched.
 *
 *   expand_x        [capacity_rows, row_bytes] bytes (row_bytes a positive multiple of 16)
 *   expand_scales   fp32 [capacity_rows, scale_cols], or NULL with scale_cols = 0
 *   expand_weights  fp32 [capacity_rows] or NULL
 *   counts, offsets int32 [E] and [E+1] as written by ep_layout (device)
 *   expert_alignment the A given to ep_layout (A = 1: nothing to do)
 * Rows at or beyond capacity_rows are never written. Errors: EP_EINVAL for
 * out-of-range scalars, NULL or misaligned pointers.
 */
int ep_zero_padding(void *expand_x, int64_t row_bytes, float *expand_scales, int64_t scale_cols,
                    float *expand_weights, const int32_t *counts, const int32_t *offsets,
                    int32_t num_experts, int32_t expert_alignment, int64_t capacity_rows,
                    void *stream);

/*
 * The experts' operators
 * ----------------------
 * What lies between dispatch and combine, on the arrays those two use. Rows
 * of expert e are [offsets[e], offsets[e] + counts[e]) of an expand buffer of
 * capacity_rows rows (int32 [E] and [E+1] as written by ep_layout, read on
 * the device); other rows (alignment padding, the buffer's tail) are neither
 * read nor written, and the part of a span outside [0, capacity_rows) is
 * skipped. With one expert, counts and offsets may both be NULL: then every
 * row of the buffer belongs to it. Shapes are run-time values (no capability
 * gate); a workgroup cap of the stream applies and changes no result.
 * Results are a pure function of the inputs. No operand may overlap an
 * output unless it is said below.
 *
 * Weights are one row-major matrix [rows, width] per expert, of dtype
 *   EP_BF16      bf16, no scales; width a multiple of 8
 *   EP_FP8_E4M3  e4m3 bytes; width a multiple of 128
 *   EP_FP4X2     e2m1 pairs, width / 2 bytes a row: the value of even index is
 *                in a byte's low half; width (counted in values, here and
 *                below) a multiple of 128
 * and for the last two one fp32 scale per 128 values of a row, [E, rows,
 * width / 128]: the weight is code * scale. One expert's matrix is below
 * 2^31 bytes. Weight products are summed in binary32 per 128 values, the sum
 * is scaled, and the scaled sums are added in binary32: no weight is rounded.
 */

/*
 * Bytes of device workspace ep_moe_layer needs: the list of active experts
 * and their entries, and 4 * intermediate bytes per (token, k) entry. 0 for
 * out-of-range arguments (and for no tokens). Scratch: its contents on entry
 * do not matter; two calls in flight at once (two streams, two graphs that
 * may replay together) must not share one.
 */
size_t ep_moe_layer_workspace_bytes(int32_t num_tokens, int32_t topk, int32_t intermediate);

/*
 * A whole expert layer for a few tokens (a decode step), in two launches,
 * without layout, dispatch and combine: per token t and k with e =
 * topk_idx[t, k] in [0, num_experts) (other ids mask the entry)
 *   [gate | up] = w_in[e] x[t]          (rows [0, I) of w_in are gate's)
 *   h           = gate / (1 + exp(-gate)) * up
 *   out[t]      = sum over k of topk_weights[t, k] * (w_out[e] h)  (+ bias[t])
 * in binary32 (gates below -87 as in ep_swiglu) with the k in ascending order,
 * rounded once to bf16; h is carried as a sum of two bf16 values (2^-17
 * relative; above bf16's largest value it is infinite), so an infinite weight
 * or scale of w_out gives NaN. An id may occur twice in a token: both entries
 * count. A token without unmasked entries gets bias[t], or +0.
 *
 *   x             bf16 [num_tokens, hidden]
 *   topk_idx      int32 [num_tokens, topk]
 *   topk_weights  fp32 [num_tokens, topk], or NULL for 1
 *   bias          bf16 [num_tokens, hidden] (a shared expert's output, a
 *                 residual) or NULL; may be out
 *   w_in          [num_experts, 2 * intermediate, hidden] of weight_dtype
 *   w_out         [num_experts, hidden, intermediate] of weight_dtype
 *   out           bf16 [num_tokens, hidden], every row written
 *   workspace     >= ep_moe_layer_workspace_bytes, 16-byte aligned
 * hidden and intermediate are multiples of 8 (128 for scaled weights).
 * Errors: EP_EUNSUPPORTED for num_tokens * topk > EP_MOE_MAX_ENTRIES (use
 * layout, dispatch, ep_expert_matvec or the caller's own grouped product, and
 * combine);
 * EP_EINVAL otherwise.
 */
int ep_moe_layer(const void *x, const int32_t *topk_idx, const float *topk_weights,
                 const void *bias, const void *w_in, const float *w_in_scales, const void *w_out,
                 const float *w_out_scales, int32_t num_tokens, int32_t hidden,
                 int32_t intermediate, int32_t topk, int32_t num_experts, int32_t weight_dtype,
                 void *out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Per-expert matrix-vector products for a few rows per expert:
 *   y[r] = w[e] x[r]  for the rows r of each expert e
 * summed in binary32, rounded once. Any number of rows is right; beyond 32
 * per expert (16 for a few small matrices) the weights are read again for
 * every 32, from cache where they fit.
 *
 *   x             bf16 [capacity_rows, in_features], an expand buffer
 *   w             [num_experts, out_features, in_features] of weight_dtype
 *   y             [capacity_rows, out_features] of y_dtype (EP_BF16, EP_FP32)
 * in_features and out_features are multiples of 8 (in_features of 128 for
 * scaled weights). One dense matrix: num_experts 1 and NULL counts, offsets.
 * Errors: EP_EINVAL.
 */
int ep_expert_matvec(const void *x, const void *w, const float *w_scales, const int32_t *counts,
                     const int32_t *offsets, int32_t num_experts, int64_t capacity_rows,
                     int32_t in_features, int32_t out_features, int32_t weight_dtype, void *y,
                     int32_t y_dtype, void *stream);

/*
 * The experts' gated activation, and an 8-bit checkpoint of its input for
 * ep_swiglu_backward. For the experts' rows [gate | up] of gate_up:
 *   h = gate / (1 + exp(-gate)) * up
 * in binary32, rounded once to the rows' type (a gate below -87, where
 * 1 / (1 + exp(-gate)) is no normal binary32 number, keeps its h); and, unless checkpoint and
 * checkpoint_scales are NULL, per 128 values of the row the scale 2^p, p the
 * smallest integer >= -126 that keeps the group's largest finite magnitude
 * within 448 * 2^p, and the e4m3 codes of value / 2^p (round to nearest
 * even). An infinity or NaN becomes the code NaN.
 *
 *   gate_up             [capacity_rows, 2 * intermediate] of dtype (EP_BF16, EP_FP32)
 *   h                   [capacity_rows, intermediate] of dtype
 *   checkpoint          e4m3 [capacity_rows, 2 * intermediate] or NULL
 *   checkpoint_scales   fp32 [capacity_rows, 2 * intermediate / 128] or NULL
 * intermediate is a multiple of 128, or without a checkpoint of 8.
 * Errors: EP_EINVAL.
 */
int ep_swiglu(const void *gate_up, const int32_t *counts, const int32_t *offsets,
              int32_t num_experts, int64_t capacity_rows, int32_t intermediate, int32_t dtype,
              void *h, void *checkpoint, float *checkpoint_scales, void *stream);

/*
 * Backward pass of ep_swiglu from its checkpoint: with gate and up = code *
 * scale, s = 1 / (1 + exp(-gate)), for the experts' rows
 *   d_gate_up = [dh * up * s * (1 + gate * (1 - s)) | dh * gate * s]
 *   h         = gate * s * up   (unless h is NULL: for the next weight gradient)
 * in binary32 (gates below -87 as in ep_swiglu), rounded once. Any finite fp32
 * scales are accepted.
 *
 *   dh          [capacity_rows, intermediate] of dtype (EP_BF16, EP_FP32)
 *   d_gate_up   [capacity_rows, 2 * intermediate] of dtype
 *   h           [capacity_rows, intermediate] of dtype or NULL; may be dh
 * intermediate is a multiple of 128. Errors: EP_EINVAL.
 */
int ep_swiglu_backward(const void *dh, const void *checkpoint, const float *checkpoint_scales,
                       const int32_t *counts, const int32_t *offsets, int32_t num_experts,
                       int64_t capacity_rows, int32_t intermediate, int32_t dtype, void *d_gate_up,
                       void *h, void *stream);

/*
 * Weight gradient of the experts' products:
 *   dw[e] = previous[e] + sum over the rows r of expert e of dy[r]^T x[r]
 * with x kept in bf16 or in 8 bits (rows as dispatch moves them, or a
 * checkpoint): x[r] = code * x_scales[r], rounded to binary32 (and to a
 * multiple of 2^-133, which matters below 2^-110). Summed in binary32, rounded
 * once. Scales that are powers of two from 2^-64 to 2^64, as ep_swiglu's are
 * but for tiny rows, take one pass of the matrix cores, others three (64
 * experts of 128 rows 1080 and 2340 us on MI355X). An expert without rows gets
 * previous[e], or zeros.
 *
 *   dy          bf16 [capacity_rows, out_features]
 *   x           bf16 or e4m3 (x_dtype) [capacity_rows, in_features]
 *   x_scales    fp32 [capacity_rows, in_features / 128] for e4m3, or NULL (scale 1)
 *   previous    [num_experts, out_features, in_features] of dw_dtype, NULL
 *               for zeros, or dw itself (accumulate in place)
 *   dw          [num_experts, out_features, in_features] of dw_dtype
 *               (EP_BF16, EP_FP32), every element written
 * out_features is a multiple of 8; in_features of 8 (bf16), 16 (e4m3) or 128
 * (with scales). Errors: EP_EINVAL.
 */
int ep_expert_wgrad(const void *dy, const void *x, const float *x_scales, const int32_t *counts,
                    const int32_t *offsets, int32_t num_experts, int64_t capacity_rows,
                    int32_t out_features, int32_t in_features, int32_t x_dtype,
                    const void *previous, void *dw, int32_t dw_dtype, void *stream);

/*
 * The router's operators
 * ----------------------
 * From a router's logits to the ids and weights that ep_layout, ep_dispatch,
 * ep_combine and ep_moe_layer take, with the losses that keep the experts
 * evenly used, and back. Shapes are run-time values (no capability gate); a
 * workgroup cap of the stream applies and changes no result. Results are a
 * pure function of the inputs (sums over tokens in a fixed order). No operand
 * may overlap an output.
 */

/*
 * Bytes of device workspace ep_router needs for counts and losses: partial
 * sums per tile of tokens and sequence. 0 for out-of-range arguments. Never
 * fewer for more tokens, experts or sequences: a buffer for the largest call
 * serves every smaller one.
 * Scratch: its contents on entry do not matter; two calls in flight at once
 * (two streams, two graphs that may replay together) must not share one.
 */
size_t ep_router_workspace_bytes(int32_t num_tokens, int32_t num_experts, int32_t num_sequences);

/*
 * Per token t, with its logits l and the scores
 *   EP_SOFTMAX  s_e = exp(l_e) / sum over j of exp(l_j)
 *   EP_SIGMOID  s_e = 1 / (1 + exp(-l_e))
 * topk_idx[t] are the topk experts of the largest l_e, or with select_bias of
 * the largest s_e + select_bias[e], in descending order; of equal ones the
 * lowest id first. s + bias is compared as if without rounding errors: sums
 * that binary32 cannot tell apart are computed again in binary64. An expert whose
 * logit is -infinity or NaN, or whose bias is -infinity or NaN, is not chosen; where no
 * more are left, and for a token whose token_mask is 0, the id is -1. A NaN logit
 * leaves out no other expert: for the choice the others' scores are those of the row
 * without it, and experts at +infinity share a softmax score of 1. (Weights and losses
 * follow their formulas: NaN where a sum over the row, or a chosen logit, makes it so.)
 * Then, for every id in [0, num_experts) of a token
 *   topk_weights[t, k] = scale * s_i                          (normalize = 0)
 *                      = scale * s_i / sum over the token's ids of s_j  (else)
 * and 0 for other ids. With given != 0, topk_idx is an input instead (ids
 * outside [0, num_experts) mask their entry, an id may occur twice).
 *
 * Unless counts is NULL, over the tokens t of each sequence s, those in
 * [seq_offsets[s], seq_offsets[s + 1]), that have an id in [0, num_experts)
 * (n_s tokens; others, masked ones among them, take no part):
 *   counts[s, e]   = number of their entries with id e
 *   seq_tokens     = n_s for each s, then the number of sequences with n_s > 0
 *                    (S'), then the sum of all n_s (n)
 *   balance_loss   = 1/S' sum over s, e of f_se P_se, f_se = counts[s, e] *
 *                    num_experts / (topk * n_s), P_se = mean over t of p_te,
 *                    p_te = s_e / sum over j of s_j: 1 for even use
 *   z_loss         = mean over the n tokens of (log sum over e of exp(l_e))^2
 * Losses of no tokens are 0. With one sequence, counts are ep_layout's.
 * Scores in binary32 (exponentials below 2^-126 may count as 0); sums over tokens in binary32 over at most 256 tokens, and
 * in binary64 beyond. A token none of whose ids' logits is above -infinity has
 * weights 0; one whose logits are all -infinity has p = 0 and log sum 0 too.
 *
 *   logits         [num_tokens, num_experts] of dtype (EP_BF16, EP_FP32)
 *   select_bias    fp32 [num_experts] or NULL; not with given
 *   token_mask     uint8 [num_tokens] or NULL for no masked token; not with
 *                  given (mask the ids)
 *   seq_offsets    int32 [num_sequences + 1], ascending, or NULL for one sequence
 *                  of all tokens; tokens outside [seq_offsets[0],
 *                  seq_offsets[num_sequences]) belong to none
 *   topk           1 .. EP_MAX_TOPK, at most num_experts unless given
 *   topk_idx       int32 [num_tokens, topk], written unless given
 *   topk_weights   fp32 [num_tokens, topk] or NULL
 *   counts         int32 [num_sequences, num_experts] or NULL, with
 *   seq_tokens     int32 [num_sequences + 2]: both or neither
 *   balance_loss   fp32 [1] or NULL; with counts
 *   z_loss         fp32 [1] or NULL; with counts, and EP_SOFTMAX only
 *   workspace      >= ep_router_workspace_bytes, 16-byte aligned; only with counts
 * Errors: EP_EINVAL.
 */
int ep_router(const void *logits, const float *select_bias, const uint8_t *token_mask,
              const int32_t *seq_offsets, int32_t num_tokens, int32_t num_experts, int32_t topk,
              int32_t num_sequences, int32_t dtype, int32_t scoring, int32_t normalize, float scale,
              int32_t given, int32_t *topk_idx, float *topk_weights, int32_t *counts,
              int32_t *seq_tokens, float *balance_loss, float *z_loss, void *workspace,
              size_t workspace_bytes, void *stream);

/*
 * Backward pass of ep_router: the logits' gradient, with the ids and counts
 * held constant, from those of topk_weights, balance_loss and z_loss (each
 * may be NULL: 0). topk_idx, counts and seq_tokens as the forward pass took
 * or wrote them (counts and seq_tokens may be NULL without a loss gradient);
 * dtype, scoring, normalize and scale as given to it. Per token, with dw =
 * scale * d_topk_weights, s and p as above and q_k = s_k / sum over the
 * token's ids of s_j, summed over the entries of an id:
 *   EP_SOFTMAX, normalize   q_k (dw_k - sum over j of q_j dw_j)
 *   EP_SOFTMAX              p_e (dp_e - sum over j of p_j dp_j), dp_i = dw_i
 *   EP_SIGMOID, normalize   q_k (1 - s_k) (dw_k - sum over j of q_j dw_j)
 *   EP_SIGMOID              s_k (1 - s_k) dw_k
 * and for a token of sequence s that takes part, with g_e = d_balance_loss *
 * num_experts * counts[s, e] / (topk n_s^2 S'):
 *   p_e (g_e - sum over j of p_j g_j) (EP_SIGMOID: times 1 - s_e)
 *   2 d_z_loss / n * log sum exp * p_e
 * in binary32, rounded once. The logits of a token without ids get 0.
 *
 *   d_topk_weights fp32 [num_tokens, topk] or NULL
 *   d_balance_loss fp32 [1] or NULL
 *   d_z_loss       fp32 [1] or NULL; EP_SOFTMAX only
 *   d_logits       [num_tokens, num_experts] of dtype, every element written
 * Errors: EP_EINVAL.
 */
int ep_router_backward(const void *logits, const int32_t *topk_idx, const int32_t *seq_offsets,
                       const int32_t *counts, const int32_t *seq_tokens,
                       const float *d_topk_weights, const float *d_balance_loss,
                       const float *d_z_loss, int32_t num_tokens, int32_t num_experts,
                       int32_t topk, int32_t num_sequences, int32_t dtype, int32_t scoring,
                       int32_t normalize, float scale, void *d_logits, void *stream);

/*
 * The experts' products in 8-bit integers
 * ---------------------------------------
 * Rows and weights as 8-bit integers with one fp32 scale per row of the
 * expand buffer (per token) and per row of a weight matrix (per output
 * channel). Rules of the experts' operators above. A layer is ep_dispatch
 * (of rows already quantised, or before it), ep_quantize_rows,
 * ep_quantized_matmul, ep_swiglu_quantize, ep_quantized_matmul, ep_combine.
 * Quantised rows move through ep_dispatch as EP_FP8_E4M3 bytes: with
 * scale_cols = hidden / 128 equal copies of a row's scale they are its scale rows.
 */

/*
 * Rows to 8-bit integers, one scale per row, for the experts' rows:
 *   a = max(2^-100, largest magnitude of the row)
 *   scales[r, :] = a / 127                (scale_cols equal copies)
 *   codes[r, i]  = x[r, i] * (127 / a), rounded to the nearest integer, halves to even
 * where 127 / a is rounded to binary32 and its product with x is not rounded
 * before the integer: the codes, from -127 to 127, are exactly determined. A
 * row that holds an infinity or NaN gets the scale NaN and codes 0, so that
 * its products are NaN.
 *
 *   x           [capacity_rows, width] of dtype (EP_BF16, EP_FP32)
 *   codes       int8 [capacity_rows, width]
 *   scales      fp32 [capacity_rows, scale_cols]
 * width is a multiple of 16; scale_cols in 1 .. 2^20. One dense matrix (token
 * rows, or a weight matrix): num_experts 1 and NULL counts, offsets. Errors: EP_EINVAL.
 */
int ep_quantize_rows(const void *x, const int32_t *counts, const int32_t *offsets,
                     int32_t num_experts, int64_t capacity_rows, int32_t width, int32_t dtype,
                     void *codes, float *scales, int32_t scale_cols, void *stream);

/*
 * The experts' gated activation, quantised: ep_quantize_rows of
 *   h = gate / (1 + exp(-gate)) * up
 * in binary32 (gates below -87 as in ep_swiglu), h not rounded to the rows'
 * type in between. A code is that of h as binary32 rounds it: where h lies
 * between two codes (one in a million) it may be the other neighbour of what
 * exact arithmetic gives.
 *
 *   gate_up     [capacity_rows, 2 * intermediate] of dtype (EP_BF16, EP_FP32)
 *   codes       int8 [capacity_rows, intermediate]
 *   scales      fp32 [capacity_rows, scale_cols]
 * intermediate is a multiple of 16. Errors: EP_EINVAL.
 */
int ep_swiglu_quantize(const void *gate_up, const int32_t *counts, const int32_t *offsets,
                       int32_t num_experts, int64_t capacity_rows, int32_t intermediate,
                       int32_t dtype, void *codes, float *scales, int32_t scale_cols,
                       void *stream);

/*
 * Per-expert products of 8-bit integers, for any number of rows:
 *   y[r, n] = x_scales[r, 0] * w_scales[e, n] * sum over k of x[r, k] w[e, n, k]
 * for the rows r of each expert e. The sum is exact in 32 bits (all 256 codes
 * are allowed); it is rounded to binary32, scaled by the row's and then the
 * channel's scale, and rounded once to y's type.
 *
 *   x             int8 [capacity_rows, in_features], an expand buffer
 *   x_scales      fp32 [capacity_rows, x_scale_cols], of which the first column is read
 *   w             int8 [num_experts, out_features, in_features]; one expert's
 *                 matrix is below 2^31 bytes
 *   w_scales      fp32 [num_experts, out_features]
 *   y             [capacity_rows, out_features] of y_dtype (EP_BF16, EP_FP32)
 * in_features is a multiple of 16 up to EP_MAX_QUANTIZED_WIDTH, out_features
 * a multiple of 8 up to 2^23. One dense matrix: num_experts 1 and NULL counts, offsets. Errors:
 * EP_EINVAL.
 */
int ep_quantized_matmul(const void *x, const float *x_scales, int32_t x_scale_cols, const void *w,
                        const float *w_scales, const int32_t *counts, const int32_t *offsets,
                        int32_t num_experts, int64_t capacity_rows, int32_t in_features,
                        int32_t out_features, void *y, int32_t y_dtype, void *stream);

/*
 * CU-limited mode ("MORI JIT v2" section 5.1: geometry buckets prefer the
 * smaller workgroup count when times are close, because compute units left
 * free overlap with the expert GEMM, and the workgroup count never exceeds the
 * CU count; the EpCfg default of sections 3.2 and 3.5 is 64 workgroups. DeepEP overall
 * architecture, design goals: communication on a few SMs, 4 to 64).
 *
 * Caps every kernel this library launches on `stream` (a hipStream_t; NULL
 * is the null stream) at max_workgroups workgroups, each sized to keep one
 * compute unit busy (1024 threads; 512 for combine; the experts' operators
 * keep their own 256 to 1024), whose waves loop over the work; the other compute units stay free for kernels on other streams.
 * Results are identical with and without a cap. max_workgroups = 0 removes
 * the cap (the default: grids cover all work with 256-thread workgroups);
 * values above the current device's compute-unit count are clamped to it.
 * The cap is kept per stream handle, process-wide, until changed: clear it
 * (0) before destroying the stream, since HIP may reuse the handle.
 * Thread-safe; takes effect for launches made after it returns. Errors:
 * EP_EINVAL for max_workgroups < 0, EP_EHIP if the compute-unit count cannot
 * be read (no device).
 */
int ep_set_workgroup_limit(void *stream, int32_t max_workgroups);

/* The cap in effect for `stream` (after clamping), or 0 if none; EP_EHIP only if the
 * registry's lock cannot be taken. */
int ep_get_workgroup_limit(void *stream);

/* Message for the last failed call on the calling thread ("" if none). */
const char *ep_last_error(void);

/*
 * 1 if (hidden, topk, dtype) has compiled kernels for the given pass
 * (0 = layout, which ignores hidden and dtype; 1 = dispatch; 2 = combine),
 * else 0. Never fails.
 */
int ep_supported(int32_t pass, int32_t hidden, int32_t topk, int32_t dtype);

#ifdef __cplusplus
}
#endif

#endif /* EP_MI355X_H */
