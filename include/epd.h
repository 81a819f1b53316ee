/*
 * epd.h -- C ABI of libepd: single-GPU MoE expert-parallel token permute and
 * unpermute for GB300 (sm_103a).
 *
 * The path, in the order a caller runs it on one stream:
 *   1. ep_dispatch_layout  counts per expert / simulated rank / simulated RDMA
 *                          node and the is_token_in_rank mask;
 *   2. ep_scan_offsets     expert_start_loc = exclusive prefix sum of the counts;
 *   3. ep_permute          ep_scatter: token rows into the expert-contiguous
 *                          buffer, with m_indices and output_index;
 *   4. ep_unpermute        combine: the topk-weighted sum of each token's expert
 *                          output rows, accumulated in fp32.
 * ep_dispatch_layout_offsets runs steps 1 and 2 in one launch, and ep_dispatch
 * steps 1 to 3 in one call (a single kernel for a decode-sized batch).
 * Around them: ep_route makes the picks and weights from router logits, and
 * ep_expert_matmul is the experts' product between steps 3 and 4; ep_route_backward,
 * ep_expert_matmul_dgrad, ep_expert_matmul_wgrad and ep_unpermute_backward are their
 * gradients and the combine's.
 * Nothing in between goes back to the host: every count, offset and total stays
 * in device memory, and the permuted buffer is sized at the T*k upper bound.
 *
 * Conventions shared by every call:
 *   - The caller owns all memory. libepd never allocates or frees device or
 *     host memory. Every pointer argument except the stream is a device
 *     pointer unless stated otherwise.
 *   - Every call is asynchronous on the caller's stream, does not synchronise
 *     and touches no host memory (the stream replaces DeepEP's previous_event /
 *     async_finish pair).
 *   - The return value reports argument errors, found on the host before any
 *     launch (EPD_ERR_INVALID_ARG, EPD_ERR_UNSUPPORTED), and launch errors
 *     (EPD_ERR_CUDA). A call that returns an error has launched nothing.
 *   - Errors that depend on the data (an expert id outside [-1, E), a slot
 *     outside the buffer, a look-back wait that gave up) are written to the
 *     caller's device word `status` with an atomic compare-and-swap from 0, so
 *     the first error sticks until the caller clears the word. Kernels never
 *     trap: the offending pair is skipped and the call completes.
 *   - Kernels are launched with programmatic dependent launch: a kernel may
 *     start while the kernel before it on the stream drains, and waits
 *     (griddepcontrol.wait) before it reads what that kernel may write; every
 *     libepd kernel waits before it lets its own dependents start. Calls on one
 *     stream may follow each other in any order on one workspace -- two layout
 *     calls back to back included: a layout kernel takes its tile ticket before
 *     that wait from a counter that every call returns to zero, and reads the
 *     rest of the workspace only after it.
 *   - Sizes: T = num_tokens >= 0, k = num_topk in [0, EPD_MAX_TOPK],
 *     E = num_experts in [1, EPD_MAX_EXPERTS], R = num_ranks with E % R == 0,
 *     N = num_rdma_ranks with R % N == 0, T*k <= INT32_MAX.
 *     Expert e lives on simulated rank e / (E/R); rank r on node r / (R/N).
 *
 * Page references (page title, section):
 *   [P1] "参考sglang代码，重构vllm021中EP高吞吐代码，消除空泡问题"
 *   [P2] "高性能专家并行（EP）内核解剖学解读"
 *   [P3] "[MoE] Deepseek的All-to-all通信: DeepEP代码解读"
 */
#ifndef EPD_H
#define EPD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define EPD_API __attribute__((visibility("default")))
#else
#define EPD_API
#endif

/* Same type as the CUDA runtime's cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *epd_stream_t;

typedef enum {
    EPD_OK = 0,
    EPD_ERR_INVALID_ARG = 1,    /* bad size, null or misaligned pointer, mismatched workspace */
    EPD_ERR_UNSUPPORTED = 2,    /* valid but beyond a documented limit */
    EPD_ERR_CUDA = 3,           /* a CUDA call failed; epd_last_cuda_error() has the cause */
    EPD_ERR_INVALID_EXPERT = 4, /* (status word) topk_idx held an id outside [-1, E) */
    EPD_ERR_TIMEOUT = 5,        /* (status word) a bounded wait gave up (look-back, products) */
    EPD_ERR_CAPACITY = 6,       /* (status word) a slot fell outside [0, capacity_rows), or a
                                   position or page outside the cache */
    EPD_ERR_NONFINITE = 7,      /* (status word) a router logit was NaN or +inf, or a bias NaN */
} epd_status_t;

typedef enum {
    EPD_BF16 = 0,      /* rows of H bfloat16 values (2H bytes), H % 8 == 0 */
    EPD_FP8_E4M3 = 1,  /* rows of H float8_e4m3fn values (H bytes) plus H/128 fp32
                          scales per row, H % 128 == 0 */
    EPD_F32 = 2,       /* float32 (router logits) */
} epd_dtype_t;

#define EPD_MAX_EXPERTS 4096
#define EPD_MAX_TOPK 64
#define EPD_MAX_ALIGNMENT 4096

/* Human-readable name of a status code (static string; never NULL). */
EPD_API const char *epd_status_string(int code);

/* Version of this ABI: major * 10000 + minor * 100 + patch. */
EPD_API int epd_version(void);

/*
 * The cudaError_t code of the last CUDA failure seen by a libepd call on this
 * host thread (0 if none). libepd reads and clears the CUDA runtime's
 * last-error state when a launch fails, so the caller's own error checks are
 * not disturbed; this is where the cause is kept.
 */
EPD_API int epd_last_cuda_error(void);

/*
 * Workspace size in bytes for one layout -> permute chain over T tokens, k
 * picks, E experts, R ranks and N nodes. The workspace holds the per-pair rank
 * inside its expert (T*k int32), the per-expert counts and, for batches beyond
 * one thread-block cluster, the per-tile state of the layout's single-pass
 * look-back (whose count rows, when the batch runs as several clusters, hold the
 * counts each cluster publishes). Returns 0 for invalid sizes. Host-only
 * arithmetic.
 */
EPD_API size_t epd_workspace_bytes(int num_tokens, int num_topk, int num_experts, int num_ranks,
                           int num_rdma_ranks);

/*
 * Zero-fills `workspace` (device, `bytes` long) on `stream`. A workspace must
 * be zero-filled once before its first use; the layout call keeps it reusable
 * from then on, for calls of any shape that fits (its look-back state words and
 * the counts clusters publish are tagged with a call counter and a mark no other
 * workspace data carries). A
 * workspace serves one stream at a time: calls on different streams that
 * overlap on the GPU and share a workspace race.
 */
EPD_API epd_status_t epd_workspace_init(void *workspace, size_t bytes, epd_stream_t stream);

/*
 * Step 1 -- dispatch layout. [P3] "Dispatch", get_dispatch_layout docstring:
 * from topk_idx [T, k] int64 (row-major; -1 = no selection) compute
 *   tokens_per_expert    [E] int32: number of (t, j) with topk_idx[t, j] == e;
 *   tokens_per_rank      [R] int32: number of tokens with a pick on rank r
 *                                   (a token counts once per rank);
 *   tokens_per_rdma_rank [N] int32: number of tokens with a pick on node n
 *                                   (once per node); may be NULL (DeepEP
 *                                   returns None for one node);
 *   is_token_in_rank  [T, R] uint8: 1 if token t has a pick on rank r, else 0
 *                                   (torch.bool layout); may be NULL.
 * and, in `workspace` (epd_workspace_bytes(T, k, E, R, N) bytes), the rank of
 * every pair among the pairs of its expert in token-major (t, then j) order,
 * which ep_permute turns into slots. The ranks come from per-tile counts and
 * an exclusive prefix over token tiles: for up to 16 x 8192 pairs (E <= 1024)
 * the tiles are the blocks of thread-block clusters of 2-16 blocks, which
 * exchange their counts through distributed shared memory -- one cluster, or,
 * where one cluster of 16 would need 8 chunks of 32 pairs per warp, up to 8
 * clusters that all fit on the device at once, whose last blocks publish each
 * cluster's counts in the workspace for the later clusters (a later cluster waits
 * for the earlier ones to run: should other work hold the SMs they need for about
 * a second, the wait gives up with EPD_ERR_TIMEOUT); larger batches use
 * a single-pass decoupled look-back over tiles taken in ticket order. Every way
 * the result does not depend on the order in which blocks run. Ids outside
 * [-1, E) set EPD_ERR_INVALID_EXPERT in *status and are treated as -1.
 */
EPD_API epd_status_t ep_dispatch_layout(const int64_t *topk_idx, int num_tokens, int num_topk,
                                int num_experts, int num_ranks, int num_rdma_ranks,
                                int32_t *tokens_per_expert, int32_t *tokens_per_rank,
                                int32_t *tokens_per_rdma_rank, uint8_t *is_token_in_rank,
                                void *workspace, int32_t *status, epd_stream_t stream);

/*
 * Steps 1 and 2 in one launch: ep_dispatch_layout, and the block of the last
 * token tile, once it has the totals, also writes expert_start_loc and *total_rows exactly as
 * ep_scan_offsets_aligned(tokens_per_expert, alignment) would (alignment 1 gives
 * ep_scan_offsets). Saves one launch and one kernel per pass; same arguments and
 * errors as ep_dispatch_layout otherwise.
 */
EPD_API epd_status_t ep_dispatch_layout_offsets(const int64_t *topk_idx, int num_tokens,
                                                int num_topk, int num_experts, int num_ranks,
                                                int num_rdma_ranks, int32_t *tokens_per_expert,
                                                int32_t *tokens_per_rank,
                                                int32_t *tokens_per_rdma_rank,
                                                uint8_t *is_token_in_rank, int alignment,
                                                int32_t *expert_start_loc, int32_t *total_rows,
                                                void *workspace, int32_t *status,
                                                epd_stream_t stream);

/*
 * Step 2 -- expert offsets. [P2] "5. 缓冲区布局与发送" (the first source starts
 * at 0, each next one where the previous ended) and [P1] 2.2.4 (ep_scatter
 * scans, then scatters): expert_start_loc[e] = sum of tokens_per_expert[e'] for
 * e' < e; *total_rows (device int32) = the sum of all counts. A negative count
 * sets EPD_ERR_INVALID_ARG in *status.
 */
EPD_API epd_status_t ep_scan_offsets(const int32_t *tokens_per_expert, int num_experts,
                             int32_t *expert_start_loc, int32_t *total_rows, int32_t *status,
                             epd_stream_t stream);

/*
 * Step 2 with expert alignment (the grouped-GEMM contiguous layout). [P1] 3.3
 * and 4 (deepgemm_moe_permute pads every expert to block_m = 256 rows;
 * compute_aligned_M) and [P3] "Dispatch" (dispatch's expert_alignment): every
 * expert's region holds round_up(tokens_per_expert[e], alignment) rows;
 * expert_start_loc[e] = sum of the padded counts of e' < e, *total_rows = the sum
 * of all padded counts. alignment in [1, EPD_MAX_ALIGNMENT]; 1 gives
 * ep_scan_offsets. A buffer of round_up(T*k + E*(alignment-1), alignment) rows
 * always holds the padded regions. ep_permute fills them and marks the padding
 * rows with m_indices = -1.
 */
EPD_API epd_status_t ep_scan_offsets_aligned(const int32_t *tokens_per_expert, int num_experts,
                                             int alignment, int32_t *expert_start_loc,
                                             int32_t *total_rows, int32_t *status,
                                             epd_stream_t stream);

/*
 * Step 3 -- permute (ep_scatter). [P1] 2.2 (ep_scatter into input_tensor,
 * input_tensor_scale, m_indices, output_index) and 3.3 (m_indices pre-set to
 * -1 so that unwritten rows are skipped): for every pair (t, j) with expert
 * e = topk_idx[t, j] != -1, its slot is s = expert_start_loc[e] + (rank of the
 * pair inside e, from ep_dispatch_layout's workspace) and
 *   out[s, :]         = x[t, :]        (row bytes copied verbatim),
 *   out_scale[s, :]   = x_scale[t, :]  (fp8 only, H/128 floats),
 *   m_indices[s]      = e,
 *   output_index[t,j] = s;
 * pairs with no selection get output_index = -1, and m_indices[s] = -1 for
 * every row s in [0, capacity_rows) that no pair fills (alignment padding and
 * the rows after the last region). expert_start_loc may come from
 * ep_scan_offsets or ep_scan_offsets_aligned. Rows of out and out_scale that no
 * pair fills are not written.
 *   x:            [T, H] dtype rows, 16-byte aligned;
 *   x_scale:      [T, H/128] float32 for EPD_FP8_E4M3, NULL for EPD_BF16;
 *   out:          [capacity_rows, H] dtype, 16-byte aligned;
 *   out_scale:    [capacity_rows, H/128] float32 (fp8) or NULL (bf16);
 *   m_indices:    [capacity_rows] int32;  output_index: [T, k] int32;
 *   capacity_rows >= T*k (the exact-allocation upper bound with alignment 1;
 *   with aligned offsets it must also hold the padded regions),
 *   capacity_rows <= INT32_MAX.
 * `workspace` must hold the layout of the same topk_idx (same T and k); a
 * mismatch sets EPD_ERR_INVALID_ARG in *status and writes nothing.
 * Over the whole expert range the kernel asks L2 for up to 32 MB of x's first
 * rows before it waits for the previous kernel on the stream (a prefetch: it
 * changes no value any load returns), marked evict-last, and releases each line
 * (evict-first) when it reads the row.
 */
EPD_API epd_status_t ep_permute(const void *x, epd_dtype_t dtype, const float *x_scale,
                        const int64_t *topk_idx, int num_tokens, int num_topk, int hidden,
                        int num_experts, const int32_t *expert_start_loc, const void *workspace,
                        int64_t capacity_rows, void *out, float *out_scale, int32_t *m_indices,
                        int32_t *output_index, int32_t *status, epd_stream_t stream);

/*
 * Steps 1 to 3 in one call: the dispatch layout with its (aligned) offsets, then
 * the permute over the whole expert range with row-major scales -- exactly the
 * outputs of ep_dispatch_layout_offsets followed by ep_permute on the same
 * arguments, workspace state included. A small batch (T*k <= 4096, T <= 1024,
 * E <= 1024, R and N <= 64; a decode step) runs as one kernel in which every
 * block counts and scans the whole batch's picks itself and copies its own
 * tokens' rows; larger batches run the two kernels. Arguments, layouts and errors
 * as in those two calls; tokens_per_rdma_rank and is_token_in_rank may be NULL.
 * capacity_rows must hold the (aligned) total (a slot outside sets
 * EPD_ERR_CAPACITY). The pages have no single call for these steps (DeepEP
 * computes the layout in get_dispatch_layout before dispatch).
 */
EPD_API epd_status_t ep_dispatch(const void *x, epd_dtype_t dtype, const float *x_scale,
                                 const int64_t *topk_idx, int num_tokens, int num_topk,
                                 int hidden, int num_experts, int num_ranks, int num_rdma_ranks,
                                 int alignment, int32_t *tokens_per_expert,
                                 int32_t *tokens_per_rank, int32_t *tokens_per_rdma_rank,
                                 uint8_t *is_token_in_rank, int32_t *expert_start_loc,
                                 int32_t *total_rows, void *workspace, int64_t capacity_rows,
                                 void *out, float *out_scale, int32_t *m_indices,
                                 int32_t *output_index, int32_t *status, epd_stream_t stream);

/*
 * Output options of ep_permute_ex.
 *   expert_begin, expert_end: the view -- only pairs whose expert is in
 *     [expert_begin, expert_end) are placed (0 and num_experts for all
 *     experts). A simulated rank r of R holds [r*E/R, (r+1)*E/R). Rows are
 *     relative to the view's first region: a pair's row is
 *     expert_start_loc[e] - expert_start_loc[expert_begin] + its rank inside e,
 *     m_indices holds the local id e - expert_begin, and pairs outside the view
 *     get output_index = -1.
 *   scale_cols: 32-bit scale words per token (H/128 fp32 scales, or
 *     ceil(H/512) words of four packed UE8M0 exponent bytes); 0 for none.
 *   scale_col_major: 0 stores word c of row s at out_scale[s * scale_cols + c];
 *     1 stores it at out_scale[c * scale_ld + s] (column-major, the layout a
 *     TMA-fed grouped GEMM reads), scale_ld >= capacity_rows.
 */
typedef struct {
    int expert_begin;
    int expert_end;
    int scale_cols;
    int scale_col_major;
    int64_t scale_ld;
} epd_permute_view_t;

/*
 * Step 3 with output options: a per-rank view ([P1] 3.1.2 and 7: after dispatch
 * a rank's topk ids are local, rank_expert_offset maps them; [P1] 3.3:
 * deepgemm_moe_permute over local_num_experts) and scale layouts ([P1] 2.2:
 * UE8M0 scales as an int tensor [ceil(H/512), M] viewed transposed; [P3]
 * low_latency_dispatch docstring: scales column-major for TMA). Rows are any
 * row_bytes (a multiple of 16) copied verbatim; `view` is a host pointer.
 * capacity_rows must hold the view's regions (a slot outside sets
 * EPD_ERR_CAPACITY). Otherwise as ep_permute, which is this call with the whole
 * expert range and row-major fp32 scales. With column-major scales of more than
 * 16 words per row and a view of at least a quarter of the experts the call
 * enqueues two kernels: the row copy, which parks each filled row's source token
 * in m_indices, then a pass that writes the scales down their columns (coalesced)
 * and the final m_indices; m_indices is only meaningful once both have run.
 */
EPD_API epd_status_t ep_permute_ex(const void *x, int64_t row_bytes, const void *x_scale,
                                   const int64_t *topk_idx, int num_tokens, int num_topk,
                                   int num_experts, const int32_t *expert_start_loc,
                                   const void *workspace, int64_t capacity_rows,
                                   const epd_permute_view_t *view, void *out, void *out_scale,
                                   int32_t *m_indices, int32_t *output_index, int32_t *status,
                                   epd_stream_t stream);

/*
 * Low-latency dispatch layout with the fused cast. [P2] "3. 解决方案：固定矩形 vs.
 * 精确分配" strategy A (a fixed rectangle of rows per expert, sized for the worst
 * case, no count exchange first) and [P3] "low_latency模式" (low_latency_dispatch:
 * bf16 tokens cast to fp8 e4m3 on the way, one fp32 scale per 128 columns with
 * the last two dimensions column-major, recv_count, per-row source info).
 * Experts [expert_begin, expert_end) each own rows_per_expert rows; the r-th pick
 * of expert e in token-major order (the pair ranks ep_dispatch_layout left in
 * `workspace`) goes to row (e - expert_begin) * rows_per_expert + r -- no
 * ep_scan_offsets is needed. For every token with a pick in the view and every
 * 128-column block c:
 *   amax = max |x[t, 128c .. 128c+127]|, scale = amax / 448 (fp32; 1 if amax = 0),
 *   q = e4m3(x / scale), fp32 division, round to nearest even, saturating at 448,
 * written to every row the token goes to.
 *   x_bf16:    [T, H] bfloat16, H % 128 == 0, 16-byte aligned;
 *   out_q:     [E_view, rows_per_expert, H] e4m3 bytes, 8-byte aligned;
 *   out_scale: [E_view, H/128, rows_per_expert] float32;
 *   recv_count [E_view] int32: rows used per expert (at most rows_per_expert);
 *   output_index [T, k] int32: row of each pair, -1 for no pick, other experts,
 *     or a pick that found its rectangle full (EPD_ERR_CAPACITY in *status);
 *   src_token [E_view, rows_per_expert] int32: token of each used row; may be NULL.
 * Rows at and beyond recv_count are not written. ep_unpermute combines expert
 * outputs laid out in the same rectangles.
 */
EPD_API epd_status_t ep_permute_lowlatency(const void *x_bf16, const int64_t *topk_idx,
                                           int num_tokens, int num_topk, int hidden,
                                           int num_experts, int expert_begin, int expert_end,
                                           int64_t rows_per_expert, const void *workspace,
                                           void *out_q, float *out_scale, int32_t *recv_count,
                                           int32_t *output_index, int32_t *src_token,
                                           int32_t *status, epd_stream_t stream);

/*
 * The low-latency dispatch in one call: the same outputs as ep_dispatch_layout (its
 * pair ranks only) followed by ep_permute_lowlatency, without the layout's count
 * outputs ([P3] low_latency_dispatch returns recv_count, not a layout). A
 * decode-sized batch (T*k <= 4096, T <= 1024, E <= 1024, a block's bf16 rows
 * within 96 KiB) runs as one kernel in which every block ranks its own tokens'
 * picks against the batch itself -- a fixed rectangle needs no offsets -- and
 * casts its own rows; the workspace is then not touched. Larger batches run the
 * layout kernel (which needs `workspace` sized by epd_workspace_bytes(T, k, E, R,
 * N)) and then ep_permute_lowlatency. Arguments, layouts, results and errors as in
 * ep_permute_lowlatency.
 */
EPD_API epd_status_t ep_dispatch_lowlatency(const void *x_bf16, const int64_t *topk_idx,
                                            int num_tokens, int num_topk, int hidden,
                                            int num_experts, int num_ranks, int num_rdma_ranks,
                                            int expert_begin, int expert_end,
                                            int64_t rows_per_expert, void *workspace, void *out_q,
                                            float *out_scale, int32_t *recv_count,
                                            int32_t *output_index, int32_t *src_token,
                                            int32_t *status, epd_stream_t stream);

/*
 * Step 4 -- unpermute (combine). [P3] "Dispatch" (combine is the reverse of
 * dispatch; topk_weights are fp32 [T, k]):
 *   y[t, h] = bf16( sum over j with output_index[t, j] != -1, in j order, of
 *                   topk_weights[t, j] * expert_out[output_index[t, j], h] )
 * with every product and sum in fp32 (no fused multiply-add) and one
 * round-to-nearest-even to bf16. A token with no valid pair gets +0.
 *   expert_out:   [capacity_rows, H] bfloat16, 16-byte aligned;
 *   output_index: [T, k] int32 (from ep_permute); topk_weights: [T, k] float32;
 *   y:            [T, H] bfloat16, 16-byte aligned; H % 8 == 0.
 * A slot outside [-1, capacity_rows) sets EPD_ERR_CAPACITY and is skipped.
 */
EPD_API epd_status_t ep_unpermute(const void *expert_out, int64_t capacity_rows,
                          const int32_t *output_index, const float *topk_weights, int num_tokens,
                          int num_topk, int hidden, void *y, int32_t *status, epd_stream_t stream);

/* ------------------------------------------------------------------ routing
 * The step before the layout: topk_idx and topk_weights from router logits. */
typedef enum {
    EPD_SCORE_SOFTMAX = 0, /* s[t, e] = exp(l[t, e] - max) / sum over the row */
    EPD_SCORE_SIGMOID = 1, /* s[t, e] = 1 / (1 + exp(-l[t, e])) */
} epd_scoring_t;

typedef enum {
    EPD_GROUP_MAX = 0,  /* a group scores as its best expert */
    EPD_GROUP_TOP2 = 1, /* a group scores as the sum of its two best experts */
} epd_group_score_t;

#define EPD_MAX_GROUPS 64

/*
 * Routing to experts. For every token, from its logits l[t, 0..E):
 *   s = softmax(l) or sigmoid(l) (fp32);
 *   c = s + bias (the balance bias; it takes part in the choice only, not in the
 *       weights; NULL for none);
 *   the experts form num_groups equal runs of consecutive experts; the topk_groups
 *       groups with the highest group score stay (all of them where topk_groups ==
 *       num_groups); EPD_GROUP_TOP2 sums what a group has where that is one expert;
 *   topk_idx[t, 0..k) = the k experts of those groups with the highest c, highest
 *       first; equal values go to the lowest index, for groups and for experts;
 *   topk_weights[t, j] = s[topk_idx[t, j]], divided by their sum over j if
 *       `renormalize` (0 where that sum is 0), times routed_scale.
 * Scores without a bias are compared by their logits, which order them exactly as
 * the scores do but never round two different ones to the same value; with a bias
 * (and in a group's sum of two) they are fp32 values within 8 units in the last place.
 * The weights' scores are computed to the last place or two. (Softmax, both: on top of
 * that the roundings of the sum over the row, and of the logit's difference from the
 * row's largest, half a unit for each unit of it.) That includes numbers below the
 * smallest normal one (a sigmoid is 0 below -103.97), and renormalised weights keep
 * their digits where all the picks' scores are that low.
 * An expert whose logit is -inf cannot be chosen; where fewer than k are left the
 * rest of the row is -1 with weight 0 (the type's lowest finite value is an ordinary
 * logit). A NaN or +inf logit sets EPD_ERR_NONFINITE in *status and counts as -inf; so
 * does a NaN bias of an expert that could be chosen. A bias of -inf takes its expert out,
 * one of +inf puts it first.
 *   logits: [T, E] float32 (EPD_F32) or bfloat16 (EPD_BF16);  bias: [E] float32;
 *   topk_idx: [T, k] int64;  topk_weights: [T, k] float32.
 * E in [1, EPD_MAX_EXPERTS], k in [1, min(E, EPD_MAX_TOPK)], num_groups in
 * [1, EPD_MAX_GROUPS] dividing E, topk_groups in [1, num_groups].
 */
EPD_API epd_status_t ep_route(const void *logits, epd_dtype_t dtype, const float *bias,
                              int num_tokens, int num_topk, int num_experts, int num_groups,
                              int topk_groups, epd_group_score_t group_score,
                              epd_scoring_t scoring, int renormalize, float routed_scale,
                              int64_t *topk_idx, float *topk_weights, int32_t *status,
                              epd_stream_t stream);

/*
 * Gradient of the weights of ep_route with respect to the logits (the choice itself
 * has none, and the bias does not enter the weights). With g = routed_scale *
 * grad_weights[t, :] and S the sum of the picks' scores:
 *   ds[topk_idx[t, j]] += g_j                                     (no renormalize)
 *                      += sum over i of (g_j - g_i) s_i / S / S   (renormalize),
 *   grad_logits = ds * s * (1 - s)                                (sigmoid)
 *               = s * (ds - sum over e of ds_e s_e)               (softmax),
 * computed so that neither 1 - s nor that difference cancels.
 * Picks of -1 have no gradient; an id outside [-1, E) sets EPD_ERR_INVALID_EXPERT and
 * counts as -1; a pick whose logit is NaN or +inf sets EPD_ERR_NONFINITE and has score 0.
 * Renormalised softmax weights are the softmax of the picks' logits alone, and are computed
 * as that, here and in ep_route. Every element of grad_logits [T, E] (the logits' type) is written, 0
 * for an expert that cannot be chosen. An expert that a row picks twice gets both
 * picks' terms. grad_logits must not overlap logits.
 */
EPD_API epd_status_t ep_route_backward(const float *grad_weights, const void *logits,
                                       epd_dtype_t dtype, const int64_t *topk_idx, int num_tokens,
                                       int num_topk, int num_experts, epd_scoring_t scoring,
                                       int renormalize, float routed_scale, void *grad_logits,
                                       int32_t *status, epd_stream_t stream);

/* ------------------------------------------------------- the experts' products
 * Matrix products over the expert-contiguous buffer that ep_permute fills (or the
 * rectangles of ep_permute_lowlatency), between permute and combine. */

/*
 * Where each expert's rows lie. Expert e owns rows [start, start + tokens_per_expert[e])
 * with start = expert_start_loc[e], or e * rows_per_expert where expert_start_loc is NULL
 * (rectangles). The counts and starts are device memory, read by the kernel: nothing goes
 * back to the host. Regions must not overlap. A negative count or start sets
 * EPD_ERR_INVALID_ARG in *status and counts as no rows; a region that does not end within
 * capacity_rows (or within its rectangle) sets EPD_ERR_CAPACITY and is cut there. The
 * products' kernels wait for their own copies and matrix instructions only; each wait is
 * bounded (two seconds, and two microseconds for each 64 elements of the longest reduction
 * that the buffers hold) and running out sets EPD_ERR_TIMEOUT: the kernel then lets what it
 * has in flight land, and returns.
 */
typedef struct {
    int num_experts;
    int64_t capacity_rows;            /* rows of every row buffer of the call, <= INT32_MAX */
    int64_t rows_per_expert;          /* rectangles only: E * rows_per_expert <= capacity_rows */
    const int32_t *expert_start_loc;  /* device [E], or NULL */
    const int32_t *tokens_per_expert; /* device [E] */
} epd_expert_rows_t;

typedef enum {
    EPD_ACT_NONE = 0,
    EPD_ACT_RELU = 1,
    EPD_ACT_SILU = 2,   /* z * sigmoid(z) */
    EPD_ACT_GELU = 3,   /* z * Phi(z), the exact form with erf */
    EPD_ACT_SWIGLU = 4, /* silu(gate) * up: the weight has 2N rows, gate first, then up */
} epd_activation_t;

/*
 * The experts' product with its epilogue. For every row s of expert e:
 *   z[s, :] = x[s, :] . w[e]^T + bias[e]           (fp32 accumulation)
 *   y[s, :] = bf16( act(z[s, :]) + residual[s, :] )
 * and, where `preact` is given, preact[s, :] = bf16(z[s, :]) for the backward pass.
 * Rows that belong to no expert are not written. Each value is rounded once, from fp32.
 *
 * Order of the sums, here and in the two gradients below: it does not depend on how blocks
 * are scheduled, so that the same call on the same device gives the same bits again. It does
 * depend on the sizes: a few tiles' long reductions are cut into two or four parts, chosen
 * from capacity_rows, num_experts, K, N, how many blocks the device runs at a time and, for
 * wgrad, the expert's rows. The same rows in a larger buffer, beside other experts or on another device may differ by the
 * roundings of their fp32 sums.
 *   x: [capacity_rows, K] bfloat16 (K % 8 == 0), or e4m3 (K % 128 == 0) with
 *      x_scale, one fp32 scale per row and 128 columns: the scale of row s of expert e and
 *      column block c is x_scale[s * scale_row_stride + c * scale_col_stride + e *
 *      scale_expert_stride] -- (K/128, 1, 0) for the rows of ep_permute, (1, scale_ld, 0)
 *      for its column-major scales and (1, rows, (K/128 - 1) * rows) for the rectangles of
 *      ep_permute_lowlatency;
 *   w: [E, NW, K] of x's type, NW = N (2N for EPD_ACT_SWIGLU); with e4m3 w_scale is
 *      [E, ceil(NW/128), K/128] float32, one scale per 128 x 128 block;
 *   bias: [E, NW] float32 or NULL; residual: [capacity_rows, N] bfloat16 or NULL;
 *   y: [capacity_rows, N], preact: [capacity_rows, NW] bfloat16 (preact may be NULL).
 * N % 8 == 0; for EPD_ACT_SWIGLU with e4m3 N % 128 == 0. All row buffers and w
 * 16-byte aligned. Outputs must not overlap inputs, here and in the gradients. One expert over the whole buffer is an ordinary linear layer.
 */
EPD_API epd_status_t ep_expert_matmul(const epd_expert_rows_t *rows, const void *x,
                                      epd_dtype_t dtype, const float *x_scale,
                                      int64_t scale_row_stride, int64_t scale_col_stride,
                                      int64_t scale_expert_stride, const void *w,
                                      const float *w_scale, int in_features, int out_features,
                                      epd_activation_t activation, const float *bias,
                                      const void *residual, void *y, void *preact,
                                      int32_t *status, epd_stream_t stream);

/*
 * Gradient of the product's input, with the gradient of the activation that made the input in
 * its epilogue. For every row s of expert e, with d[s, :] = dy[s, :] . w[e] (fp32):
 *   dx[s, :] = d[s, :]                                     (EPD_ACT_NONE, preact NULL)
 *            = d[s, :] * act'(preact[s, :])                (the gradient of preact)
 *            = [d * up * silu'(gate), d * silu(gate)]      (EPD_ACT_SWIGLU, 2K columns)
 * rounded once to bfloat16.
 *   dy: [capacity_rows, N], w: [E, N, K], dx and preact: [capacity_rows, K or 2K], all
 *   bfloat16 and 16-byte aligned; N % 8 == 0, K % 8 == 0.
 */
EPD_API epd_status_t ep_expert_matmul_dgrad(const epd_expert_rows_t *rows, const void *dy,
                                            const void *w, int in_features, int out_features,
                                            epd_activation_t activation, const void *preact,
                                            void *dx, int32_t *status, epd_stream_t stream);

/*
 * Gradients of the weights and the bias: for every expert e
 *   dw[e] = sum over its rows s of dy[s, :]^T x[s, :]   (fp32, rounded once to bfloat16)
 *   dbias[e] = sum over its rows s of dy[s, :]          (float32; NULL to leave it out)
 * in an order that is fixed for given sizes (see ep_expert_matmul); 0 for an expert without
 * rows. Rows outside the experts' regions are not used, whatever they hold.
 *   dy: [capacity_rows, N], x: [capacity_rows, K], dw: [E, N, K] bfloat16, 16-byte aligned;
 *   dbias: [E, N] float32; N % 8 == 0, K % 8 == 0, both up to 2^30 (EPD_ERR_UNSUPPORTED).
 */
EPD_API epd_status_t ep_expert_matmul_wgrad(const epd_expert_rows_t *rows, const void *dy,
                                            const void *x, int in_features, int out_features,
                                            void *dw, float *dbias, int32_t *status,
                                            epd_stream_t stream);

/*
 * Gradient of the combine (ep_unpermute). For every pair with slot = output_index[t, j]:
 *   grad_expert_out[slot, :] = bf16( topk_weights[t, j] * grad_y[t, :] )
 *   grad_weights[t, j]       = sum over h of grad_y[t, h] * expert_out[slot, h]   (fp32)
 * and grad_weights[t, j] = 0 where output_index is -1. Rows of grad_expert_out that no pair
 * fills are not written (the products above do not read them). The gradient of ep_permute's
 * input is ep_unpermute of the rows' gradients with weights of 1.
 *   grad_y: [T, H], expert_out and grad_expert_out: [capacity_rows, H] bfloat16, 16-byte
 *   aligned, H % 8 == 0; topk_weights and grad_weights: [T, k] float32.
 * A slot outside [-1, capacity_rows) sets EPD_ERR_CAPACITY and is skipped. Outputs must not
 * overlap inputs.
 */
EPD_API epd_status_t ep_unpermute_backward(const void *grad_y, const void *expert_out,
                                           int64_t capacity_rows, const int32_t *output_index,
                                           const float *topk_weights, int num_tokens,
                                           int num_topk, int hidden, void *grad_expert_out,
                                           float *grad_weights, int32_t *status,
                                           epd_stream_t stream);

/* ------------------------------------------------------------------ the norm
 * Ahead of the router, the dispatch and the projections. */
typedef enum {
    EPD_NORM_LAYER = 0, /* centred, divided by the standard deviation */
    EPD_NORM_RMS = 1,   /* divided by the root mean square */
} epd_norm_t;

/*
 * Layer norm. For every row, with s = x + residual (s = x where residual is NULL):
 *   mean = sum of s / H (EPD_NORM_RMS: 0), rstd = (sum of (s - mean)^2 / H + eps)^-1/2,
 *   n = (s - mean) * rstd * weight + bias,
 * in fp32 and rounded once to each of
 *   sum  [T, H] of x's type: s, the residual stream from here on (only with residual);
 *   y    [T, H] bfloat16: n, what the router's projection and the products read;
 *   y_q  [T, H] e4m3 with y_scale [T, H/128] float32: n / scale with one scale per 128
 *        columns, amax / 448 (1 where amax is 0, never below 2^-149), as ep_dispatch and
 *        ep_permute take rows (H % 128 == 0);
 *   mean, rstd [T] float32, for ep_layer_norm_backward;
 * each of which may be NULL, but not y and y_q both. n is computed from s before s is rounded.
 *   x, residual: [T, H] float32 (EPD_F32) or bfloat16 (EPD_BF16); weight, bias: [H]
 *   float32, NULL for ones and zeros. H % 8 == 0, H <= 16384 (EPD_ERR_UNSUPPORTED beyond);
 *   rows, weight and bias 16-byte aligned. sum may be the buffer of x or residual itself, and
 *   y that of bfloat16 x; otherwise outputs must not overlap inputs. eps >= 0.
 */
EPD_API epd_status_t ep_layer_norm(const void *x, epd_dtype_t dtype, const void *residual,
                                   const float *weight, const float *bias, int num_tokens,
                                   int hidden, float eps, epd_norm_t kind, void *sum, void *y,
                                   void *y_q, float *y_scale, float *mean, float *rstd,
                                   epd_stream_t stream);

/* Workspace size in bytes of ep_layer_norm_backward for rows of `hidden` columns (0 for a size it
 * does not take). It holds nothing between calls; it serves one stream at a time. */
EPD_API size_t epd_norm_workspace_bytes(int hidden);

/*
 * Gradients of ep_layer_norm. With xh = (x - mean) * rstd and g = dy * weight, for every row
 *   dx = rstd * (g - sum of g / H - xh * (sum of g * xh) / H) + grad_sum
 * (EPD_NORM_RMS: xh = x * rstd, without the sum of g; mean is not read), and over all rows
 *   dweight = sum of dy * xh,  dbias = sum of dy   (float32; each NULL to leave it out),
 * 0 where there are no rows. x is what was normalised: `sum` where a residual was added, whose
 * gradient is dx as well; grad_sum (NULL for none) is the gradient that `sum` has from
 * elsewhere. The order of the sums over the rows is fixed for given T, H and a device: the same
 * call gives the same bits again.
 *   dy: [T, H] bfloat16; x, grad_sum, dx: [T, H] of `dtype`; mean, rstd: [T] float32;
 *   dweight, dbias: [H] float32; workspace: epd_norm_workspace_bytes(H) bytes (NULL where neither
 *   dweight nor dbias is asked for). All but mean and rstd 16-byte aligned. dx may be the buffer
 *   of x or grad_sum itself, or of dy where x is bfloat16; otherwise outputs must not overlap inputs.
 */
EPD_API epd_status_t ep_layer_norm_backward(const void *dy, const void *x, epd_dtype_t dtype,
                                            const float *weight, const float *mean,
                                            const float *rstd, const void *grad_sum,
                                            int num_tokens, int hidden, epd_norm_t kind,
                                            void *workspace, void *dx, float *dweight,
                                            float *dbias, epd_stream_t stream);

/* ------------------------------------------------------------------ positions and the cache
 * For the attention ahead of the layer: rotary positions, the paged key-value cache and what
 * reads it in a decode step. */

/*
 * Rotary positions. In every head the first rotary_dim = R elements are R/2 pairs -- elements
 * (i, i + R/2), or (2i, 2i + 1) with `interleaved` -- and pair i of token t becomes
 *   (a, b) -> rotary_scale * (a cos p - b sin p, a sin p + b cos p),
 *   p = 2 pi * positions[t] * steps[i] / 2^64,
 * in fp32 (sine and cosine within 2^-20) and rounded once; the other elements are copied. steps[i] is the fraction of a turn
 * that one position adds to pair i, in units of 2^-64: round(f_i / (2 pi) * 2^64) mod 2^64 for
 * an angular frequency f_i. The product is taken modulo 2^64, a whole turn, so that the angle is
 * as good at position 2^31 - 1 as at 1: within 2^-24 of half a turn. With `inverse` the rotation is
 * by -p: the gradient of the rotation.
 *   x, out: [T, num_heads, head_dim] bfloat16 with the strides given (in elements, multiples of
 *   8; the elements of a head lie together), 16-byte aligned; out may be x itself with the same
 *   strides (the elements past R are then left alone), otherwise they must not overlap; out's
 *   strides are not 0 where there is more than one to a stride.
 *   positions: [T] int32, any sign; steps: [R/2] uint64.
 * head_dim % 8 == 0, up to 256 (EPD_ERR_UNSUPPORTED beyond); R even, in [2, head_dim].
 */
EPD_API epd_status_t ep_rotary(const void *x, int64_t token_stride, int64_t head_stride,
                               const int32_t *positions, const uint64_t *steps, int num_tokens,
                               int num_heads, int head_dim, int rotary_dim, int interleaved,
                               float rotary_scale, int inverse, void *out,
                               int64_t out_token_stride, int64_t out_head_stride,
                               epd_stream_t stream);

/*
 * A paged key-value cache. Position p of sequence s lies on page n = page_table[s * table_stride
 * + p / page_size], in its row p % page_size; head h of that row is the head_dim elements from
 *   k (or v) + n * page_stride + (p % page_size) * token_stride + h * head_stride   (elements),
 * so that [page, row, head, dim] and [page, head, row, dim] orders are both a matter of strides.
 * With EPD_FP8_E4M3 every row and head has one float32 scale for its keys and one for its
 * values, at n * scale_page_stride + (p % page_size) * scale_token_stride + h *
 * scale_head_stride of k_scale and v_scale: a value is e4m3 * scale.
 * head_dim % 8 == 0 (e4m3: % 16), up to 256 (EPD_ERR_UNSUPPORTED beyond); strides multiples of 16
 * bytes; k and v 16-byte aligned; max_pages * page_size <= INT32_MAX. Pages may be shared by
 * sequences and lie in any order; entries past a sequence's last position are not read. The
 * struct itself is a host pointer.
 */
typedef struct {
    epd_dtype_t dtype; /* EPD_BF16, or EPD_FP8_E4M3 */
    int num_kv_heads;
    int head_dim;
    int page_size;
    int64_t num_pages;
    void *k, *v;
    float *k_scale, *v_scale; /* EPD_FP8_E4M3 only, else NULL */
    int64_t page_stride, token_stride, head_stride;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    const int32_t *page_table; /* device [num_seqs, max_pages], rows table_stride apart (0: one
                                * row for all sequences) */
    int num_seqs;
    int max_pages;
    int64_t table_stride;
} epd_cache_t;

/*
 * Appends keys and values to the cache, the keys (and the queries, where given) rotated as
 * ep_rotary does. Token t is position positions[t] of sequence token_seq[t] (of sequence t where
 * token_seq is NULL): its keys and values are written to that position's row, its rotated
 * queries to q_out. Prompts and single tokens are the same call. An e4m3 cache takes
 * scale = amax / 448 of the head's fp32 values (1 if amax = 0, never below 2^-149) and
 * e4m3(value / scale), nearest even of the fp32 quotient.
 * A token of sequence -1 is padding: nothing of it is written. A sequence outside
 * [-1, num_seqs), a position outside the sequence's pages or a page outside [0, num_pages) sets
 * EPD_ERR_CAPACITY, and the token is left out like padding. Two tokens at one position must not
 * be: what that row then holds is unspecified (nothing else is touched).
 *   q, q_out: [T, num_heads, head_dim], k, v: [T, num_kv_heads, head_dim] bfloat16, the heads of a
 *   token next to each other, tokens the given strides apart (elements, multiples of 8), 16-byte
 *   aligned: parts of one projection's rows are taken as they are. q may be NULL; q_out may be q
 *   itself with the same stride. rotary_dim 0 (steps NULL): no rotation. Strides of what is written
 *   (the cache's, q_out's) are not 0 where there is more than one to a stride.
 */
EPD_API epd_status_t ep_cache_append(const epd_cache_t *cache, const void *q,
                                     int64_t q_token_stride, int num_heads, const void *k,
                                     int64_t k_token_stride, const void *v, int64_t v_token_stride,
                                     const int32_t *positions, const int32_t *token_seq,
                                     int num_tokens, const uint64_t *steps, int rotary_dim,
                                     int interleaved, float rotary_scale, void *q_out,
                                     int64_t q_out_token_stride, int32_t *status,
                                     epd_stream_t stream);

/*
 * Workspace size in bytes of ep_decode_attention for up to num_seqs sequences (0 for sizes it
 * does not take). Host-only arithmetic. The workspace must be zero-filled once before its first use
 * (epd_workspace_init); every call leaves it ready for calls of any lengths and of any sizes
 * that fit. It serves one stream at a time: calls that overlap on the GPU and share a
 * workspace race, two captured graphs included.
 */
EPD_API size_t epd_attention_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads,
                                             int head_dim);

/*
 * Attention of one new token of every sequence over the paged cache (the token's own keys and
 * values appended before). With G = num_heads / num_kv_heads, for sequence b and head h,
 * over its live positions t -- [0, lengths[b]), or the last `window` of them where window > 0:
 *   s_t = softmax_scale * q[b, h] . k[t, h / G],
 *   out[b, h] = sum of exp(s_t) v[t, h / G] / sum of exp(s_t),  lse[b, h] = ln sum of exp(s_t)
 * with fp32 sums and one rounding of out; 0 and -inf for a sequence of length 0, NaN where a score is
 * NaN. What lies in the cache outside the live positions is not used, whatever it is.
 * On the way a bf16 cache's weights exp(s_t) are held to 2^-15 of their size and 2^-100 of the
 * largest; an e4m3 cache's to 2^-11 of their size (an eighth of out's rounding) and 2^-26 of the
 * largest, with values' scales up to 2^64 apart, and its queries to 2^-31 of a head's largest element.
 * lengths are device memory, read by the kernel: work is split evenly over the device for any mix
 * of them. The order of the sums depends on the sizes, the lengths and the device, not on how blocks
 * are scheduled: the same call gives the same bits again.
 * A length outside [0, max_pages * page_size] sets EPD_ERR_INVALID_ARG (below) or
 * EPD_ERR_CAPACITY (above) and counts as the nearer end; a page outside [0, num_pages) sets
 * EPD_ERR_CAPACITY and its positions are left out.
 *   q: [num_seqs, num_heads, head_dim] bfloat16, the heads of a sequence next to each other,
 *   sequences q_token_stride elements apart (a multiple of 8); out: [num_seqs, num_heads,
 *   head_dim] bfloat16; both 16-byte aligned; lse: [num_seqs, num_heads] float32 or NULL;
 *   lengths: [num_seqs] int32. num_seqs is the cache's. Any G; heads are taken 16 at a time, so
 *   that beyond 16 a key is read more than once. out must not overlap q.
 */
EPD_API epd_status_t ep_decode_attention(const epd_cache_t *cache, const void *q,
                                         int64_t q_token_stride, int num_heads,
                                         const int32_t *lengths, float softmax_scale, int window,
                                         void *workspace, void *out, float *lse, int32_t *status,
                                         epd_stream_t stream);

/*
 * Allocation-free variant of ep_dispatch_layout. The pages have no counterpart:
 * this entry point exists for callers that cannot allocate device memory at
 * the moment they need the layout -- for example code running inside an
 * inference engine or plugin whose device memory is planned up front and
 * handed out by the host framework, or code that must not touch the allocator
 * on a hot serving path. Such callers own the inputs and outputs but have no
 * way to provide the workspace.
 *
 * It computes exactly what ep_dispatch_layout computes (tokens_per_expert,
 * tokens_per_rank, tokens_per_rdma_rank, is_token_in_rank, same arguments and
 * errors) but keeps its scratch -- the look-back state and the per-pair ranks --
 * in a file-scope device array of EPD_NOALLOC_SCRATCH_BYTES (8 MiB) inside
 * libepd. Every GPU that loads the library holds that array until the process
 * exits. The call allocates nothing: no cudaMalloc, no cudaFree, no allocating
 * library routine.
 *   - Sizes whose scratch need, epd_workspace_bytes(T, k, E, R, N), exceeds
 *     EPD_NOALLOC_SCRATCH_BYTES are rejected with EPD_ERR_UNSUPPORTED before
 *     anything is launched (T*k up to about 1.8 million pairs fits at E = 256,
 *     R = 32, N = 4, k = 8).
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls share the one array, which keeps the previous call's contents.
 *     Nothing needs clearing between calls, whatever their shapes: every call
 *     leaves the tile ticket and finished-block count at zero, and the
 *     look-back only accepts state words tagged with the running call's
 *     counter, never an earlier call's ranks, counts or states. Calls in order
 *     on one stream are safe; calls that overlap on the GPU (other streams)
 *     race with each other.
 *   - The per-pair ranks it leaves in the shared array are not an input to
 *     ep_permute; a caller running the whole path uses ep_dispatch_layout with
 *     its own workspace.
 */
#define EPD_NOALLOC_SCRATCH_BYTES (8u << 20)

EPD_API epd_status_t ep_dispatch_layout_noalloc(const int64_t *topk_idx, int num_tokens,
                                                int num_topk, int num_experts, int num_ranks,
                                                int num_rdma_ranks, int32_t *tokens_per_expert,
                                                int32_t *tokens_per_rank,
                                                int32_t *tokens_per_rdma_rank,
                                                uint8_t *is_token_in_rank, int32_t *status,
                                                epd_stream_t stream);

/*
 * Test hook for failure detection, not part of the path: runs ep_dispatch_layout
 * in its tile form (whatever the batch size) with the look-back wait bounded by
 * `spin_limit` polls and with token tile
 * `stalled_tile` never publishing its state, so that every later tile's wait
 * runs out. The call still completes; *status then holds EPD_ERR_TIMEOUT and
 * the counts are meaningless. The workspace stays reusable afterwards.
 */
EPD_API epd_status_t epd_test_layout_stalled_tile(const int64_t *topk_idx, int num_tokens, int num_topk,
                                          int num_experts, int num_ranks, int num_rdma_ranks,
                                          int32_t *tokens_per_expert, int32_t *tokens_per_rank,
                                          int32_t *tokens_per_rdma_rank,
                                          uint8_t *is_token_in_rank, void *workspace,
                                          int32_t *status, int stalled_tile,
                                          uint32_t spin_limit, epd_stream_t stream);

/*
 * Test hook for failure detection, not part of the path: runs ep_expert_matmul (without bias,
 * residual and preact) with every wait bounded by `wait_ns` nanoseconds (>= 1) and with each
 * pair of blocks leaving out the matrix instructions from its tile number `stalled_tile` on
 * (-1: none), so that the waits for them run out. The call still completes; *status then
 * holds EPD_ERR_TIMEOUT and y is meaningless.
 */
EPD_API epd_status_t epd_test_expert_matmul_stalled(
    const epd_expert_rows_t *rows, const void *x, epd_dtype_t dtype, const float *x_scale,
    int64_t scale_row_stride, int64_t scale_col_stride, int64_t scale_expert_stride, const void *w,
    const float *w_scale, int in_features, int out_features, epd_activation_t activation, void *y,
    int32_t *status, int stalled_tile, int64_t wait_ns, epd_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EPD_H */
