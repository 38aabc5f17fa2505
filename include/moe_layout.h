/*
 * moe_layout.h -- C ABI of the single-GPU MoE layout / dispatch / combine
 * library (libmoe_layout.so, CUDA, sm_103a).
 *
 * The operations follow Perplexity, "Enabling trillion-parameter models on
 * AWS EFA" (2025-11-04).  The page splits MoE routing into a dispatch that
 * takes the tokens and their per-token experts and packs each token into
 * contiguous per-destination buffers, and its dual, combine, that brings the
 * processed rows back and forms their routing-weighted average (sections
 * "MoE all-to-all over EFA" and "Dispatch and Combine").  Here the R
 * expert-parallel destinations are R row ranges of one packed buffer in the
 * GPU's own memory; there is no network, peer or collective.
 *
 * Conventions for every call:
 *  - All pointers are device pointers unless stated otherwise.  The caller
 *    allocates and owns every buffer; the library allocates nothing and
 *    never synchronises, and apart from moe_layout_static's scratch array
 *    (described with that call) it keeps no state between calls.
 *  - moe_layout, moe_dispatch, moe_combine, moe_combine_fp8,
 *    moe_combine_rank_partial, moe_dispatch_send, moe_dispatch_recv,
 *    moe_layout_dispatch, moe_route, moe_route_backward, moe_route_grouped,
 *    moe_route_grouped_backward, moe_dispatch_int8, moe_expert_matmul_int8,
 *    moe_expert_matmul, moe_expert_activation_backward
 *    and moe_expert_matmul_backward are asynchronous on `stream` (0 = legacy
 *    default stream) and may be captured into a CUDA graph.
 *  - Arguments are checked on the host before anything is enqueued.  A
 *    failed check returns an error status and enqueues nothing.
 *  - Matrices are row-major and dense: a [rows, H] matrix has row stride H.
 *  - bf16 means IEEE binary32 truncated to its top 16 bits (stored as 2-byte
 *    words); e4m3 means the 8-bit "fn" float format (bias 7, largest finite
 *    448, no infinities).
 *  - Indices are int32: T*K must stay below 2^31.
 *  - Notation: T tokens, H hidden size, E experts, R destination ranks,
 *    K experts per token, Epr = E/R experts per rank.  Expert e belongs to
 *    rank e / Epr.
 */
#ifndef MOE_LAYOUT_H
#define MOE_LAYOUT_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status returned synchronously by every call. */
typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* null pointer, size out of range, E % R != 0 ... */
    MOE_ERR_ALIGNMENT = 2,    /* a pointer misses its required alignment       */
    MOE_ERR_CUDA = 3,         /* the CUDA runtime refused a launch             */
    MOE_ERR_WORKSPACE = 4     /* workspace missing or smaller than required    */
} moe_status_t;

/* Bits of the device error word written by moe_layout (read it after the
 * stream has reached that point). */
#define MOE_DEV_ERR_EXPERT_RANGE 1u  /* some topk_ids entry is outside [0, E)   */
#define MOE_DEV_ERR_DUPLICATE    2u  /* some token lists one expert twice       */
#define MOE_DEV_ERR_REGION_OVERFLOW 4u /* moe_dispatch_send: a rank's rows exceed
                                          its private + bulk capacity          */
#define MOE_DEV_ERR_TIMEOUT 8u       /* moe_layout_dispatch, moe_expert_matmul,
                                        its backward and moe_expert_matmul_int8:
                                        a bounded wait between the kernel's
                                        blocks or warps expired; outputs
                                        unspecified                            */

/* Scores of moe_route_grouped. */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1

/* Activations of moe_expert_matmul, a(z); s is the logistic function. */
#define MOE_ACT_NONE 0    /* z                                                      */
#define MOE_ACT_SILU 1    /* z s(z)                                                 */
#define MOE_ACT_GELU 2    /* z s(2 sqrt(2/pi) (z + 0.044715 z^3)): GELU's tanh form */
#define MOE_ACT_SWIGLU 3  /* gated: z[n] s(z[n]) z[N/2 + n], n < N/2                */

/* Limits of this implementation. */
#define MOE_MAX_EXPERTS 1024
#define MOE_MAX_TOPK 32
#define MOE_MAX_GROUPS 32

/* Human-readable name of a status code (static storage, never NULL). */
MOE_API const char *moe_status_string(moe_status_t status);

/* Bytes of device workspace moe_layout needs for these sizes (0 when the
 * whole layout fits one thread block).  Returns 0 for invalid sizes, which
 * moe_layout then rejects. */
MOE_API size_t moe_layout_workspace_bytes(int32_t T, int32_t K, int32_t E);

/* Number of kernel launches moe_layout makes for these sizes: 1 when the
 * whole layout fits one launch of self-counting blocks, 2 (count in
 * clusters of blocks that sum their histograms together, then one ranking
 * block per chunk) when the ranking blocks' shared memory fits, otherwise 3
 * (count, scan, rank; large batches with E near 1024).  0 for invalid
 * sizes.  A query: nothing is launched. */
MOE_API int32_t moe_layout_kernels(int32_t T, int32_t K, int32_t E);

/*
 * moe_layout -- routing histogram, exclusive scan and stable slot map.
 *
 * The page's dispatch-send first counts tokens per expert in shared memory,
 * then takes the cumulative sum of the counts to find the offsets at which
 * tokens are packed into contiguous per-destination send buffers ("Dispatch
 * and Combine"); the per-expert counts are also the routing information that
 * ranks exchange before writing ("Send/receive buffers").  This call computes
 * that metadata for all T*K (token, k) entries:
 *
 *   expert_counts[e]  = #{(t,k) : topk_ids[t,k] == e}                      [E]
 *   expert_offsets[e] = sum of expert_counts[e'] for e' < e;
 *   expert_offsets[E] = number of valid entries (T*K when no error)       [E+1]
 *   rank_offsets[r]   = expert_offsets[r*Epr]                              [R+1]
 *   dst_row[t,k]      = expert_offsets[e] + #{(t',k') before (t,k) in
 *                       row-major order with topk_ids[t',k'] == e}         [T*K]
 *   src_token[row]    = t for row = dst_row[t,k]                           [T*K]
 *
 * So packed row ranges [expert_offsets[e], expert_offsets[e+1]) hold expert
 * e's tokens in ascending token order, and rank r's region is rows
 * [rank_offsets[r], rank_offsets[r+1]).
 *
 * topk_ids     [T,K] int32, 4-byte aligned.
 * T >= 0, 1 <= K <= min(E, MOE_MAX_TOPK), 1 <= E <= MOE_MAX_EXPERTS,
 * R >= 1 with E % R == 0, T*K < 2^31, and T*K small enough for the kernels'
 * shared memory: at least 6.5 * 10^8 / E entries (671 K for E = 1024, 6.4 M
 * for E = 128); larger batches return MOE_ERR_INVALID_ARG.
 * Outputs (int32, 4-byte aligned): expert_counts, expert_offsets,
 * rank_offsets, src_token, dst_row.  dst_row and src_token may be NULL only
 * when T == 0.
 * dev_error    [1] uint32 or NULL.  Overwritten with MOE_DEV_ERR_* bits.
 *              An id outside [0,E) is not counted, gets dst_row -1 and no
 *              src_token row; src_token rows at or after expert_offsets[E]
 *              are then left untouched.  A duplicated id still gets its own
 *              slot, in k order.
 * workspace    device scratch of at least moe_layout_workspace_bytes(T,K,E)
 *              bytes, 16-byte aligned (may be NULL when that is 0).  Its
 *              contents on entry do not matter; it is in use until the
 *              stream passes this call.
 * T == 0 writes zero counts and offsets.
 */
MOE_API moe_status_t moe_layout(const int32_t *topk_ids, int32_t T, int32_t K,
                                int32_t E, int32_t R,
                                int32_t *expert_counts, int32_t *expert_offsets,
                                int32_t *rank_offsets, int32_t *src_token,
                                int32_t *dst_row, uint32_t *dev_error,
                                void *workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/*
 * moe_dispatch -- pack every token row into each of its K slots.
 *
 * The page's dispatch sender shuffles the tokens into send buffers so that
 * each destination receives one contiguous write ("Dispatch and Combine"),
 * and the evaluated setting quantises that payload to block-scaled FP8
 * ("Evaluation").  For every token t and k with 0 <= dst_row[t,k] < T*K:
 *
 *   fp8 == 0:  packed[dst_row[t,k], :] = tokens[t, :]            (bit copy)
 *   fp8 == 1:  for each 1x128 block b of row t:
 *                amax  = max |tokens[t, 128b .. 128b+127]|       (fp32)
 *                scale = amax / 448                              (fp32, RN)
 *                packed[dst_row[t,k], 128b+j] =
 *                    e4m3_satfinite_rn(tokens[t,128b+j] / scale) (fp32 divide)
 *                scales[dst_row[t,k], b] = scale
 *              a block with amax == 0 stores scale 0 and codes 0x00 / 0x80
 *              (the sign of each zero).
 * Entries with dst_row outside [0, T*K) are skipped.
 *
 * tokens   [T,H] bf16, 16-byte aligned.   dst_row [T,K] int32 (moe_layout).
 * packed   [T*K,H] bf16 (fp8 == 0) or e4m3 bytes (fp8 == 1), 16-byte aligned.
 * scales   [T*K,H/128] fp32, 4-byte aligned; required when fp8 == 1,
 *          ignored otherwise.
 * H >= 8 with H % 8 == 0 (H % 128 == 0 when fp8 == 1).  T == 0 is a no-op.
 */
MOE_API moe_status_t moe_dispatch(const void *tokens, int32_t T, int32_t H, int32_t K,
                                  const int32_t *dst_row, int32_t fp8, void *packed,
                                  float *scales, cudaStream_t stream);

/*
 * moe_combine -- routing-weighted sum of each token's K expert outputs.
 *
 * The page's combine receives the processed rows of every token and computes
 * their weighted average, accumulating only on the receiving side ("MoE
 * all-to-all over EFA", "Dispatch and Combine", "Evaluation").  With router
 * weights that already sum to one the weighted sum is that average, so no
 * division by the weight sum is made:
 *
 *   acc = +0 (fp32);  for k = 0 .. K-1:  acc = fma(topk_weights[t,k],
 *                                              expert_out[dst_row[t,k], j], acc)
 *   out[t, j] = bf16 round-to-nearest-even(acc)
 *
 * Terms whose dst_row is outside [0, T*K) are skipped.
 *
 * expert_out    [T*K,H] bf16, 16-byte aligned (rows in dispatch order).
 * topk_weights  [T,K] fp32, 4-byte aligned.   dst_row [T,K] int32.
 * out           [T,H] bf16, 16-byte aligned; must not overlap expert_out.
 * H >= 8 with H % 8 == 0.  T == 0 is a no-op.
 */
MOE_API moe_status_t moe_combine(const void *expert_out, const float *topk_weights,
                         const int32_t *dst_row, int32_t T, int32_t H,
                         int32_t K, void *out, cudaStream_t stream);

/*
 * moe_combine_fp8 -- moe_combine for expert outputs held as block-scaled e4m3.
 *
 * The evaluated setting dispatches block-scaled FP8 ("Evaluation"); when the
 * expert outputs stay in that form (e4m3 codes plus one fp32 scale per 1x128
 * block, as moe_dispatch with fp8 == 1 writes them), combine can read them
 * directly, moving about half the bytes of a bf16 combine.  Each value is
 * y = f32(code) * scale (fp32, round to nearest), then the same chain:
 *
 *   acc = +0;  for k = 0 .. K-1:  acc = fma(topk_weights[t,k], y[dst_row[t,k], j], acc)
 *   out[t, j] = bf16 round-to-nearest-even(acc)
 *
 * Terms whose dst_row is outside [0, T*K) are skipped.
 *
 * expert_out     [T*K,H] e4m3 bytes, 16-byte aligned.
 * expert_scales  [T*K,H/128] fp32, 4-byte aligned.
 * topk_weights   [T,K] fp32.   dst_row [T,K] int32.
 * out            [T,H] bf16, 16-byte aligned.
 * H >= 128 with H % 128 == 0.  T == 0 is a no-op.
 */
MOE_API moe_status_t moe_combine_fp8(const void *expert_out, const float *expert_scales,
                                     const float *topk_weights, const int32_t *dst_row,
                                     int32_t T, int32_t H, int32_t K, void *out,
                                     cudaStream_t stream);

/*
 * moe_combine_rank_partial -- combine with sender-side partial sums.
 *
 * The page accumulates only on the receiving side and contrasts this with
 * DeepEP, which sums in the sender to cut the bytes transferred, at some cost
 * in accuracy ("Evaluation").  This call computes that scheme on the same
 * data: each token's entries are grouped by the rank r = e / (E/R) hosting
 * their expert; each group is summed as the fp32 FMA chain in k order from
 * +0 and rounded to bf16 (the transfer format); the receiver adds the
 * groups' values as fp32 in ascending rank order from +0 and rounds to bf16.
 * With R == 1 or K == 1 it equals moe_combine.
 *
 * expert_out [T*K,H] bf16 (16-byte aligned), topk_weights [T,K] fp32,
 * topk_ids [T,K] int32 (the layout's input), dst_row [T,K] int32,
 * out [T,H] bf16 (16-byte aligned).  1 <= E <= MOE_MAX_EXPERTS, E % R == 0,
 * H % 8 == 0.  Entries whose expert id or dst_row is invalid are skipped.
 */
MOE_API moe_status_t moe_combine_rank_partial(const void *expert_out,
                                              const float *topk_weights,
                                              const int32_t *topk_ids,
                                              const int32_t *dst_row, int32_t T,
                                              int32_t H, int32_t K, int32_t E, int32_t R,
                                              void *out, cudaStream_t stream);

/*
 * moe_dispatch_send / moe_dispatch_recv -- dispatch through per-destination
 * send regions, then back into the grouped-GEMM input.
 *
 * The page's send-buffer design ("Send/receive buffers"): senders lay their
 * writes out contiguously once the per-expert counts are known; a small
 * private area per sender on each receiver takes the first tokens before
 * that, and the rest travel in one write per peer.  With one sender and R
 * destination ranks (rank r hosts experts r*E/R .. (r+1)*E/R - 1), rank r's
 * rows in slot order i = 0 .. n_r - 1 (n_r = rank_offsets[r+1] -
 * rank_offsets[r], from moe_layout) are written to
 *   priv[r, i]      for i < P          (the private area), or
 *   bulk[r, i - P]  for P <= i < P + C (the contiguous area),
 * and rows at i >= P + C are not written.  Rows are what moe_dispatch writes:
 * bf16 copies (fp8 == 0) or e4m3 codes with their 1x128 block scales
 * (fp8 == 1).  A region of T * min(K, E/R) rows can never overflow.
 * moe_dispatch_recv puts every region row back at its slot of `packed`
 * (and `scales`), so send + recv gives exactly the moe_dispatch output.
 *
 * priv   [R, P, row] and bulk [R, C, row], row = H bf16 or H e4m3 bytes;
 *        16-byte aligned.  priv_scales [R, P, H/128], bulk_scales [R, C, H/128]
 *        fp32 (fp8 == 1 only).  P >= 0, C >= 0.
 * topk_ids, dst_row [T, K] int32 and rank_offsets [R+1] int32 from moe_layout.
 *        rank_offsets must be moe_layout's output (non-decreasing, starting at
 *        0); moe_dispatch_recv skips packed rows outside
 *        [rank_offsets[0], rank_offsets[R]).
 * dev_error (send; may be NULL) is overwritten with
 *        MOE_DEV_ERR_REGION_OVERFLOW when some n_r exceeds P + C, else 0.
 * H % 8 == 0 (H % 128 == 0 for fp8), E % R == 0.  T == 0 is a no-op.
 */
MOE_API moe_status_t moe_dispatch_send(const void *tokens, int32_t T, int32_t H, int32_t K,
                                       int32_t E, int32_t R, const int32_t *topk_ids,
                                       const int32_t *dst_row, const int32_t *rank_offsets,
                                       int32_t fp8, int32_t P, void *priv, float *priv_scales,
                                       int32_t C, void *bulk, float *bulk_scales,
                                       uint32_t *dev_error, cudaStream_t stream);

MOE_API moe_status_t moe_dispatch_recv(const void *priv, const float *priv_scales, int32_t P,
                                       const void *bulk, const float *bulk_scales, int32_t C,
                                       const int32_t *rank_offsets, int32_t R, int32_t T,
                                       int32_t H, int32_t K, int32_t fp8, void *packed,
                                       float *scales, cudaStream_t stream);

/*
 * moe_layout_dispatch -- moe_layout followed by moe_dispatch, as one call.
 *
 * The page's dispatch-send kernel counts, scans and packs in one pass
 * ("Dispatch and Combine").  Every output is bit-identical to calling
 * moe_layout and then moe_dispatch with the same arguments.  For small
 * batches (decode shapes: T*K <= 8192 and a bounded amount of redundant
 * histogram work) it runs as a single kernel launch.  Larger batches run a
 * counting kernel and then one grid in which ranking blocks compute the
 * slots of each chunk of tokens while packing blocks copy every row as soon
 * as its chunk is ranked (two launches); where that grid's shared memory
 * would cost too much occupancy (E near 1024) they run moe_layout's kernels
 * and then the dispatch kernel.  moe_layout_dispatch_kernels() tells which.
 *
 * Arguments are those of moe_layout and moe_dispatch together, with the same
 * layouts, alignment and limits.  workspace: as for moe_layout (a buffer of
 * moe_layout_workspace_bytes(T,K,E) bytes always suffices; the single-kernel
 * path uses none).  dev_error gets moe_layout's bits and, on the two-launch
 * path, MOE_DEV_ERR_TIMEOUT when a bounded wait (1 s) expired: a packing
 * block's wait for its chunk's slots; the outputs are then unspecified.
 */
MOE_API moe_status_t moe_layout_dispatch(const int32_t *topk_ids, const void *tokens,
                                         int32_t T, int32_t H, int32_t K, int32_t E,
                                         int32_t R, int32_t fp8, int32_t *expert_counts,
                                         int32_t *expert_offsets, int32_t *rank_offsets,
                                         int32_t *src_token, int32_t *dst_row,
                                         uint32_t *dev_error, void *packed, float *scales,
                                         void *workspace, size_t workspace_bytes,
                                         cudaStream_t stream);

/* Number of kernel launches moe_layout_dispatch makes for these sizes: 1
 * when it runs as a single kernel, 2 on the two-launch path, otherwise
 * moe_layout_kernels() plus moe_dispatch's one.  0 for invalid sizes. */
MOE_API int32_t moe_layout_dispatch_kernels(int32_t T, int32_t H, int32_t K,
                                            int32_t E, int32_t fp8);

/* Bytes of the fixed scratch array that moe_layout_static uses (96 KiB). */
#define MOE_LAYOUT_STATIC_SCRATCH_BYTES (96u << 10)

/*
 * moe_layout_static -- moe_layout for callers that cannot allocate device
 * memory.  (The paper has no counterpart; this is a library convenience.)
 *
 * Some callers cannot call cudaMalloc where they need the layout: a plugin or
 * custom op run by an inference engine whose memory planner owns every device
 * allocation, or a latency-critical serving loop that must not enter the
 * device allocator once it runs (an allocation can block, synchronise or
 * fail).  This
 * call takes the same arguments and gives the same results as moe_layout, but
 * has no workspace argument: the scratch that large batches need lives in a
 * fixed array of MOE_LAYOUT_STATIC_SCRATCH_BYTES in the library's own device
 * memory, which every GPU that loads the library keeps until the process
 * exits.  The call allocates nothing (no cudaMalloc, no cudaFree).
 *
 * - Limit: a batch whose moe_layout_workspace_bytes(T,K,E) exceeds
 *   MOE_LAYOUT_STATIC_SCRATCH_BYTES is rejected with MOE_ERR_WORKSPACE.
 *   That covers every batch moe_layout accepts with E >= 2; with E = 1,
 *   batches above about 12.5 million entries are rejected.
 * - Set-up: the first call on a device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture.  Set-up failure returns MOE_ERR_CUDA.  The
 *   address is kept for the life of the process: after cudaDeviceReset on a
 *   device the kept address is stale, so do not call moe_layout_static on
 *   that device again in the same process.
 * - Sharing: all calls on a device share the one array, and it keeps the last
 *   call's contents.  Nothing in it needs to start at zero: each call writes
 *   every scratch entry before reading it.  Calls that can run at the same
 *   time on the GPU (different streams with no ordering between them) race
 *   on the array; order them on one stream or with events.
 */
MOE_API moe_status_t moe_layout_static(const int32_t *topk_ids, int32_t T, int32_t K,
                                       int32_t E, int32_t R, int32_t *expert_counts,
                                       int32_t *expert_offsets, int32_t *rank_offsets,
                                       int32_t *src_token, int32_t *dst_row,
                                       uint32_t *dev_error, cudaStream_t stream);

/*
 * moe_route -- from router logits to the routing that the calls above take,
 * with the per-expert counts and the balance loss, in one pass.
 *
 * An expert is open for a token when the token is not masked and its logit is
 * not -inf; a token with an open expert is routed.  With x the logits:
 *
 *   p[t,e]  = exp(x[t,e] - m_t) / sum over open e' of exp(x[t,e'] - m_t),
 *             0 for an expert that is not open or whose exp is below 2^-126
 *   topk_ids[t,:]      the K open experts of largest logit, largest first, ties
 *                      to the lowest index; -1 where fewer than K are open
 *   topk_weights[t,k]  p at topk_ids[t,k], divided by the sum of the token's K
 *                      when renormalize == 1; 0 where topk_ids is -1
 *   expert_counts[e]   entries of topk_ids equal to e (moe_layout's counts)  [E]
 *   routed_tokens      n, the number of routed tokens                        [1]
 *   loss               coef * E * sum over e of (expert_counts[e] / (K n)) *
 *                      (sum over t of p[t,e] / n); 0 when n == 0             [1]
 *
 * All sums are fp32 in an order that the sizes and the alignment of logits fix:
 * the same inputs give the same bits.  A NaN logit ranks below every number: it
 * is chosen only where fewer than K open logits are numbers, the lowest index
 * first.  A NaN or +inf logit of a token that is not masked makes the weights of
 * the token's chosen experts and the loss NaN, and moe_route_backward the
 * token's gradient.  A masked token's logits are not looked at.  An id of -1 is
 * what moe_layout reports as MOE_DEV_ERR_EXPERT_RANGE and then skips.
 *
 * logits      [T,E], fp32 (bf16 == 0) or bf16 (bf16 == 1), aligned to their type.
 * token_mask  [T] bytes or NULL; 0 masks the token (padding).
 * topk_ids [T,K] int32, topk_weights [T,K] fp32, expert_counts [E] int32,
 * routed_tokens [1] int32, loss [1] fp32: 4-byte aligned.
 * workspace   moe_route_workspace_bytes(T,E) bytes (never 0 for valid sizes),
 *             16-byte aligned; its contents on entry do not matter.
 * 0 <= T <= 2^31 - 65536, 1 <= E <= MOE_MAX_EXPERTS,
 * 1 <= K <= min(E, MOE_MAX_TOPK), T*K < 2^31 - 1.  T == 0 writes zero counts and
 * loss.  Asynchronous on `stream`; may be captured.
 */
MOE_API size_t moe_route_workspace_bytes(int32_t T, int32_t E);

MOE_API moe_status_t moe_route(const void *logits, int32_t bf16, int32_t T, int32_t E, int32_t K,
                               int32_t renormalize, float loss_coef, const uint8_t *token_mask,
                               int32_t *topk_ids, float *topk_weights, int32_t *expert_counts,
                               int32_t *routed_tokens, float *loss, void *workspace,
                               size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_route_backward -- the gradient of moe_route's weights and loss with
 * respect to the logits.
 *
 * The choice of experts and the counts are constants.  With dw = grad_weights,
 * w the weights, a[e] = grad_loss * coef * E * expert_counts[e] / (K n^2):
 *
 *   grad_logits[t,e] = p[t,e] (a[e] - sum over j of p[t,j] a[j])
 *     + renormalize == 1:  w[t,k] (dw[t,k] - sum over j of w[t,j] dw[t,j])
 *                          at e = topk_ids[t,k]
 *     + renormalize == 0:  p[t,e] ([e == topk_ids[t,k]] dw[t,k]
 *                          - sum over j of w[t,j] dw[t,j])
 *
 * computed in fp32 and rounded once to the logits' type.  The probabilities
 * are computed again from the logits.  A token whose ids are all outside [0,E)
 * gets zeros (so the mask need not be given again).
 *
 * topk_ids, expert_counts, routed_tokens: moe_route's outputs for the same
 * logits.  grad_weights [T,K] fp32 or NULL (zeros); grad_loss [1] fp32 on the
 * device or NULL (zero).  grad_logits [T,E] in the logits' type; must not
 * overlap the logits.  Sizes as for moe_route; T == 0 is a no-op.
 */
MOE_API moe_status_t moe_route_backward(const void *logits, int32_t bf16, int32_t T, int32_t E,
                                        int32_t K, int32_t renormalize, float loss_coef,
                                        const int32_t *topk_ids, const int32_t *expert_counts,
                                        const int32_t *routed_tokens, const float *grad_weights,
                                        const float *grad_loss, void *grad_logits,
                                        cudaStream_t stream);

/*
 * moe_route_grouped -- moe_route with softmax or sigmoid scores, a bias that
 * takes part in the choice alone, and groups of experts.
 *
 * Open experts and routed tokens are moe_route's.  With x the logits:
 *
 *   s[t,e]  MOE_SCORE_SIGMOID: 1 / (1 + exp(-x[t,e])), 0 where that is below
 *           2^-126 (x below -87.3); MOE_SCORE_SOFTMAX: moe_route's p[t,e]; 0 for an
 *           expert that is not open
 *   c[t,e]  s[t,e] + bias[e] of an open expert: what the choice goes by
 *   groups  expert e is in group e / (E / groups).  A group's value is the sum of
 *           its group_top (1 or 2) largest c (of its one open expert, the one c);
 *           the top_groups groups of largest value stay, ties to the lowest
 *           index, and only their experts can be chosen.
 *   topk_ids[t,:]      the K experts of largest c left, largest first, ties to
 *                      the lowest index; -1 where fewer are open
 *   topk_weights[t,k]  scale * s at topk_ids[t,k], s divided by the sum of the
 *                      token's K first when renormalize == 1 (all 0 where that is
 *                      0); 0 where topk_ids is -1
 *   expert_counts, routed_tokens, loss   moe_route's, with p[t,e] = s[t,e] / sum
 *                      over e' of s[t,e'] (0 where that is 0)
 *
 * The choice is that of exact arithmetic on the given logits and bias, as far as
 * 64 bits tell two values apart (equal ones go by index): where fp32 might order
 * two of them wrongly they are computed again more finely.  Scores, weights and
 * sums are fp32, the sums in an order that the sizes and the
 * alignment of logits fix.  A c that is NaN ranks below every number, and so does
 * a group's value with a NaN in it, before a group without an open expert; such
 * ones are equal.  Where the bias is the same for all, experts go by their logits,
 * NaN behind the numbers (fp32's lowest value ranks with it).  A NaN logit
 * of an open expert makes the loss NaN, and the weights in which its score takes
 * part; +inf is a score of 1 (sigmoid), or makes its token NaN (softmax).
 *
 * bias        [E] fp32 or NULL (zeros), 4-byte aligned; finite.  (A balance
 *             bias is moved between steps by expert_counts, with any rule.)
 * 1 <= groups <= MOE_MAX_GROUPS with E % groups == 0, 1 <= top_groups <= groups
 * (equal: all experts), K <= top_groups * (E / groups).
 * workspace   moe_route_grouped_workspace_bytes(T,E) bytes (0 for invalid sizes).
 * All else, and the limits, as for moe_route.
 */
MOE_API size_t moe_route_grouped_workspace_bytes(int32_t T, int32_t E);

MOE_API moe_status_t moe_route_grouped(const void *logits, int32_t bf16, int32_t T, int32_t E,
                                       int32_t K, int32_t scoring, const float *bias,
                                       int32_t groups, int32_t top_groups, int32_t group_top,
                                       int32_t renormalize, float scale, float loss_coef,
                                       const uint8_t *token_mask, int32_t *topk_ids,
                                       float *topk_weights, int32_t *expert_counts,
                                       int32_t *routed_tokens, float *loss, void *workspace,
                                       size_t workspace_bytes, cudaStream_t stream);

/*
 * moe_route_grouped_backward -- the gradient of moe_route_grouped's weights and
 * loss with respect to the logits.
 *
 * The choice and the counts are constants, so the bias and the groups play no
 * part.  With dw = scale * grad_weights, S the sum of the token's scores, sK that
 * of the chosen ones, a[e] = grad_loss * coef * E * expert_counts[e] / (K n^2):
 *
 *   g[t,e] = (a[e] - sum over j of p[t,j] a[j]) / S
 *     + renormalize == 1:  (dw[t,k] - sum over j of s[t,j] dw[t,j] / sK) / sK  and
 *     + renormalize == 0:  dw[t,k]                       at e = topk_ids[t,k]
 *   grad_logits[t,e] = sigmoid:  s[t,e] (1 - s[t,e]) g[t,e]
 *                      softmax:  s[t,e] (g[t,e] - sum over j of s[t,j] g[t,j])
 *
 * computed in fp32 and rounded once to the logits' type; the scores are computed
 * again from the logits.  A token whose ids are all outside [0,E) gets zeros.
 * Arguments, sizes and no-ops as for moe_route_backward.
 */
MOE_API moe_status_t moe_route_grouped_backward(const void *logits, int32_t bf16, int32_t T,
                                                int32_t E, int32_t K, int32_t scoring,
                                                int32_t renormalize, float scale, float loss_coef,
                                                const int32_t *topk_ids,
                                                const int32_t *expert_counts,
                                                const int32_t *routed_tokens,
                                                const float *grad_weights, const float *grad_loss,
                                                void *grad_logits, cudaStream_t stream);

/*
 * moe_dispatch_int8 -- moe_dispatch with rows quantised to int8.
 *
 * For every token t and k with 0 <= dst_row[t,k] < T*K:
 *
 *   scale = max |tokens[t, :]| * (1/127)                    (fp32 product with
 *                                                           the fp32 nearest 1/127)
 *   packed[dst_row[t,k], j] = rint(tokens[t, j] / scale)    (fp32 divide; ties
 *                             to even; in [-127, 127])
 *   scales[dst_row[t,k]] = scale
 *
 * A row of zeros stores scale 0 and codes 0.  A row that holds a NaN or an
 * infinity stores scale NaN and codes 0, so that what is computed from it is
 * NaN.  With K == 1 and dst_row[t] = t it quantises a matrix row by row.
 *
 * tokens  [T,H] bf16, 16-byte aligned.   dst_row [T,K] int32.
 * packed  [T*K,H] int8, 16-byte aligned.  scales [T*K] fp32, 4-byte aligned.
 * H >= 16 with H % 16 == 0.  T == 0 is a no-op.  Asynchronous on `stream`; may
 * be captured.
 */
MOE_API moe_status_t moe_dispatch_int8(const void *tokens, int32_t T, int32_t H, int32_t K,
                                       const int32_t *dst_row, void *packed, float *scales,
                                       cudaStream_t stream);

/*
 * moe_expert_matmul_int8 -- the experts' matrix product on packed int8 rows.
 *
 * The page multiplies the packed rows with the experts' weights between
 * dispatch and combine ("MoE all-to-all over EFA"); here both are 8-bit
 * integers, with a scale for each row and for each expert's output channel.
 * For the rows r of expert e, expert_offsets[e] <= r < expert_offsets[e+1]:
 *
 *   s = sum over h of x[r,h] * weights[e,n,h]
 *   out[r,n] = bf16(float(s) * x_scales[r] * w_scales[e,n])      (RN, ties to even)
 *
 * s is exact while its partial sums stay below 2^24.  Past that each step of the
 * sum (16 terms) may round or truncate to 24 bits: its error is then at most
 * 2^-23 of the sum of the terms' magnitudes for every 16 terms.  Rows outside
 * all experts' ranges are not written.  E == 1 with offsets {0, rows} is the
 * plain matrix product.
 *
 * x              [rows,H] int8, 16-byte aligned.   x_scales [rows] fp32.
 * weights        [E,N,H] int8, 16-byte aligned (a channel's H values together).
 * w_scales       [E,N] fp32.
 * expert_offsets [E+1] int32, moe_layout's; non-decreasing.  Offsets outside
 *                [0, rows] are taken as the nearer end.
 * out            [rows,N] bf16, 16-byte aligned; must not overlap the inputs.
 * dev_error      [1] uint32 or NULL.  Overwritten with 0, or with
 *                MOE_DEV_ERR_TIMEOUT when a bounded wait (2 s) between the
 *                kernel's warps expired; the outputs are then unspecified.
 * 0 <= rows <= 2^31 - 65536, 16 <= H <= 65536 with H % 16 == 0, N >= 1,
 * E*N <= 2^31 - 65536, 1 <= E <= MOE_MAX_EXPERTS.  rows == 0 is a no-op.
 * Asynchronous on `stream`; may be captured.
 */
MOE_API moe_status_t moe_expert_matmul_int8(const void *x, const float *x_scales,
                                            const void *weights, const float *w_scales,
                                            const int32_t *expert_offsets, int32_t rows,
                                            int32_t H, int32_t N, int32_t E, void *out,
                                            uint32_t *dev_error, cudaStream_t stream);

/*
 * moe_expert_matmul -- the experts' matrix product on packed bf16 rows, with
 * bias, activation and residual in the same pass.
 *
 * The page multiplies the packed rows with the experts' weights between
 * dispatch and combine ("MoE all-to-all over EFA").  For the rows r of expert e,
 * expert_offsets[e] <= r < expert_offsets[e+1]:
 *
 *   z[n]      = sum over h of x[r,h] * weights[e,n,h] + bias[e,n]    (fp32)
 *   pre[r,n]  = bf16(z[n])
 *   out[r,c]  = bf16(a(z)[c] + residual[r,c])      (RN, ties to even, rounded once)
 *
 * with a the activation (MOE_ACT_*).  MOE_ACT_SWIGLU takes z's first half as the
 * gate and its second as what it opens: out has C = N/2 channels, else C = N.
 * The activation takes z unrounded.  Rows outside all experts' ranges are not
 * written.  E == 1 with offsets {0, rows} is the plain matrix product (a shared
 * expert, whose residual may be the routed experts' sum).
 *
 * x              [rows,H] bf16.   weights [E,N,H] bf16 (a channel's H values together).
 * bias           [E,N] fp32 or NULL (zeros), 4-byte aligned.
 * expert_offsets [E+1] int32, moe_layout's; non-decreasing.  Offsets outside
 *                [0, rows] are taken as the nearer end.
 * residual       [rows,C] bf16 or NULL (zeros); may be out itself.
 * pre            [rows,N] bf16 or NULL: what the gradient needs.
 * out            [rows,C] bf16.  pre and out must not overlap the other inputs.
 * x, weights, residual, pre and out are 16-byte aligned.
 * dev_error      [1] uint32 or NULL.  Overwritten with 0, or with
 *                MOE_DEV_ERR_TIMEOUT when a bounded wait (2 s) between the
 *                kernel's warps expired; the outputs are then unspecified.
 * 0 <= rows <= 2^31 - 65536, 8 <= H <= 65536 with H % 8 == 0, N >= 1 (even for
 * MOE_ACT_SWIGLU), E*N <= 2^31 - 65536, 1 <= E <= MOE_MAX_EXPERTS.  rows == 0 is
 * a no-op.  Asynchronous on `stream`; may be captured.
 */
MOE_API moe_status_t moe_expert_matmul(const void *x, const void *weights, const float *bias,
                                       const int32_t *expert_offsets, int32_t rows, int32_t H,
                                       int32_t N, int32_t E, int32_t activation,
                                       const void *residual, void *pre, void *out,
                                       uint32_t *dev_error, cudaStream_t stream);

/*
 * moe_expert_activation_backward -- from the gradient at moe_expert_matmul's
 * out to the gradient at z, and its sum over each expert's rows.
 *
 *   grad_pre[r,n]  = bf16(g[r,n]),  g = grad_out[r,n] * a'(pre[r,n]); with
 *                    MOE_ACT_SWIGLU, for c < N/2 and s the logistic function of
 *                    pre[r,c]:  g[r,c] = grad_out[r,c] pre[r,N/2+c] s (1 + pre[r,c] (1 - s)),
 *                    g[r,N/2+c] = grad_out[r,c] pre[r,c] s
 *   grad_bias[e,n] = sum over the rows r of expert e of g[r,n]   (fp32, unrounded
 *                    g; in an order that the sizes and offsets fix)
 *
 * (The residual's gradient is grad_out.)  Rows outside all experts' ranges are
 * not written; an expert without rows gets zeros in grad_bias.
 *
 * pre        [rows,N] bf16, moe_expert_matmul's; may be NULL with MOE_ACT_NONE.
 * grad_out   [rows,C] bf16.   expert_offsets as for moe_expert_matmul.
 * grad_pre   [rows,N] bf16 or NULL (not wanted); may be pre itself, and without
 *            MOE_ACT_SWIGLU grad_out itself.
 * grad_bias  [E,N] fp32 or NULL (not wanted).  One of the two is wanted.
 * workspace  with grad_bias: moe_expert_activation_backward_workspace_bytes
 *            (0 for invalid sizes) bytes, 16-byte aligned; its contents on entry
 *            do not matter, and it is in use until the stream passes this call.
 * pre, grad_out and grad_pre are 16-byte aligned.  Sizes as for
 * moe_expert_matmul, with N % 8 == 0 (N % 16 == 0 for MOE_ACT_SWIGLU).  rows == 0
 * writes zeros to grad_bias.  Asynchronous on `stream`; may be captured.
 */
MOE_API size_t moe_expert_activation_backward_workspace_bytes(int32_t rows, int32_t N, int32_t E);

MOE_API moe_status_t moe_expert_activation_backward(const void *pre, const void *grad_out,
                                                    const int32_t *expert_offsets, int32_t rows,
                                                    int32_t N, int32_t E, int32_t activation,
                                                    void *grad_pre, float *grad_bias,
                                                    void *workspace, size_t workspace_bytes,
                                                    cudaStream_t stream);

/*
 * moe_expert_matmul_backward -- the gradients of moe_expert_matmul's product
 * with respect to its rows and weights.
 *
 *   grad_x[r,h]         = bf16(sum over n of grad_pre[r,n] * weights[e,n,h])
 *   grad_weights[e,n,h] = sum over the rows r of expert e of grad_pre[r,n] * x[r,h],
 *                         in bf16, or in fp32 (weights_f32 == 1), where
 *                         accumulate == 1 adds it to what grad_weights holds
 *
 * with fp32 sums.  Rows of grad_x outside all experts' ranges are not written;
 * an expert without rows gets zeros in grad_weights (with accumulate, it is left
 * as it is).
 *
 * grad_pre      [rows,N] bf16.   x [rows,H] bf16 (may be NULL without grad_weights).
 * weights       [E,N,H] bf16 (may be NULL without grad_x).
 * grad_x        [rows,H] bf16 or NULL (not wanted).
 * grad_weights  [E,N,H] bf16 or fp32, or NULL (not wanted).  One of the two is wanted.
 * All of these are 16-byte aligned; the outputs must not overlap the inputs.
 * expert_offsets, dev_error and sizes as for moe_expert_matmul, with N % 8 == 0.
 * rows == 0 writes zeros to grad_weights (without accumulate); dev_error is then
 * not written.  Asynchronous on `stream`; may be captured.
 */
MOE_API moe_status_t moe_expert_matmul_backward(const void *grad_pre, const void *x,
                                                const void *weights, const int32_t *expert_offsets,
                                                int32_t rows, int32_t H, int32_t N, int32_t E,
                                                void *grad_x, void *grad_weights,
                                                int32_t weights_f32, int32_t accumulate,
                                                uint32_t *dev_error, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LAYOUT_H */
