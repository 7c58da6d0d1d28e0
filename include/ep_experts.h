/*
 * ep_experts.h — C ABI of the operators on both sides of the plan: the router
 * that feeds it (ep_route and its backward) and the experts' 8-bit products
 * between dispatch and combine (ep_quantize_int8, ep_matmul_int8).
 *
 * The conventions of ep_plan.h hold: caller-owned buffers, calls asynchronous
 * on `stream`, host-checkable errors returned before anything is enqueued, no
 * device allocation, every call capturable in a CUDA graph.  Zero rows or
 * tokens are a call that does nothing.
 */
#ifndef EP_EXPERTS_GB300_H
#define EP_EXPERTS_GB300_H

#include "ep_plan.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EP_SCORE_SOFTMAX = 0, /* softmax over the token's experts */
    EP_SCORE_SIGMOID = 1  /* sigmoid of each logit */
} ep_score_t;

/* Flags of ep_route and ep_route_backward. */
#define EP_ROUTE_RENORMALIZE 1 /* divide the weights by their sum over the chosen experts */

/* Limits (checked; EP_ERR_INVALID beyond them). */
#define EP_MAX_GROUPS 32
#define EP_MAX_MATMUL_DIM 131056 /* the sum of so many products of codes stays below 2^31 */

/*
 * ep_route — the top-k experts of each token and their weights: the plan's
 * topk_idx and the combine's topk_weights.
 *
 * With s[t,e] = softmax(logits[t,:])[e] or sigmoid(logits[t,e]):
 *   - the experts of a token compete by s + bias (bias NULL: by s, compared as
 *     the logits, which order the same way);
 *   - with num_groups G > 1 the experts e*G/E.. form G equal blocks; a block's
 *     score is the sum of its two best experts' s + bias (of its one expert's,
 *     where it has only one available), and only the topk_groups best
 *     blocks' experts compete;
 *   - slot k of topk_idx is the (k+1)-th best expert; equal scores (and equal
 *     groups) go to the lower index;
 *   - topk_weights[t,k] = scale * s[t, topk_idx[t,k]], without the bias, with
 *     EP_ROUTE_RENORMALIZE divided by the sum over the chosen experts first
 *     (0 where that sum is 0).
 * An expert whose logit is -inf or NaN, or whose score is NaN, is not
 * available to the token and is left out of the softmax.  Slots without an
 * expert get index -1, the plan's unused slot, and weight 0; a token without
 * an available expert is a row of those.  A logit of +inf makes a softmax's
 * weights NaN (inf - inf).  Scores and sums are fp32; where the order of two
 * groups, or with a bias of two experts, hangs on scores that differ by less
 * than their rounding (2^-22 of the scores' range), either may come out; scores
 * that round to the same number are equal.
 *
 * logits_dev     [T,E], rows row_stride elements apart; EP_DTYPE_F32 or EP_DTYPE_BF16.
 * num_experts    E, 1..EP_MAX_EXPERTS; num_topk K, 1..min(E, EP_MAX_TOPK).
 * bias_dev       [E] fp32 or NULL; has no gradient.
 * num_groups     1..EP_MAX_GROUPS, divides E; topk_groups 1..num_groups.
 * topk_idx_dev   [T,K] int64; topk_weights_dev [T,K] fp32.
 */
ep_status_t ep_route(const void *logits_dev, ep_dtype_t logits_dtype, int64_t num_tokens, int num_experts,
                     int64_t row_stride, int num_topk, ep_score_t score, const float *bias_dev, int num_groups,
                     int topk_groups, int flags, float scale, int64_t *topk_idx_dev, float *topk_weights_dev,
                     ep_stream_t stream);

/*
 * ep_route_backward — grad_logits [T,E] (contiguous, the logits' type, every
 * element written) from grad_weights [T,K], the gradient of ep_route's
 * weights (the combine backward's grad_weights).  logits, score, flags and
 * scale are the forward's; topk_idx is its output: distinct experts in a row.
 * Entries outside [0,E) contribute nothing.
 */
ep_status_t ep_route_backward(const void *logits_dev, ep_dtype_t logits_dtype, int64_t num_tokens, int num_experts,
                              int64_t row_stride, int num_topk, ep_score_t score, int flags, float scale,
                              const int64_t *topk_idx_dev, const float *grad_weights_dev, void *grad_logits_dev,
                              ep_stream_t stream);

/*
 * ep_quantize_int8 — rows to 8-bit codes, one scale per row:
 * scale = max|v| * (1/127), code = round_half_even(v / scale) (IEEE fp32, 1/127
 * rounded to fp32 first), v = x, or with `gated` v = silu(x[:, :width]) * x[:, width:] in fp32.  A row of
 * zeros gets scale 0 and codes 0.  NaN elements are left out of the maximum
 * and get code 0; a row with an infinite element gets scale +inf and codes 0.
 *
 * x_dev          [rows, width] ([rows, 2*width] gated), rows row_stride elements
 *                apart; bf16 or fp32, 16-byte aligned rows; width % 8 == 0.
 * num_rows_dev   NULL, or a device count: rows at or beyond it are neither
 *                read nor written (the plan's N_exp, expert_offsets + E).
 * codes_dev      [rows,width] int8, 8-byte aligned; scales_dev [rows] fp32.
 */
ep_status_t ep_quantize_int8(const void *x_dev, ep_dtype_t x_dtype, int64_t rows, int64_t width, int64_t row_stride,
                             int gated, const int32_t *num_rows_dev, int8_t *codes_dev, float *scales_dev,
                             ep_stream_t stream);

/*
 * ep_matmul_int8 — rows of 8-bit codes times the experts' 8-bit weights:
 *
 *   out[r,n] = round( a_scales[s] * w_scales[e,n] * sum_k a[s,k] * w[e,n,k] )
 *
 * for offsets[e] <= r < offsets[e+1], s = rows[r] (s = r without rows).
 * Output rows whose s is -1 are zero; rows outside every expert's range are
 * not written.  The padding rows of the plan's segments are inside.
 * The sum is the exact integer as long as its running value stays within 2^24
 * (for k <= 1024 always); a longer sum beyond that is rounded like a sum in
 * fp32.  Results do not depend on timing: the same call gives the same bits.
 *
 * a_dev          [a_rows,k] int8, 16-byte aligned, k % 16 == 0, k >= 16.
 * w_dev          [num_experts,n,k] int8, 16-byte aligned; w_scales_dev
 *                [num_experts,n] fp32.
 * offsets_dev    [num_experts+1] int32, ascending (the plan's expert_offsets);
 *                NULL with one expert: all out_rows rows.  Values are clamped
 *                to [0,out_rows]; a last value beyond out_rows records
 *                EP_ERR_CAPACITY.
 * rows_dev       [out_rows] int32 (the plan's exp_src), or NULL.  An entry at
 *                or beyond a_rows gives a zero row and EP_ERR_CAPACITY.
 * out_dev        [out_rows,n] bf16 or fp32, 16-byte aligned.
 * Device-side errors are kept in one status word per device, which
 * ep_matmul_status reads.  The kernels' waits are bounded (EP_ERR_TIMEOUT).
 * Make the first call on a device before any stream capture: it loads the
 * library's device code.
 */
ep_status_t ep_matmul_int8(const int8_t *a_dev, const float *a_scales_dev, int64_t a_rows, const int8_t *w_dev,
                           const float *w_scales_dev, int num_experts, int64_t n, int64_t k,
                           const int32_t *offsets_dev, const int32_t *rows_dev, ep_dtype_t out_dtype, void *out_dev,
                           int64_t out_rows, ep_stream_t stream);

/*
 * ep_expert_matmul_int8 — ep_matmul_int8 over a plan: offsets are the handle's
 * expert_offsets; with `gather`, rows are its exp_src, so that a holds one row
 * per token and no dispatch is needed.  Device-side errors go to the handle's
 * status word (ep_sync_status); as after a plan's, later plans of the handle do
 * no work after EP_ERR_TIMEOUT until it is read there.
 */
ep_status_t ep_expert_matmul_int8(ep_handle_t handle, const int8_t *a_dev, const float *a_scales_dev, int64_t a_rows,
                                  const int8_t *w_dev, const float *w_scales_dev, int64_t n, int64_t k, int gather,
                                  ep_dtype_t out_dtype, void *out_dev, int64_t out_rows, ep_stream_t stream);

/*
 * ep_matmul_status — synchronises `stream`, returns an error that
 * ep_matmul_int8 calls recorded on the current device (EP_OK if none) and
 * clears it, and only it: of two errors the second is returned by the next
 * call, and one that a product on another stream records meanwhile is kept.
 */
ep_status_t ep_matmul_status(ep_stream_t stream);

/*
 * ep_debug_set_matmul_wait — test hook for the product kernels' bounded waits:
 * limit_us > 0 sets after how long a wait gives up and records EP_ERR_TIMEOUT
 * (0 restores the default, 2 s; a CTA's copies and products in flight are
 * waited for by the default always, before it ends); suppress nonzero makes one CTA load no
 * weights, so that the waits on them run out.  Process-wide; affects calls
 * made afterwards.
 */
void ep_debug_set_matmul_wait(int64_t limit_us, int suppress);

#ifdef __cplusplus
}
#endif

#endif /* EP_EXPERTS_GB300_H */
