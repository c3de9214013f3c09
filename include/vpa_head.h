/*
 * vpa_head.h -- C ABI of the language-model head's operators in libvpa: the
 * layer norm before the head, the head's products (residual block and LM
 * head) and the token log probabilities of the resulting logits, each with
 * its backward pass.
 *
 * They stand next to the greedy path of vpa.h: a draft or target model's
 * hidden states go through vpa_layer_norm and vpa_head_linear to the logits
 * that vpa_top_tokens and vpa_verify_stats reduce; requests that ask for log
 * probabilities, which the greedy path cannot serve, take
 * vpa_token_logprobs on the same sharded logits; and a draft head is trained
 * with the backward passes.
 *
 * The conventions of vpa.h hold: pointers are device memory owned by the
 * caller unless said otherwise, calls validate on the host, only enqueue on
 * `stream` and never allocate or synchronise, errors are reported by status
 * and vpa_last_error(), zero rows are a no-op, results are deterministic.
 *  - Matrices are row-major with a row stride (ld) in elements; columns are
 *    contiguous.  Data pointers must be aligned to their element.
 *  - Element types are VPA_F32 and VPA_BF16.  Sums, statistics and products
 *    are accumulated in fp32 (or in more than fp32's 24 bits) whatever the
 *    element type; an output is rounded once, to nearest even.
 *  - Outputs must not overlap inputs unless a call says so.
 */
#ifndef VPA_HEAD_H
#define VPA_HEAD_H

#include "vpa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Token log probabilities
 *
 * For a row x of V logits, lse = log sum_c exp(x_c), p_c = exp(x_c - lse),
 * entropy = -sum_c p_c log p_c (a term with p_c = 0 is 0), and the log
 * probability of token t is x_t - lse, computed as (x_t - M) - log sum_c
 * exp(x_c - M) for a logit M near the largest.
 *
 *  - A masked column holds -inf: its p is 0 and its log probability -inf.
 *  - A row whose valid columns are all -inf (the mask leaves nothing) has
 *    lse = -inf, every log probability -inf, entropy 0 and gradient 0.
 *  - A row that holds a NaN or +inf has no distribution: its lse, entropy,
 *    log probabilities and gradient are NaN.  Its top ids are still the
 *    first ids in the order below.
 *  - Token id -1 is a placeholder (a padding position): its log probability
 *    is 0 and it adds nothing to the gradient.  Any other id outside
 *    [0, V) gives NaN and adds nothing to the gradient.
 *  - Top alternatives are the first n_top columns in the order of vpa.h's
 *    argmax: larger value first, equal values by the lower id, NaN before
 *    every number.  n_top <= V.
 * ------------------------------------------------------------------------ */
#define VPA_MAX_TOP 64          /* most top alternatives per row */
#define VPA_MAX_ROW_TOKENS 64   /* most given tokens per row */

/* Workspace bytes vpa_token_logprobs and vpa_logprob_stats need for these
 * sizes (0 if they are invalid or n_rows is 0). */
size_t vpa_logprobs_workspace(vpa_vocab v, int32_t n_local_shards, int64_t n_rows, int32_t n_top);

/* int32 words of one (shard, row) record of vpa_logprob_stats:
 * 3 + n_tokens + 2*n_top, or -1 if the counts are invalid.  A record holds
 *   [0] the fp32 bits of M, a logit near the shard's maximum (-inf: none),
 *   [1] of sum 2^z over the shard's columns, z = (x - M) log2(e),
 *   [2] of sum z 2^z,
 *   [3, 3+n_tokens) of the row's given tokens' logits (tokens of other
 *       shards hold 0 there),
 *   then n_top pairs {fp32 bits, global id} in the order above, padded with
 *   {VPA_EMPTY_BITS, VPA_EMPTY_ID}. */
int32_t vpa_logprob_words(int32_t n_tokens, int32_t n_top);

/* Per-shard records of the local shards, for a job whose ranks hold one
 * vocabulary shard each: the records of all shards, gathered in rank order
 * along dim 0, are what vpa_combine_logprobs takes.
 *  logits, dtype, ld, v, first_shard, n_local_shards  as vpa_block_stats.
 *  token_ids  int32 [n_rows][n_tokens], or NULL with n_tokens = 0.
 *  workspace  at least vpa_logprobs_workspace(v, n_local_shards, ...) bytes,
 *             16-byte aligned; its contents do not matter.
 *  stats      out, int32 [n_local_shards][n_rows][words], 4-byte aligned. */
vpa_status vpa_logprob_stats(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                             int32_t first_shard, int32_t n_local_shards, int64_t n_rows,
                             const int32_t* token_ids, int32_t n_tokens, int32_t n_top,
                             void* workspace, size_t workspace_bytes, int32_t* stats,
                             void* stream);

/* Combination of all S shards' records.
 *  stats         int32 [S][n_rows][words].
 *  logprobs      out, float [n_rows][n_tokens]; NULL iff n_tokens = 0.
 *  lse           out, float [n_rows], or NULL.
 *  row_stats     out, float [n_rows][3]: a logit M near the row's maximum,
 *                log sum exp(x - M) and the entropy.  M and the log of the sum
 *                stay apart for the backward pass: lse = M + log sum has lost
 *                the second where M is large.
 *  top_ids       out, int32 [n_rows][n_top]; NULL iff n_top = 0.
 *  top_logprobs  out, float [n_rows][n_top]; NULL iff n_top = 0. */
vpa_status vpa_combine_logprobs(const int32_t* stats, vpa_vocab v, int64_t n_rows,
                                const int32_t* token_ids, int32_t n_tokens, int32_t n_top,
                                float* logprobs, float* lse, float* row_stats,
                                int32_t* top_ids, float* top_logprobs, void* stream);

/* Both steps on one GPU that holds every shard of a row side by side
 * (ld >= V); arguments as above, workspace for n_local_shards = S. */
vpa_status vpa_token_logprobs(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                              int64_t n_rows, const int32_t* token_ids, int32_t n_tokens,
                              int32_t n_top, void* workspace, size_t workspace_bytes,
                              float* logprobs, float* lse, float* row_stats, int32_t* top_ids,
                              float* top_logprobs, void* stream);

/* Gradient of sum(grad_logprobs * logprobs) + sum(grad_entropy * entropy) by
 * the logits of the local shards:
 *   grad_c = sum_j g_j [c = t_j] - p_c (sum_j g_j + g_H (log p_c + entropy)).
 *  row_stats      of the whole rows, as the forward call returned them.
 *  grad_logprobs  float [n_rows][n_tokens]; NULL iff n_tokens = 0.
 *  grad_entropy   float [n_rows], or NULL.
 *  grad_logits    out, [n_rows][grad_ld] of the logits' type: columns
 *                 [0, grad_cols) are written, those past the valid local
 *                 columns with 0; grad_ld >= grad_cols >= the valid local
 *                 columns.  It may be the logits themselves (same pointer,
 *                 grad_ld = ld), which are then replaced. */
vpa_status vpa_token_logprobs_backward(const void* logits, vpa_dtype dtype, int64_t ld,
                                       vpa_vocab v, int32_t first_shard, int32_t n_local_shards,
                                       int64_t n_rows, const int32_t* token_ids,
                                       int32_t n_tokens, const float* row_stats,
                                       const float* grad_logprobs, const float* grad_entropy,
                                       void* grad_logits, int64_t grad_ld, int64_t grad_cols,
                                       void* stream);

/* ------------------------------------------------------------------------
 * The head's products
 *
 * y = residual + act(x W^T + bias), x [rows][inner], W [outer][inner] (an LM
 * head's or a linear layer's weight as stored), y [rows][outer].  The
 * residual and the bias are optional.
 * ------------------------------------------------------------------------ */
typedef enum {
    VPA_ACT_NONE = 0,
    VPA_ACT_RELU = 1, /* max(z, 0); NaN stays NaN; slope 0 at z = 0 */
    VPA_ACT_GELU = 2, /* z Phi(z), Phi the normal distribution (erf) */
    VPA_ACT_SILU = 3  /* z / (1 + exp(-z)) */
} vpa_act;

/* Workspace bytes of vpa_head_linear and of vpa_head_linear_backward (which
 * may be 0; 0 too if the sizes are invalid). */
size_t vpa_head_linear_workspace(vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner);
size_t vpa_head_linear_backward_workspace(vpa_dtype dtype, int64_t rows, int64_t outer,
                                          int64_t inner);

/* What one call of the backward pass needs of it: with_dz is 0 only where act
 * is VPA_ACT_NONE, the gradient is of type `dtype`, its address is a multiple
 * of 16 bytes and its row stride too, so that the products read the gradient
 * itself; need_x, need_weight and need_bias say which outputs are not NULL. */
size_t vpa_head_linear_backward_need(vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner,
                                     int32_t with_dz, int32_t need_x, int32_t need_weight,
                                     int32_t need_bias);

/*  x, weight, bias, residual  of type `dtype`; bias [outer], residual
 *             [rows][outer], either may be NULL.  outer, inner >= 1, below
 *             2^31; rows below 2^31.
 *  y          out, of type out_dtype: `dtype`, or VPA_F32 (e.g. fp32 logits
 *             from bf16 operands).  y may be the residual itself (same
 *             pointer, row stride and type).
 *  pre        out, [rows][outer] of type `dtype` or NULL: x W^T + bias before
 *             the activation, which the backward pass of an activation needs.
 *  workspace  vpa_head_linear_workspace() bytes, 16-byte aligned (NULL if 0). */
vpa_status vpa_head_linear(const void* x, int64_t ldx, const void* weight, int64_t ldw,
                           const void* bias, const void* residual, int64_t ldr, vpa_dtype dtype,
                           int64_t rows, int64_t outer, int64_t inner, int32_t act, void* y,
                           int64_t ldy, vpa_dtype out_dtype, void* pre, int64_t ldp,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Backward pass for the gradient `grad` [rows][outer] of y.  With dz =
 * grad * act'(pre):
 *   grad_x      = dz W        [rows][inner]
 *   grad_weight = dz^T x      [outer][inner]
 *   grad_bias   = sum of dz's rows  [outer]
 * (the residual's gradient is `grad` itself).  All of type `dtype`; each
 * output may be NULL.  pre is required unless act is VPA_ACT_NONE; weight is
 * required for grad_x and x for grad_weight.  rows = 0 clears grad_weight and
 * grad_bias.  For bf16, dz is rounded to bf16 for the two products (their
 * operands' type) where an activation makes it differ from grad; grad_bias
 * sums the unrounded fp32 values.  With that rounding and pre's the gradients
 * of a silu layer are 0.0024 (relative) off 64 bits, where the rounding of the
 * results alone is 0.0017; callers who need more pass fp32 operands. */
vpa_status vpa_head_linear_backward(const void* grad, int64_t ldg, const void* x, int64_t ldx,
                                    const void* weight, int64_t ldw, const void* pre, int64_t ldp,
                                    vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner,
                                    int32_t act, void* grad_x, int64_t ldgx, void* grad_weight,
                                    int64_t ldgw, void* grad_bias, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* The same for a gradient of type grad_dtype: `dtype`, or VPA_F32 where
 * vpa_head_linear stored y in fp32 from bf16 operands.  dz is rounded to
 * `dtype` for the two products as with an activation; grad_bias sums the fp32
 * values.  Its workspace is vpa_head_linear_backward's. */
vpa_status vpa_head_linear_backward_typed(const void* grad, int64_t ldg, vpa_dtype grad_dtype,
                                          const void* x, int64_t ldx, const void* weight,
                                          int64_t ldw, const void* pre, int64_t ldp,
                                          vpa_dtype dtype, int64_t rows, int64_t outer,
                                          int64_t inner, int32_t act, void* grad_x, int64_t ldgx,
                                          void* grad_weight, int64_t ldgw, void* grad_bias,
                                          void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Layer norm
 *
 * y = (x - mean) rstd w + b over the `cols` elements of a row, mean and
 * variance of the row (biased), rstd = 1 / sqrt(variance + eps).  weight and
 * bias are optional.  Rows that a workgroup's registers hold (to 16384 bf16 or
 * 8192 fp32 columns, in the backward pass to 8192 of either) may be any
 * number below 2^31; of longer ones a call takes fewer than 2^22.
 * ------------------------------------------------------------------------ */
/*  x, y       [rows][cols] of type `dtype`, 1 <= cols < 2^31; y may be x
 *             itself (same pointer and row stride).
 *  weight, bias  [cols] of type wdtype (`dtype` or VPA_F32), or NULL.
 *  eps        finite and >= 0.
 *  mean, rstd out, float [rows], or NULL. */
vpa_status vpa_layer_norm(const void* x, int64_t ldx, vpa_dtype dtype, const void* weight,
                          const void* bias, vpa_dtype wdtype, int64_t rows, int64_t cols,
                          float eps, void* y, int64_t ldy, float* mean, float* rstd,
                          void* stream);

/* Workspace bytes of vpa_layer_norm_backward (0 if the sizes are invalid). */
size_t vpa_layer_norm_backward_workspace(int64_t rows, int64_t cols);

/* Backward pass for the gradient `grad` [rows][cols] of y.  With xh =
 * (x - mean) rstd and u = grad * w:
 *   grad_x      = rstd (u - mean(u) - xh mean(u xh))   [rows][cols]
 *   grad_weight = sum over rows of grad * xh           [cols], type wdtype
 *   grad_bias   = sum over rows of grad                [cols], type wdtype
 * Each output may be NULL; grad_x may be grad itself (same pointer and row
 * stride) where grad_weight and grad_bias are NULL.  rows = 0 clears
 * grad_weight and grad_bias.  The sums over rows have a fixed order. */
vpa_status vpa_layer_norm_backward(const void* grad, int64_t ldg, const void* x, int64_t ldx,
                                   vpa_dtype dtype, const void* weight, vpa_dtype wdtype,
                                   const float* mean, const float* rstd, int64_t rows,
                                   int64_t cols, void* grad_x, int64_t ldgx, void* grad_weight,
                                   void* grad_bias, void* workspace, size_t workspace_bytes,
                                   void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VPA_HEAD_H */
