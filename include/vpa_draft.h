/*
 * vpa_draft.h -- C ABI of the operators in libvpa that train a draft head from
 * a target's top tokens, run it in 8 bits and verify its drafts by sampling:
 * the distillation loss with its gradient, the root-mean-square norm with the
 * residual's addition, its backward pass and its form with an 8-bit output,
 * the product of 8-bit operands, and the sampled verification.
 *
 * They stand next to the operators of vpa.h and vpa_head.h:
 * vpa_sampled_verify takes the logits that vpa_verify_stats takes, for
 * requests that sample; the distillation takes the top ids and log
 * probabilities that vpa_token_logprobs returns; the norm and the product are
 * the 8-bit forms of the head's layers.
 *
 * The conventions of vpa_head.h hold: device pointers owned by the caller,
 * calls validate on the host, only enqueue on `stream` and never allocate or
 * synchronise, errors by status and vpa_last_error(), zero rows are a no-op,
 * results are deterministic.  Matrices are row-major with a row stride (ld)
 * in elements and contiguous columns; data pointers are aligned to their
 * element unless a call says more.  Element types VPA_F32 and VPA_BF16; sums
 * are fp32 or more; an output is rounded once, to nearest even.  Outputs must
 * not overlap inputs unless a call says so.  A workspace belongs to one call
 * at a time.
 *
 * An 8-bit matrix is OCP e4m3 (4 bits of exponent, 3 of mantissa, largest
 * value 448, no infinity) with an fp32 scale for each block of 128 columns:
 * element (r, c) stands for value(r, c) * scale(r, c / 128).
 */
#ifndef VPA_DRAFT_H
#define VPA_DRAFT_H

#include "vpa_head.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Sampled verification
 *
 * Request r owns logits rows r*(K+1) .. r*(K+1)+K, as in vpa_verify_stats.
 * p_j is the distribution of row j at the request's temperature T:
 * p_j(c) = exp(x_c / T) / sum exp(x / T).  Draft d = draft_ids[r][j], drawn
 * from q_j, is accepted iff
 *     accept_uniforms[r][j] * q_j(d) < p_j(d),
 * drafts after the first one that is not are dropped, and the position of
 * that one (position K if all are accepted) emits a token drawn from
 *     w = max(p_j - q_j, 0) at a rejected draft, w = p_j otherwise:
 * the least c with  sum of w(0..c) > sample_uniforms[r] * sum of w.
 * Sums and comparisons of that draw are in 64 bits, and those of an acceptance
 * where it is near: p_j(d) counts to within 2^-36 of its value, relatively.
 *
 *  - Without draft_probs q_j is 1 at the draft and 0 elsewhere (drafts that no
 *    model drew).
 *  - A placeholder draft (any id outside [0, V), such as -1) is not accepted,
 *    and its position draws from p_j: a request with fewer drafts ends in
 *    placeholders.  What rows after the first placeholder hold does not matter.
 *  - A temperature that is not a finite number of at least 2^-100 (0, negative,
 *    NaN) makes p_j 1 at the argmax in vpa.h's order and 0 elsewhere.  So does
 *    a row that has no distribution: all columns -inf, a NaN or +inf among them.
 *  - Where w is 0 everywhere (q_j above p_j at every column), w = p_j.
 *  - A NaN in draft_probs: a draft with it is not accepted, a column with it has
 *    w = 0.
 *  - A sample_uniforms value below 0 (or NaN) counts as 0; from 1 on it draws
 *    the last column with w > 0.
 * ------------------------------------------------------------------------ */

/* Workspace bytes of vpa_sampled_verify (0 if the sizes are invalid). */
size_t vpa_sampled_verify_workspace(vpa_vocab v, int64_t n_req, int32_t k);

/*  logits     [n_req*(K+1)][ld], every shard of a row side by side, ld >= V;
 *             n_req*(K+1) below 2^31; 0 <= K <= VPA_MAX_DRAFTS.
 *  draft_ids  int32 [n_req][K] (NULL iff K = 0).
 *  draft_probs  [n_req*K][ldq] of type probs_dtype, row r*K+j is q_j; ldq >= V;
 *             or NULL.
 *  accept_uniforms  float [n_req][K] (NULL iff K = 0), in [0, 1).
 *  sample_uniforms  double [n_req], in [0, 1).
 *  temperature  float [n_req], or NULL for 1.
 *  out_tokens   out, int32 [n_req][K+1]: accepted drafts, the drawn token, -1.
 *  num_sampled  out, int32 [n_req]: accepted + 1.
 *  num_rejected out, int32 [n_req]: K - accepted. */
vpa_status vpa_sampled_verify(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                              int64_t n_req, int32_t k, const int32_t* draft_ids,
                              const void* draft_probs, vpa_dtype probs_dtype, int64_t ldq,
                              const float* accept_uniforms, const double* sample_uniforms,
                              const float* temperature, void* workspace, size_t workspace_bytes,
                              int32_t* out_tokens, int32_t* num_sampled, int32_t* num_rejected,
                              void* stream);

/* ------------------------------------------------------------------------
 * Distillation from a teacher's top tokens
 *
 * q = softmax(x / t) over a row's V logits.  The temperature t is the student's
 * alone: the teacher names n_top tokens id_j with log probabilities l_j, which are
 * taken as they are.  A teacher softened by t as well is given by the log
 * probabilities of its own logits / t (vpa_token_logprobs of those); without a
 * tail l_j / t says the same, since p is made to sum to 1.
 *  - tail = 0: p_j = exp(l_j) / sum exp(l) over the named tokens, and
 *        loss = sum_j p_j (log p_j - log q(id_j)).
 *  - tail = 1: p_j = exp(l_j), and what they leave, p_0 = max(1 - sum p, 0), is
 *    compared with q_0, the sum of q over the columns not named:
 *        loss = sum_j p_j (log p_j - log q(id_j)) + p_0 (log p_0 - log q_0).
 * Terms with p = 0 are 0.  With P = sum p (+ p_0), the gradient by x_c is
 *        (q(c) P - sum_j p_j [c = id_j] - [c not named] p_0 q(c) / q_0) / t.
 *
 *  - An id of -1 names nothing.  A row that names nothing is a padding
 *    position: loss 0 and gradient 0, whatever its logits.
 *  - Any other id outside [0, V), a log probability that is NaN or +inf, or a
 *    row with a NaN or +inf among its logits gives loss and gradient NaN.
 *  - A named column that the student masks (-inf) with p > 0 gives loss +inf
 *    and the gradient of the formula.  A row whose columns are all -inf has
 *    loss +inf (0 where no p is positive) and gradient 0.
 * ------------------------------------------------------------------------ */
#define VPA_MAX_TEACHER_TOP 64  /* most named tokens of a row */
#define VPA_DISTILL_STATS 8     /* floats of a row in row_stats */

/* Workspace bytes of vpa_distill_loss and vpa_distill_loss_and_grad (0 if the
 * sizes are invalid). */
size_t vpa_distill_workspace(vpa_vocab v, int64_t n_rows);

/*  logits       [n_rows][ld], every shard of a row side by side, ld >= V.
 *  teacher_ids, teacher_logprobs  int32 and float [n_rows][n_top], as
 *               vpa_token_logprobs returns them; 1 <= n_top <= VPA_MAX_TEACHER_TOP.
 *  temperature  finite, from 2^-100 on.
 *  loss         out, float [n_rows].
 *  row_stats    out, float [n_rows][VPA_DISTILL_STATS], for the backward pass. */
vpa_status vpa_distill_loss(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                            int64_t n_rows, const int32_t* teacher_ids,
                            const float* teacher_logprobs, int32_t n_top, int32_t tail,
                            float temperature, void* workspace, size_t workspace_bytes,
                            float* loss, float* row_stats, void* stream);

/* Gradient of sum(grad_loss * loss) by the logits.
 *  temperature  the forward call's, as are the teacher's arrays.
 *  grad_loss    float [n_rows].
 *  grad_logits  out, [n_rows][grad_ld] of the logits' type: columns
 *               [0, grad_cols) are written, those past V with 0; grad_ld >=
 *               grad_cols >= V.  It may be the logits themselves (same
 *               pointer, grad_ld = ld), which are then replaced. */
vpa_status vpa_distill_loss_backward(const void* logits, vpa_dtype dtype, int64_t ld,
                                     vpa_vocab v, int64_t n_rows, const int32_t* teacher_ids,
                                     const float* teacher_logprobs, int32_t n_top,
                                     float temperature, const float* row_stats,
                                     const float* grad_loss, void* grad_logits, int64_t grad_ld,
                                     int64_t grad_cols, void* stream);

/* Both at once, for a step that knows grad_loss beforehand (the rows' weights
 * in a mean): the logits need not come from memory twice. */
vpa_status vpa_distill_loss_and_grad(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                                     int64_t n_rows, const int32_t* teacher_ids,
                                     const float* teacher_logprobs, int32_t n_top, int32_t tail,
                                     float temperature, const float* grad_loss, void* workspace,
                                     size_t workspace_bytes, float* loss, float* row_stats,
                                     void* grad_logits, int64_t grad_ld, int64_t grad_cols,
                                     void* stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm
 *
 * s = x + residual, rounded to x's type (s = x without a residual);
 * y = s rstd w, rstd = 1 / sqrt(mean of s^2 over the row + eps).  Squares are
 * summed in 64 bits; rstd is fp32 (so +inf where the root is below 2^-128: with
 * eps = 0, rows of zeros and of the smallest subnormals).  The weight is optional.
 * 1 <= cols < 2^31, and fewer than 2^22 rows of those that a workgroup's registers
 * do not hold (past 16384 bf16 or 8192 fp32 columns; in the backward pass 8192 of
 * either).
 * ------------------------------------------------------------------------ */
/*  x, residual, y  [rows][cols] of type `dtype`; residual may be NULL.  y may
 *              be x or residual (same pointer and row stride).
 *  weight      [cols] of type wdtype (`dtype` or VPA_F32), or NULL.
 *  eps         finite and >= 0.
 *  summed      out, [rows][cols] of type `dtype`: s; NULL iff residual is.  It
 *              may be x or residual (same pointer and row stride), not y.
 *  rstd        out, float [rows], or NULL. */
vpa_status vpa_rms_norm(const void* x, int64_t ldx, vpa_dtype dtype, const void* residual,
                        int64_t ldr, const void* weight, vpa_dtype wdtype, int64_t rows,
                        int64_t cols, float eps, void* summed, int64_t lds, void* y, int64_t ldy,
                        float* rstd, void* stream);

/* The same with y in 8 bits: each block of 128 columns of a row (the last may
 * be shorter) has the scale amax / 448, amax its largest |y| (at least
 * 2^-100), and y / scale, a division rounded to fp32, is rounded to nearest
 * even.  A block that holds a NaN or an infinity has scale NaN, and its
 * elements stand for NaN.
 *  y       out, e4m3 [rows][ldy].
 *  scale   out, float [rows][ld_scale], ld_scale >= ceil(cols / 128). */
vpa_status vpa_rms_norm_fp8(const void* x, int64_t ldx, vpa_dtype dtype, const void* residual,
                            int64_t ldr, const void* weight, vpa_dtype wdtype, int64_t rows,
                            int64_t cols, float eps, void* summed, int64_t lds, void* y,
                            int64_t ldy, float* scale, int64_t ld_scale, void* stream);

/* Workspace bytes of vpa_rms_norm_backward (0 if the sizes are invalid). */
size_t vpa_rms_norm_backward_workspace(int64_t rows, int64_t cols);

/* Backward pass for the gradients `grad` of y and, optionally, `grad_summed` of
 * s (what comes back along the residual).  With xh = s rstd and u = grad * w:
 *   grad_x      = grad_summed + rstd (u - xh mean(u xh))   [rows][cols]
 *   grad_weight = sum over rows of grad * xh               [cols], type wdtype
 * grad_x is the gradient of x and of the residual.  Either output may be NULL;
 * grad_x may be grad_summed, or grad where grad_weight is NULL (same pointer and
 * row stride).  rows = 0
 * clears grad_weight. */
vpa_status vpa_rms_norm_backward(const void* grad, int64_t ldg, const void* summed, int64_t lds,
                                 vpa_dtype dtype, const void* weight, vpa_dtype wdtype,
                                 const float* rstd, const void* grad_summed, int64_t ldgs,
                                 int64_t rows, int64_t cols, void* grad_x, int64_t ldgx,
                                 void* grad_weight, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ------------------------------------------------------------------------
 * 8-bit products
 * ------------------------------------------------------------------------ */
/* e4m3 values and scales of a matrix: blocks of block_rows x 128, block_rows 1
 * (activations) or 128 (weights), by the rule of vpa_rms_norm_fp8.
 *  y      out, e4m3 [rows][ldy].
 *  scale  out, float [ceil(rows / block_rows)][ld_scale]. */
vpa_status vpa_quantize_fp8(const void* x, int64_t ldx, vpa_dtype dtype, int64_t rows,
                            int64_t cols, int32_t block_rows, void* y, int64_t ldy, float* scale,
                            int64_t ld_scale, void* stream);

/* Workspace bytes of vpa_head_linear_fp8 and of vpa_head_linear_fp8_fast (may be
 * 0; 0 too if the sizes are invalid). */
size_t vpa_head_linear_fp8_workspace(int64_t rows, int64_t outer, int64_t inner);
size_t vpa_head_linear_fp8_fast_workspace(int64_t rows, int64_t outer, int64_t inner);

/* y = residual + act(x W^T + bias) of 8-bit operands: with blocks b of 128 of
 * the inner dimension,
 *   (x W^T)(m, n) = sum_b x_scale(m, b) w_scale(n / 128, b) sum_{k in b} x(m, k) W(n, k),
 * the inner sums exact products added in fp32, whatever the sizes and types.
 *  x        e4m3 [rows][ldx], x_scale float [rows][ldxs] (blocks of 1 x 128).
 *  weight   e4m3 [outer][ldw], w_scale float [ceil(outer/128)][ldws] (128 x 128).
 *           Rows of x and weight begin at multiples of 16 bytes (pointer, and
 *           ldx and ldw; all four strides are at most 2^21); what lies past a
 *           row's `inner` values does not matter.
 *  bias, residual  VPA_BF16, [outer] and [rows][outer], either may be NULL.
 *  y        out, of type out_dtype: VPA_BF16 or VPA_F32.  It may be the residual
 *           itself (same pointer and row stride, VPA_BF16).
 *  outer, inner >= 1, below 2^31; rows below 2^31.
 *  workspace  vpa_head_linear_fp8_workspace() bytes, 16-byte aligned (NULL if 0). */
vpa_status vpa_head_linear_fp8(const void* x, int64_t ldx, const float* x_scale, int64_t ldxs,
                               const void* weight, int64_t ldw, const float* w_scale,
                               int64_t ldws, const void* bias, const void* residual, int64_t ldr,
                               int64_t rows, int64_t outer, int64_t inner, int32_t act, void* y,
                               int64_t ldy, vpa_dtype out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The same with fewer digits in the inner sums, for callers who choose that: where
 * y is bf16 and has more than 64 rows they come from the matrix cores' 8-bit
 * instruction, at up to twice the rate of the others.  It cuts in every group of 8
 * products what lies below 2^-13 of the largest, so an inner sum is off by up to
 * 7 * 2^-13 of sum |x W|: little beside a result of about that size (random normal
 * operands end 1.4e-5 off, relatively; a step of bf16 is 2^-8), everything where
 * large products cancel.  Other results are vpa_head_linear_fp8's.  Workspace:
 * vpa_head_linear_fp8_fast_workspace() bytes. */
vpa_status vpa_head_linear_fp8_fast(const void* x, int64_t ldx, const float* x_scale, int64_t ldxs,
                                    const void* weight, int64_t ldw, const float* w_scale,
                                    int64_t ldws, const void* bias, const void* residual,
                                    int64_t ldr, int64_t rows, int64_t outer, int64_t inner,
                                    int32_t act, void* y, int64_t ldy, vpa_dtype out_dtype,
                                    void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VPA_DRAFT_H */
