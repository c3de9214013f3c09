// draft_api.hip -- the C ABI of include/vpa_draft.h: host-side validation,
// workspace layout and launches.  As in api.hip, no HIP call happens before
// every argument has been checked.
#include <math.h>

#include "vpa_checks.h"
#include "vpa_draft_internal.h"

namespace {

using namespace vpa;

// Whole rows of logits: types, sizes, the row stride.
vpa_status check_logits(const char* call, int dt, int64_t ld, const vpa_vocab& v, int64_t rows) {
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_vocab(v)) != VPA_OK ||
        (st = check_rows(call, rows)) != VPA_OK)
        return st;
    if (ld < v.vocab || ld > ((int64_t)1 << 40))
        return fail(VPA_ERR_INVALID, "%s: ld %lld outside [%lld, 2^40]", call, (long long)ld,
                    (long long)v.vocab);
    return ok();
}

// ---- distillation ----

// Everything but the loss's outputs and the gradient.
vpa_status check_distill(const char* call, const void* logits, int dt, int64_t ld,
                         const vpa_vocab& v, int64_t n_rows, const int32_t* ids,
                         const float* logprobs, int32_t n_top, float temperature,
                         DistillTask& t) {
    vpa_status st = check_logits(call, dt, ld, v, n_rows);
    if (st != VPA_OK)
        return st;
    if (n_top < 1 || n_top > VPA_MAX_TEACHER_TOP)
        return fail(VPA_ERR_INVALID, "%s: n_top %d outside [1, %d]", call, (int)n_top,
                    VPA_MAX_TEACHER_TOP);
    // (of less, 1 / t times a difference of logits would leave fp32)
    if (!(temperature >= 0x1p-100f) || !(temperature < INFINITY))
        return fail(VPA_ERR_INVALID, "%s: temperature %g is not finite and > 0 (from 2^-100 on)",
                    call, (double)temperature);
    if (n_rows > 0 && ((st = check_vector("logits", logits, esize_of(dt))) != VPA_OK ||
                       (st = check_vector("teacher_ids", ids, 4)) != VPA_OK ||
                       (st = check_vector("teacher_logprobs", logprobs, 4)) != VPA_OK))
        return st;
    t = DistillTask{};
    t.logits = logits;
    t.ld = ld;
    t.vocab = (int32_t)v.vocab;
    t.n_rows = (int32_t)n_rows;
    t.ids = ids;
    t.logprobs = logprobs;
    t.n_top = n_top;
    t.temperature = temperature;
    return ok();
}

vpa_status check_distill_loss(const char* call, int dt, const DistillTask& t, const void* ws,
                              size_t ws_bytes) {
    vpa_status st;
    if ((st = check_vector("loss", t.loss, 4)) != VPA_OK ||
        (st = check_vector("row_stats", t.row_stats, 4)) != VPA_OK ||
        (st = check_dispatch(distill_threads(esize_of(dt), t.vocab, t.n_rows), call)) != VPA_OK)
        return st;
    return check_workspace(call, ws, ws_bytes, distill_workspace(t.vocab, t.n_rows));
}

vpa_status check_distill_grad(const char* call, int dt, const DistillTask& t) {
    const int esize = esize_of(dt);
    if (t.grad_cols < t.vocab || t.grad_cols > kMaxSize || t.grad_ld < t.grad_cols ||
        t.grad_ld > ((int64_t)1 << 40))
        return fail(VPA_ERR_INVALID, "grad_cols %lld (row stride %lld) for %d columns",
                    (long long)t.grad_cols, (long long)t.grad_ld, (int)t.vocab);
    if (t.n_rows == 0)
        return ok();
    vpa_status st;
    if ((st = check_vector("grad_loss", t.grad_loss, 4)) != VPA_OK ||
        (st = check_vector("grad_logits", t.grad, esize)) != VPA_OK)
        return st;
    if (t.logits == t.grad && t.ld != t.grad_ld)
        return fail(VPA_ERR_INVALID, "a gradient in the logits' place needs grad_ld = ld");
    return check_dispatch(distill_grad_threads(esize, t.grad_cols, t.n_rows), call);
}

// ---- norm ----

vpa_status check_norm_sizes(const char* call, int dt, int wdt, bool weight, int64_t rows,
                            int64_t cols) {
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_dtype(wdt)) != VPA_OK ||
        (st = check_rows(call, rows)) != VPA_OK)
        return st;
    if (weight && wdt != dt && wdt != VPA_F32)
        return fail(VPA_ERR_UNSUPPORTED, "weight type %d: the matrix's type or VPA_F32", wdt);
    if (cols < 1 || cols > kMaxSize)
        return fail(VPA_ERR_INVALID, "%s: %lld columns outside [1, 2^31)", call, (long long)cols);
    return ok();
}

// Both forms of the forward pass; scale is null for y of x's type.
vpa_status rms_forward(const char* call, const void* x, int64_t ldx, int dt, const void* residual,
                       int64_t ldr, const void* weight, int wdt, int64_t rows, int64_t cols,
                       float eps, void* summed, int64_t lds, void* y, int64_t ldy, float* rstd,
                       bool fp8, float* scale, int64_t ld_scale, hipStream_t stream) {
    vpa_status st = check_norm_sizes(call, dt, wdt, weight != nullptr, rows, cols);
    if (st != VPA_OK)
        return st;
    if (!(eps >= 0.0f) || !(eps < INFINITY))
        return fail(VPA_ERR_INVALID, "%s: eps %g is not finite and >= 0", call, (double)eps);
    if ((residual != nullptr) != (summed != nullptr))
        return fail(VPA_ERR_INVALID, "%s: summed goes with a residual", call);
    if (rows == 0)
        return ok();
    const int e = esize_of(dt);
    if ((st = check_matrix("x", x, e, ldx, cols)) != VPA_OK ||
        (residual && (st = check_matrix("residual", residual, e, ldr, cols)) != VPA_OK) ||
        (summed && (st = check_matrix("summed", summed, e, lds, cols)) != VPA_OK) ||
        (st = check_matrix("y", y, fp8 ? 1 : e, ldy, cols)) != VPA_OK ||
        (fp8 && (st = check_matrix("scale", scale, 4, ld_scale,
                                   (cols + kScaleBlock - 1) / kScaleBlock)) != VPA_OK) ||
        (weight && (st = check_vector("weight", weight, esize_of(wdt))) != VPA_OK))
        return st;
    if (!aligned(rstd, 4))
        return fail(VPA_ERR_INVALID, "rstd not 4-byte aligned");
    if (y == summed)
        return fail(VPA_ERR_INVALID, "%s: y and summed are the same", call);
    if ((summed == x && lds != ldx) || (summed && summed == residual && lds != ldr) ||
        (y == x && (fp8 || ldy != ldx)) || (y == residual && (fp8 || ldy != ldr)))
        return fail(VPA_ERR_INVALID, "%s: an output in an input's place needs its row stride and type",
                    call);
    if ((st = check_dispatch(rms_threads(e, rows, cols), call)) != VPA_OK)
        return st;
    RmsTask t{};
    t.x = x;
    t.ldx = ldx;
    t.residual = residual;
    t.ldr = ldr;
    t.weight = weight;
    t.wsize = esize_of(wdt);
    t.rows = rows;
    t.cols = cols;
    t.eps = eps;
    t.summed = summed;
    t.lds = lds;
    t.y = y;
    t.ldy = ldy;
    t.rstd = rstd;
    t.scale = scale;
    t.ld_scale = ld_scale;
    const hipError_t he = launch_rms(e, t, stream);
    return he == hipSuccess ? ok() : hip_fail(he, call);
}

// ---- 8-bit products ----

// Both forms of the product.
vpa_status linear_fp8(const char* call, bool fast, const void* x, int64_t ldx,
                      const float* x_scale, int64_t ldxs, const void* weight, int64_t ldw,
                      const float* w_scale, int64_t ldws, const void* bias, const void* residual,
                      int64_t ldr, int64_t rows, int64_t outer, int64_t inner, int32_t act, void* y,
                      int64_t ldy, int odt, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
    vpa_status st;
    if ((st = check_dtype(odt)) != VPA_OK || (st = check_act(act)) != VPA_OK ||
        (st = check_sizes(call, rows, outer, inner)) != VPA_OK)
        return st;
    if (rows == 0)
        return ok();
    const int64_t blocks = (inner + kScaleBlock - 1) / kScaleBlock;
    if ((st = check_matrix("x", x, 16, ldx, inner)) != VPA_OK ||
        (st = check_matrix("x_scale", x_scale, 4, ldxs, blocks)) != VPA_OK ||
        (st = check_matrix("weight", weight, 16, ldw, inner)) != VPA_OK ||
        (st = check_matrix("w_scale", w_scale, 4, ldws, blocks)) != VPA_OK ||
        (bias && (st = check_vector("bias", bias, 2)) != VPA_OK) ||
        (residual && (st = check_matrix("residual", residual, 2, ldr, outer)) != VPA_OK) ||
        (st = check_matrix("y", y, esize_of(odt), ldy, outer)) != VPA_OK)
        return st;
    const int64_t most = (int64_t)1 << 21;
    if (ldx % 16 || ldw % 16 || ldx > most || ldw > most || ldxs > most || ldws > most)
        return fail(VPA_ERR_INVALID,
                    "%s: row strides %lld, %lld (multiples of 16), %lld or %lld (scales) above 2^21",
                    call, (long long)ldx, (long long)ldw, (long long)ldxs, (long long)ldws);
    if (y == residual && (ldy != ldr || odt != VPA_BF16))
        return fail(VPA_ERR_INVALID, "%s: y in the residual's place needs its stride and type",
                    call);
    const bool exact = !fast || odt == VPA_F32;
    if ((st = check_dispatch(fp8_threads(rows, outer, inner, exact), call)) != VPA_OK ||
        (st = check_workspace(call, workspace, workspace_bytes,
                              fp8_workspace(rows, outer, inner, exact))) != VPA_OK)
        return st;
    Fp8Task t{};
    t.exact = exact;
    GemmTask& g = t.g;
    g.a = x;
    g.a_m = ldx;
    g.a_k = 1;
    g.b = weight;
    g.b_n = ldw;
    g.b_k = 1;
    g.a_k1 = g.b_k1 = true;
    g.m = g.m_readable = rows;
    g.n = g.n_readable = outer;
    g.k = inner;
    g.bias = bias;
    g.residual = residual;
    g.ldr = ldr;
    g.y = y;
    g.ldy = ldy;
    g.out_f32 = odt == VPA_F32;
    g.act = act;
    g.ws = workspace;
    t.a_scale = x_scale;
    t.lda_scale = ldxs;
    t.b_scale = w_scale;
    t.ldb_scale = ldws;
    const hipError_t e = launch_fp8(t, stream);
    return e == hipSuccess ? ok() : hip_fail(e, call);
}

}  // namespace

extern "C" {

size_t vpa_sampled_verify_workspace(vpa_vocab v, int64_t n_req, int32_t k) {
    if (check_vocab(v) != VPA_OK || n_req < 1 || k < 0 || k > VPA_MAX_DRAFTS ||
        n_req > kMaxSize / (k + 1))
        return 0;
    // either element type's cut
    const size_t b2 = sample_workspace(sample_cut(2, v.vocab, n_req, k), n_req, k);
    const size_t b4 = sample_workspace(sample_cut(4, v.vocab, n_req, k), n_req, k);
    return b2 > b4 ? b2 : b4;
}

vpa_status vpa_sampled_verify(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                              int64_t n_req, int32_t k, const int32_t* draft_ids,
                              const void* draft_probs, vpa_dtype probs_dtype, int64_t ldq,
                              const float* accept_uniforms, const double* sample_uniforms,
                              const float* temperature, void* workspace, size_t workspace_bytes,
                              int32_t* out_tokens, int32_t* num_sampled, int32_t* num_rejected,
                              void* stream) {
    const char* call = "vpa_sampled_verify";
    const int dt = dtype_value(&dtype), qdt = dtype_value(&probs_dtype);
    vpa_status st = check_logits(call, dt, ld, v, n_req);
    if (st != VPA_OK)
        return st;
    if (k < 0 || k > VPA_MAX_DRAFTS)
        return fail(VPA_ERR_INVALID, "%s: k %d outside [0, %d]", call, (int)k, VPA_MAX_DRAFTS);
    if (n_req > kMaxSize / (k + 1))
        return fail(VPA_ERR_INVALID, "%s: %lld requests of %d rows exceed 2^31-1", call,
                    (long long)n_req, (int)k + 1);
    if (draft_probs) {
        if ((st = check_dtype(qdt)) != VPA_OK)
            return st;
        if (k == 0)
            return fail(VPA_ERR_INVALID, "%s: draft_probs without drafts", call);
    }
    if (n_req == 0)
        return ok();
    if ((st = check_vector("logits", logits, esize_of(dt))) != VPA_OK ||
        (draft_probs && (st = check_matrix("draft_probs", draft_probs, esize_of(qdt), ldq,
                                           v.vocab)) != VPA_OK) ||
        (k > 0 && ((st = check_vector("draft_ids", draft_ids, 4)) != VPA_OK ||
                   (st = check_vector("accept_uniforms", accept_uniforms, 4)) != VPA_OK)) ||
        (st = check_vector("sample_uniforms", sample_uniforms, 8)) != VPA_OK ||
        (st = check_vector("out_tokens", out_tokens, 4)) != VPA_OK ||
        (st = check_vector("num_sampled", num_sampled, 4)) != VPA_OK ||
        (st = check_vector("num_rejected", num_rejected, 4)) != VPA_OK)
        return st;
    if (!aligned(temperature, 4))
        return fail(VPA_ERR_INVALID, "temperature not 4-byte aligned");
    const SampleCut c = sample_cut(esize_of(dt), v.vocab, n_req, k);
    if ((st = check_dispatch(sample_threads(c, n_req, k), call)) != VPA_OK ||
        (st = check_workspace(call, workspace, workspace_bytes,
                              vpa_sampled_verify_workspace(v, n_req, k))) != VPA_OK)
        return st;
    SampleTask t{};
    t.logits = logits;
    t.ld = ld;
    t.vocab = (int32_t)v.vocab;
    t.n_req = (int32_t)n_req;
    t.k = k;
    t.draft_ids = draft_ids;
    t.probs = draft_probs;
    t.ldq = ldq;
    t.accept_u = accept_uniforms;
    t.sample_u = sample_uniforms;
    t.temperature = temperature;
    t.out_tokens = out_tokens;
    t.num_sampled = num_sampled;
    t.num_rejected = num_rejected;
    const hipError_t e = launch_sample(esize_of(dt), draft_probs ? esize_of(qdt) : 4, t, workspace,
                                       (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_sampled_verify launch");
}

size_t vpa_distill_workspace(vpa_vocab v, int64_t n_rows) {
    if (check_vocab(v) != VPA_OK || n_rows < 1 || n_rows > kMaxSize)
        return 0;
    return distill_workspace(v.vocab, n_rows);
}

vpa_status vpa_distill_loss(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                            int64_t n_rows, const int32_t* teacher_ids,
                            const float* teacher_logprobs, int32_t n_top, int32_t tail,
                            float temperature, void* workspace, size_t workspace_bytes,
                            float* loss, float* row_stats, void* stream) {
    const char* call = "vpa_distill_loss";
    const int dt = dtype_value(&dtype);
    DistillTask t;
    vpa_status st = check_distill(call, logits, dt, ld, v, n_rows, teacher_ids, teacher_logprobs,
                                  n_top, temperature, t);
    if (st != VPA_OK || n_rows == 0)
        return st;
    t.tail = tail != 0;
    t.loss = loss;
    t.row_stats = row_stats;
    if ((st = check_distill_loss(call, dt, t, workspace, workspace_bytes)) != VPA_OK)
        return st;
    const hipError_t e = launch_distill(esize_of(dt), t, workspace, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_distill_loss launch");
}

vpa_status vpa_distill_loss_backward(const void* logits, vpa_dtype dtype, int64_t ld,
                                     vpa_vocab v, int64_t n_rows, const int32_t* teacher_ids,
                                     const float* teacher_logprobs, int32_t n_top,
                                     float temperature, const float* row_stats,
                                     const float* grad_loss, void* grad_logits, int64_t grad_ld,
                                     int64_t grad_cols, void* stream) {
    const char* call = "vpa_distill_loss_backward";
    const int dt = dtype_value(&dtype);
    DistillTask t;
    vpa_status st = check_distill(call, logits, dt, ld, v, n_rows, teacher_ids, teacher_logprobs,
                                  n_top, temperature, t);
    if (st != VPA_OK)
        return st;
    t.row_stats = const_cast<float*>(row_stats);
    t.grad_loss = grad_loss;
    t.grad = grad_logits;
    t.grad_ld = grad_ld;
    t.grad_cols = grad_cols;
    if ((st = check_distill_grad(call, dt, t)) != VPA_OK || n_rows == 0)
        return st;
    if ((st = check_vector("row_stats", row_stats, 4)) != VPA_OK)
        return st;
    const hipError_t e = launch_distill_grad(esize_of(dt), t, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_distill_loss_backward launch");
}

vpa_status vpa_distill_loss_and_grad(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                                     int64_t n_rows, const int32_t* teacher_ids,
                                     const float* teacher_logprobs, int32_t n_top, int32_t tail,
                                     float temperature, const float* grad_loss, void* workspace,
                                     size_t workspace_bytes, float* loss, float* row_stats,
                                     void* grad_logits, int64_t grad_ld, int64_t grad_cols,
                                     void* stream) {
    const char* call = "vpa_distill_loss_and_grad";
    const int dt = dtype_value(&dtype);
    DistillTask t;
    vpa_status st = check_distill(call, logits, dt, ld, v, n_rows, teacher_ids, teacher_logprobs,
                                  n_top, temperature, t);
    if (st != VPA_OK)
        return st;
    t.tail = tail != 0;
    t.loss = loss;
    t.row_stats = row_stats;
    t.grad_loss = grad_loss;
    t.grad = grad_logits;
    t.grad_ld = grad_ld;
    t.grad_cols = grad_cols;
    if ((st = check_distill_grad(call, dt, t)) != VPA_OK || n_rows == 0 ||
        (st = check_distill_loss(call, dt, t, workspace, workspace_bytes)) != VPA_OK)
        return st;
    const hipError_t e = launch_distill_both(esize_of(dt), t, workspace, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_distill_loss_and_grad launch");
}

vpa_status vpa_rms_norm(const void* x, int64_t ldx, vpa_dtype dtype, const void* residual,
                        int64_t ldr, const void* weight, vpa_dtype wdtype, int64_t rows,
                        int64_t cols, float eps, void* summed, int64_t lds, void* y, int64_t ldy,
                        float* rstd, void* stream) {
    return rms_forward("vpa_rms_norm", x, ldx, dtype_value(&dtype), residual, ldr, weight,
                       dtype_value(&wdtype), rows, cols, eps, summed, lds, y, ldy, rstd, false,
                       nullptr, 0, (hipStream_t)stream);
}

vpa_status vpa_rms_norm_fp8(const void* x, int64_t ldx, vpa_dtype dtype, const void* residual,
                            int64_t ldr, const void* weight, vpa_dtype wdtype, int64_t rows,
                            int64_t cols, float eps, void* summed, int64_t lds, void* y,
                            int64_t ldy, float* scale, int64_t ld_scale, void* stream) {
    return rms_forward("vpa_rms_norm_fp8", x, ldx, dtype_value(&dtype), residual, ldr, weight,
                       dtype_value(&wdtype), rows, cols, eps, summed, lds, y, ldy, nullptr, true,
                       scale, ld_scale, (hipStream_t)stream);
}

size_t vpa_rms_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 1 || rows > kMaxSize || cols < 1 || cols > kMaxSize)
        return 0;
    const int32_t s2 = rms_splits(2, rows, cols), s4 = rms_splits(4, rows, cols);
    return round256((size_t)(s2 > s4 ? s2 : s4) * (size_t)cols * 4);
}

vpa_status vpa_rms_norm_backward(const void* grad, int64_t ldg, const void* summed, int64_t lds,
                                 vpa_dtype dtype, const void* weight, vpa_dtype wdtype,
                                 const float* rstd, const void* grad_summed, int64_t ldgs,
                                 int64_t rows, int64_t cols, void* grad_x, int64_t ldgx,
                                 void* grad_weight, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    const char* call = "vpa_rms_norm_backward";
    const int dt = dtype_value(&dtype), wdt = dtype_value(&wdtype);
    vpa_status st = check_norm_sizes(call, dt, wdt, weight || grad_weight, rows, cols);
    if (st != VPA_OK)
        return st;
    const int e = esize_of(dt);
    if (rows > 0) {
        if ((st = check_matrix("grad", grad, e, ldg, cols)) != VPA_OK ||
            (st = check_matrix("summed", summed, e, lds, cols)) != VPA_OK ||
            (st = check_vector("rstd", rstd, 4)) != VPA_OK ||
            (weight && (st = check_vector("weight", weight, esize_of(wdt))) != VPA_OK) ||
            (grad_summed &&
             (st = check_matrix("grad_summed", grad_summed, e, ldgs, cols)) != VPA_OK) ||
            (grad_x && (st = check_matrix("grad_x", grad_x, e, ldgx, cols)) != VPA_OK))
            return st;
        if (grad_x && ((grad_x == grad && (ldgx != ldg || grad_weight)) ||
                       (grad_x == grad_summed && ldgx != ldgs) || grad_x == summed))
            return fail(VPA_ERR_INVALID,
                        "%s: grad_x in the place of grad (without grad_weight) or grad_summed "
                        "needs its row stride",
                        call);
    }
    if (grad_weight && (st = check_vector("grad_weight", grad_weight, esize_of(wdt))) != VPA_OK)
        return st;
    if ((st = check_dispatch(rms_grad_threads(e, rows, cols, grad_x && rows > 0,
                                              grad_weight != nullptr),
                             call)) != VPA_OK)
        return st;
    const int32_t splits = rms_splits(e, rows, cols);
    if (rows > 0 && grad_weight &&
        (st = check_workspace(call, workspace, workspace_bytes,
                              round256((size_t)splits * (size_t)cols * 4))) != VPA_OK)
        return st;
    if ((!grad_x || rows == 0) && !grad_weight)
        return ok();
    RmsGradTask t{};
    t.grad = grad;
    t.ldg = ldg;
    t.summed = summed;
    t.lds = lds;
    t.weight = weight;
    t.wsize = esize_of(wdt);
    t.rstd = rstd;
    t.grad_summed = grad_summed;
    t.ldgs = ldgs;
    t.rows = rows;
    t.cols = cols;
    t.dx = rows > 0 ? grad_x : nullptr;
    t.lddx = ldgx;
    t.dweight = grad_weight;
    t.part = (float*)workspace;
    const hipError_t he = launch_rms_grad(e, t, (hipStream_t)stream);
    return he == hipSuccess ? ok() : hip_fail(he, "vpa_rms_norm_backward launch");
}

vpa_status vpa_quantize_fp8(const void* x, int64_t ldx, vpa_dtype dtype, int64_t rows,
                            int64_t cols, int32_t block_rows, void* y, int64_t ldy, float* scale,
                            int64_t ld_scale, void* stream) {
    const char* call = "vpa_quantize_fp8";
    const int dt = dtype_value(&dtype);
    vpa_status st = check_norm_sizes(call, dt, dt, false, rows, cols);
    if (st != VPA_OK)
        return st;
    if (block_rows != 1 && block_rows != kScaleBlock)
        return fail(VPA_ERR_INVALID, "%s: block_rows %d is neither 1 nor %d", call,
                    (int)block_rows, kScaleBlock);
    if (rows == 0)
        return ok();
    if ((st = check_matrix("x", x, esize_of(dt), ldx, cols)) != VPA_OK ||
        (st = check_matrix("y", y, 1, ldy, cols)) != VPA_OK ||
        (st = check_matrix("scale", scale, 4, ld_scale,
                           (cols + kScaleBlock - 1) / kScaleBlock)) != VPA_OK ||
        (st = check_dispatch(quant_threads(esize_of(dt), rows, cols, block_rows), call)) != VPA_OK)
        return st;
    const QuantTask t = {x, ldx, rows, cols, block_rows, y, ldy, scale, ld_scale};
    const hipError_t e = launch_quant(esize_of(dt), t, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_quantize_fp8 launch");
}

size_t vpa_head_linear_fp8_workspace(int64_t rows, int64_t outer, int64_t inner) {
    if (rows < 1 || check_sizes("", rows, outer, inner) != VPA_OK)
        return 0;
    return fp8_workspace(rows, outer, inner, true);
}

size_t vpa_head_linear_fp8_fast_workspace(int64_t rows, int64_t outer, int64_t inner) {
    if (rows < 1 || check_sizes("", rows, outer, inner) != VPA_OK)
        return 0;
    // for results of either type
    const size_t a = fp8_workspace(rows, outer, inner, false);
    const size_t b = fp8_workspace(rows, outer, inner, true);
    return a > b ? a : b;
}

vpa_status vpa_head_linear_fp8(const void* x, int64_t ldx, const float* x_scale, int64_t ldxs,
                               const void* weight, int64_t ldw, const float* w_scale,
                               int64_t ldws, const void* bias, const void* residual,
                               int64_t ldr, int64_t rows, int64_t outer, int64_t inner,
                               int32_t act, void* y, int64_t ldy, vpa_dtype out_dtype,
                               void* workspace, size_t workspace_bytes, void* stream) {
    return linear_fp8("vpa_head_linear_fp8", false, x, ldx, x_scale, ldxs, weight, ldw, w_scale, ldws,
                      bias, residual, ldr, rows, outer, inner, act, y, ldy, dtype_value(&out_dtype),
                      workspace, workspace_bytes, (hipStream_t)stream);
}

vpa_status vpa_head_linear_fp8_fast(const void* x, int64_t ldx, const float* x_scale, int64_t ldxs,
                                    const void* weight, int64_t ldw, const float* w_scale,
                                    int64_t ldws, const void* bias, const void* residual,
                                    int64_t ldr, int64_t rows, int64_t outer, int64_t inner,
                                    int32_t act, void* y, int64_t ldy, vpa_dtype out_dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    return linear_fp8("vpa_head_linear_fp8_fast", true, x, ldx, x_scale, ldxs, weight, ldw, w_scale, ldws,
                      bias, residual, ldr, rows, outer, inner, act, y, ldy, dtype_value(&out_dtype),
                      workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
