// head_api.hip -- the C ABI of include/vpa_head.h: host-side validation,
// workspace layout and launches.  As in api.hip, no HIP call happens before
// every argument has been checked.
#include <math.h>

#include "vpa_checks.h"
#include "vpa_head_internal.h"

namespace {

using namespace vpa;

// ---- token log probabilities ----

vpa_status check_counts(const vpa_vocab& v, int32_t n_tokens, int32_t n_top) {
    if (n_tokens < 0 || n_tokens > VPA_MAX_ROW_TOKENS)
        return fail(VPA_ERR_INVALID, "n_tokens %d outside [0, %d]", (int)n_tokens,
                    VPA_MAX_ROW_TOKENS);
    if (n_top < 0 || n_top > VPA_MAX_TOP || n_top > v.vocab)
        return fail(VPA_ERR_INVALID, "n_top %d outside [0, %d] or beyond the vocabulary",
                    (int)n_top, VPA_MAX_TOP);
    return ok();
}

// The task of a range of shards; n_parts = 0 makes one part of the whole row.
vpa_status check_logprob_task(const char* call, int dt, int64_t ld, const vpa_vocab& v,
                              int32_t first_shard, int32_t n_local, int64_t n_rows,
                              bool whole_rows, int32_t n_top, LogprobTask& t) {
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_vocab(v)) != VPA_OK ||
        (st = check_rows(call, n_rows)) != VPA_OK)
        return st;
    if (first_shard < 0 || n_local < 1 || (int64_t)first_shard + n_local > v.n_shards)
        return fail(VPA_ERR_INVALID, "shard range [%d, %d+%d) outside [0, %d)", (int)first_shard,
                    (int)first_shard, (int)n_local, (int)v.n_shards);
    const int64_t col0 = (int64_t)first_shard * v.shard_width;
    int64_t need = (int64_t)n_local * v.shard_width;
    need = v.vocab - col0 < need ? v.vocab - col0 : need;
    need = need < 1 ? 1 : need;
    if (ld < need || ld > ((int64_t)1 << 40))
        return fail(VPA_ERR_INVALID, "ld %lld outside [%lld valid local columns, 2^40]",
                    (long long)ld, (long long)need);
    t = LogprobTask{};
    t.ld = ld;
    t.vocab = (int32_t)v.vocab;
    // a range that starts past the vocabulary holds padding alone
    t.col0 = (int32_t)(col0 < v.vocab ? col0 : v.vocab);
    t.part_width = (int32_t)(whole_rows || v.shard_width > v.vocab ? v.vocab : v.shard_width);
    t.part_stride = v.shard_width;
    t.n_parts = whole_rows ? 1 : n_local;
    t.n_rows = (int32_t)n_rows;
    t.n_top = n_top;
    return ok();
}

vpa_status check_tokens(const int32_t* token_ids, int32_t n_tokens) {
    if (n_tokens > 0 && (!token_ids || !aligned(token_ids, 4)))
        return fail(VPA_ERR_INVALID, "token_ids is NULL or not 4-byte aligned");
    return ok();
}

// Shared checks of the calls that scan logits.
vpa_status check_logprob_scan(const char* call, int esize, const LogprobTask& t,
                              const void* logits, const void* ws, size_t ws_bytes) {
    if (!logits || !aligned(logits, (size_t)esize))
        return fail(VPA_ERR_INVALID, "logits is NULL or not aligned to its element size");
    const int64_t slots = (int64_t)t.n_parts * t.n_rows;
    if (slots > kMaxSize)
        return fail(VPA_ERR_INVALID, "%s: %lld rows over all shards exceed 2^31-1", call,
                    (long long)slots);
    const LogprobCut c = logprob_cut(esize, t.part_width, t.n_parts, t.n_rows);
    vpa_status st;
    if ((st = check_dispatch(logprob_threads(c), call)) != VPA_OK ||
        (st = check_dispatch(slots * 256, call)) != VPA_OK)
        return st;
    return check_workspace(call, ws, ws_bytes, logprob_workspace(c, t.n_top));
}

vpa_status check_logprob_out(const LogprobOut& o, int32_t n_top) {
    if (!o.row_stats || !aligned(o.row_stats, 4) || (o.lse && !aligned(o.lse, 4)))
        return fail(VPA_ERR_INVALID, "row_stats is NULL, or row_stats/lse not 4-byte aligned");
    if ((o.n_tokens > 0) != (o.logprobs != nullptr) || !aligned(o.logprobs, 4))
        return fail(VPA_ERR_INVALID, "logprobs is required exactly when tokens are given");
    if ((n_top > 0) != (o.top_ids != nullptr) || (n_top > 0) != (o.top_logprobs != nullptr) ||
        !aligned(o.top_ids, 4) || !aligned(o.top_logprobs, 4))
        return fail(VPA_ERR_INVALID, "top_ids and top_logprobs are required exactly when n_top > 0");
    return ok();
}

// ---- products ----

// A row stride at which rows begin at cache lines, so that products load them
// directly, and no load of 64 bytes touches two lines (2048 x 50257 x 2048,
// dz included: with dz's rows at multiples of 16 bytes the gradient of x takes
// 518 us and the weight's 617, at multiples of 128 bytes 455 and 594).
int64_t line_stride(int esize, int64_t n) {
    const int64_t vec = 128 / esize;
    return (n + vec - 1) / vec * vec;
}
size_t line_bytes(int esize, int64_t rows, int64_t cols) {
    return round256((size_t)rows * (size_t)line_stride(esize, cols) * (size_t)esize);
}
bool chunk_rows(int esize, const void* p, int64_t ld) {
    return ld % (16 / esize) == 0 && aligned(p, 16);
}

// Where inner is no multiple of 16 bytes, contiguous rows of x and weight are
// not aligned, and the products would load them through registers.  A large
// bf16 product copies them to aligned rows first: a pass at about 5 TB/s, a
// launch, against the products' loss, which is 0.6 of the time of the direct
// product forward and twice it in the backward pass (2048 x 8192 x 4097
// forward 200 -> 145 us; the gradients of 2048 x 8192 x 2047 239 -> 113 of x,
// 237 -> 104 of the weight).  fp32
// products lose less than a copy takes.
constexpr double kCopyUsAByte = 2.0 / 5e6, kProductUsAFlop = 1 / 1.1e9;
bool copy_pays(int esize, int64_t elements, double flops, double loss, double launches) {
    return esize == 2 && loss * flops * kProductUsAFlop >
                             (double)elements * esize * kCopyUsAByte + 4.0 * launches;
}
bool copies_forward(int esize, int64_t rows, int64_t outer, int64_t inner) {
    return rows > 64 && inner % (16 / esize) != 0 &&
           copy_pays(esize, (rows + outer) * inner, 2.0 * rows * outer * inner, 0.6, 2);
}
bool copies_backward(int esize, int64_t operand_rows, int64_t inner, double flops) {
    return inner % (16 / esize) != 0 &&
           copy_pays(esize, operand_rows * inner, flops, 2.0, 1);
}
// `p` in rows of line_stride() at `copy`
hipError_t copy_rows(int esize, const void* p, int64_t ld, int64_t rows, int64_t cols, void* copy,
                     hipStream_t stream) {
    DzTask d{};
    d.grad = p;
    d.ldg = ld;
    d.act = VPA_ACT_NONE;
    d.rows = rows;
    d.cols = cols;
    d.dz = copy;
    d.ldz = line_stride(esize, cols);
    return launch_dz(esize, d, stream);
}

// Workspace of the product: copies of x and weight, its slices of k.
struct LinearSizes {
    size_t x, w, gemm;
    size_t total() const { return x + w + gemm; }
};
LinearSizes linear_sizes(int esize, int64_t rows, int64_t outer, int64_t inner) {
    LinearSizes z{};
    if (copies_forward(esize, rows, outer, inner)) {
        z.x = line_bytes(esize, rows, inner);
        z.w = line_bytes(esize, outer, inner);
    }
    z.gemm = round256(gemm_workspace(esize, rows, outer, inner, true, true));
    return z;
}

// Workspace of the backward pass: dz, the bias sums' slices, copies of weight
// (for grad_x) and x (for grad_weight), the products'.
struct LinearGradSizes {
    size_t dz, part, w, x, gemm;
    size_t total() const { return dz + part + w + x + gemm; }
};
LinearGradSizes linear_grad_sizes(int esize, int64_t rows, int64_t outer, int64_t inner,
                                  bool dz, bool bias, bool gx, bool gw) {
    LinearGradSizes z{};
    const double flops = 2.0 * rows * outer * inner;
    if (dz && (gx || gw))
        z.dz = line_bytes(esize, rows, outer);
    if (bias)
        z.part = round256((size_t)dz_splits(rows, outer) * (size_t)outer * 4);
    if (gx && copies_backward(esize, outer, inner, flops))
        z.w = line_bytes(esize, outer, inner);
    if (gw && copies_backward(esize, rows, inner, flops))
        z.x = line_bytes(esize, rows, inner);
    const size_t wx = gx ? gemm_workspace(esize, rows, inner, outer, true, false) : 0;
    const size_t ww = gw ? gemm_workspace(esize, outer, inner, rows, false, false) : 0;
    z.gemm = round256(wx > ww ? wx : ww);
    return z;
}

// grad of type gdt, everything else of type dt.
vpa_status linear_backward(const void* grad, int64_t ldg, int gdt, const void* x, int64_t ldx,
                           const void* weight, int64_t ldw, const void* pre, int64_t ldp, int dt,
                           int64_t rows, int64_t outer, int64_t inner, int32_t act, void* grad_x,
                           int64_t ldgx, void* grad_weight, int64_t ldgw, void* grad_bias,
                           void* workspace, size_t workspace_bytes, hipStream_t s) {
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_dtype(gdt)) != VPA_OK ||
        (st = check_act(act)) != VPA_OK ||
        (st = check_sizes("vpa_head_linear_backward", rows, outer, inner)) != VPA_OK)
        return st;
    if (gdt != dt && gdt != VPA_F32)
        return fail(VPA_ERR_UNSUPPORTED, "grad_dtype %d: the operands' type or VPA_F32", gdt);
    const int e = esize_of(dt), ge = esize_of(gdt);
    const bool has_act = act != VPA_ACT_NONE;
    if (rows > 0) {
        if ((st = check_matrix("grad", grad, ge, ldg, outer)) != VPA_OK ||
            (has_act && (st = check_matrix("pre", pre, e, ldp, outer)) != VPA_OK) ||
            (grad_x && (st = check_matrix("weight", weight, e, ldw, inner)) != VPA_OK) ||
            (grad_x && (st = check_matrix("grad_x", grad_x, e, ldgx, inner)) != VPA_OK) ||
            (grad_weight && (st = check_matrix("x", x, e, ldx, inner)) != VPA_OK))
            return st;
    }
    if ((grad_weight &&
         (st = check_matrix("grad_weight", grad_weight, e, ldgw, inner)) != VPA_OK) ||
        (grad_bias && (st = check_vector("grad_bias", grad_bias, e)) != VPA_OK))
        return st;
    // without an activation dz is grad, unless it is of another type or its rows
    // are not aligned: a copy costs one pass over grad, the products' unaligned
    // loads more
    const bool copy = has_act || gdt != dt || !chunk_rows(e, grad, ldg);
    const LinearGradSizes z = linear_grad_sizes(e, rows, outer, inner, copy,
                                                grad_bias != nullptr, grad_x != nullptr,
                                                grad_weight != nullptr);
    if ((grad_x && (st = check_dispatch(gemm_threads(e, rows, inner, outer, true, false),
                                        "vpa_head_linear_backward")) != VPA_OK) ||
        (grad_weight && (st = check_dispatch(gemm_threads(e, outer, inner, rows, false, false),
                                             "vpa_head_linear_backward")) != VPA_OK) ||
        ((z.dz || grad_bias) &&
         (st = check_dispatch(dz_threads(rows, outer, grad_bias != nullptr),
                              "vpa_head_linear_backward")) != VPA_OK) ||
        ((z.w || z.x) && (st = check_dispatch(dz_threads(rows > outer ? rows : outer, inner, false),
                                              "vpa_head_linear_backward")) != VPA_OK))
        return st;
    if (rows > 0 && (st = check_workspace("vpa_head_linear_backward", workspace, workspace_bytes,
                                          z.total())) != VPA_OK)
        return st;
    char* ws = (char*)workspace;
    const void* dz = grad;
    int64_t lddz = ldg, dz_cols = outer;
    hipError_t he = hipSuccess;
    if (z.dz || grad_bias) {
        DzTask d{};
        d.grad = grad;
        d.ldg = ldg;
        d.grad_f32 = gdt == VPA_F32;
        d.pre = pre;
        d.ldp = ldp;
        d.act = act;
        d.rows = rows;
        d.cols = outer;
        d.dz = z.dz ? ws : nullptr;
        d.ldz = line_stride(e, outer);
        d.bias = grad_bias;
        // no rows: the sums have no slices, and the finishing kernel writes 0
        d.part = grad_bias && rows > 0 ? (float*)(ws + z.dz) : nullptr;
        if ((he = launch_dz(e, d, s)) != hipSuccess)
            return hip_fail(he, "vpa_head_linear_backward (dz) launch");
        if (z.dz) {
            dz = ws;
            lddz = dz_cols = d.ldz;
        }
    }
    char* wcopy = ws + z.dz + z.part;
    char* xcopy = wcopy + z.w;
    void* gws = ws ? xcopy + z.x : nullptr;
    if (grad_x && rows > 0) {
        GemmTask t{};
        t.a = dz;
        t.a_m = lddz;
        t.a_k = 1;
        t.b = weight;
        t.b_n = 1;
        t.b_k = ldw;
        t.a_k1 = true;
        t.m = t.m_readable = rows;
        t.n = t.n_readable = inner;
        if (z.w && !chunk_rows(e, weight, ldw)) {
            if ((he = copy_rows(e, weight, ldw, outer, inner, wcopy, s)) != hipSuccess)
                return hip_fail(he, "vpa_head_linear_backward (weight) launch");
            t.b = wcopy;
            t.b_k = t.n_readable = line_stride(e, inner);
        }
        t.k = outer;
        t.y = grad_x;
        t.ldy = ldgx;
        t.out_f32 = dt == VPA_F32;
        t.ws = gws;
        if ((he = launch_gemm(e, t, s)) != hipSuccess)
            return hip_fail(he, "vpa_head_linear_backward (grad_x) launch");
    }
    if (grad_weight) {
        GemmTask t{};
        t.a = dz;
        t.a_m = 1;
        t.a_k = lddz;
        t.b = x;
        t.b_n = 1;
        t.b_k = ldx;
        t.m = outer;
        t.m_readable = dz_cols;
        t.n = t.n_readable = inner;
        if (z.x && !chunk_rows(e, x, ldx)) {
            if ((he = copy_rows(e, x, ldx, rows, inner, xcopy, s)) != hipSuccess)
                return hip_fail(he, "vpa_head_linear_backward (x) launch");
            t.b = xcopy;
            t.b_k = t.n_readable = line_stride(e, inner);
        }
        t.k = rows;
        t.y = grad_weight;
        t.ldy = ldgw;
        t.out_f32 = dt == VPA_F32;
        t.ws = gws;
        if ((he = launch_gemm(e, t, s)) != hipSuccess)
            return hip_fail(he, "vpa_head_linear_backward (grad_weight) launch");
    }
    return ok();
}

}  // namespace

extern "C" {

size_t vpa_logprobs_workspace(vpa_vocab v, int32_t n_local_shards, int64_t n_rows, int32_t n_top) {
    if (check_vocab(v) != VPA_OK || n_local_shards < 1 || n_local_shards > v.n_shards ||
        n_rows < 1 || n_rows > kMaxSize || check_counts(v, 0, n_top) != VPA_OK)
        return 0;
    // either cut (whole rows or a part per shard), either element type
    const int64_t width = v.shard_width < v.vocab ? v.shard_width : v.vocab;
    size_t most = 0;
    for (int esize = 2; esize <= 4; esize += 2) {
        const int64_t cuts[2][2] = {{v.vocab, 1}, {width, n_local_shards}};
        for (const auto& c : cuts) {
            const size_t bytes = logprob_workspace(logprob_cut(esize, c[0], c[1], n_rows), n_top);
            most = bytes > most ? bytes : most;
        }
    }
    return most;
}

int32_t vpa_logprob_words(int32_t n_tokens, int32_t n_top) {
    if (n_tokens < 0 || n_tokens > VPA_MAX_ROW_TOKENS || n_top < 0 || n_top > VPA_MAX_TOP)
        return -1;
    return 3 + n_tokens + 2 * n_top;
}

vpa_status vpa_logprob_stats(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                             int32_t first_shard, int32_t n_local_shards, int64_t n_rows,
                             const int32_t* token_ids, int32_t n_tokens, int32_t n_top,
                             void* workspace, size_t workspace_bytes, int32_t* stats,
                             void* stream) {
    const int dt = dtype_value(&dtype);
    LogprobTask t;
    vpa_status st = check_logprob_task("vpa_logprob_stats", dt, ld, v, first_shard,
                                       n_local_shards, n_rows, false, n_top, t);
    if (st != VPA_OK || (st = check_counts(v, n_tokens, n_top)) != VPA_OK)
        return st;
    if (n_rows == 0)
        return ok();
    const int esize = esize_of(dt);
    if ((st = check_logprob_scan("vpa_logprob_stats", esize, t, logits, workspace,
                                 workspace_bytes)) != VPA_OK ||
        (st = check_tokens(token_ids, n_tokens)) != VPA_OK)
        return st;
    if (!stats || !aligned(stats, 4))
        return fail(VPA_ERR_INVALID, "stats is NULL or not 4-byte aligned");
    t.logits = logits;
    hipError_t e = launch_logprob_records(esize, t, workspace, token_ids, n_tokens, stats,
                                          (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_logprob_stats launch");
}

vpa_status vpa_combine_logprobs(const int32_t* stats, vpa_vocab v, int64_t n_rows,
                                const int32_t* token_ids, int32_t n_tokens, int32_t n_top,
                                float* logprobs, float* lse, float* row_stats, int32_t* top_ids,
                                float* top_logprobs, void* stream) {
    vpa_status st;
    if ((st = check_vocab(v)) != VPA_OK ||
        (st = check_rows("vpa_combine_logprobs", n_rows)) != VPA_OK ||
        (st = check_counts(v, n_tokens, n_top)) != VPA_OK)
        return st;
    if (n_rows == 0)
        return ok();
    if (!stats || !aligned(stats, 4))
        return fail(VPA_ERR_INVALID, "stats is NULL or not 4-byte aligned");
    const LogprobOut o = {token_ids, n_tokens, logprobs, lse, row_stats, top_ids, top_logprobs};
    if ((st = check_tokens(token_ids, n_tokens)) != VPA_OK ||
        (st = check_logprob_out(o, n_top)) != VPA_OK ||
        (st = check_dispatch(n_rows * 256, "vpa_combine_logprobs")) != VPA_OK)
        return st;
    hipError_t e = launch_logprob_combine(stats, v.n_shards, v.shard_width, (int32_t)v.vocab,
                                          (int32_t)n_rows, n_top, o, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_combine_logprobs launch");
}

vpa_status vpa_token_logprobs(const void* logits, vpa_dtype dtype, int64_t ld, vpa_vocab v,
                              int64_t n_rows, const int32_t* token_ids, int32_t n_tokens,
                              int32_t n_top, void* workspace, size_t workspace_bytes,
                              float* logprobs, float* lse, float* row_stats, int32_t* top_ids,
                              float* top_logprobs, void* stream) {
    const int dt = dtype_value(&dtype);
    LogprobTask t;
    vpa_status st = check_logprob_task("vpa_token_logprobs", dt, ld, v, 0, v.n_shards, n_rows,
                                       true, n_top, t);
    if (st != VPA_OK || (st = check_counts(v, n_tokens, n_top)) != VPA_OK)
        return st;
    if (n_rows == 0)
        return ok();
    const int esize = esize_of(dt);
    const LogprobOut o = {token_ids, n_tokens, logprobs, lse, row_stats, top_ids, top_logprobs};
    if ((st = check_logprob_scan("vpa_token_logprobs", esize, t, logits, workspace,
                                 workspace_bytes)) != VPA_OK ||
        (st = check_tokens(token_ids, n_tokens)) != VPA_OK ||
        (st = check_logprob_out(o, n_top)) != VPA_OK)
        return st;
    t.logits = logits;
    hipError_t e = launch_token_logprobs(esize, t, workspace, o, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_token_logprobs launch");
}

vpa_status vpa_token_logprobs_backward(const void* logits, vpa_dtype dtype, int64_t ld,
                                       vpa_vocab v, int32_t first_shard, int32_t n_local_shards,
                                       int64_t n_rows, const int32_t* token_ids,
                                       int32_t n_tokens, const float* row_stats,
                                       const float* grad_logprobs, const float* grad_entropy,
                                       void* grad_logits, int64_t grad_ld, int64_t grad_cols,
                                       void* stream) {
    const int dt = dtype_value(&dtype);
    LogprobTask t;
    vpa_status st = check_logprob_task("vpa_token_logprobs_backward", dt, ld, v, first_shard,
                                       n_local_shards, n_rows, false, 0, t);
    if (st != VPA_OK || (st = check_counts(v, n_tokens, 0)) != VPA_OK)
        return st;
    const int esize = esize_of(dt);
    int64_t cols = (int64_t)n_local_shards * v.shard_width;
    cols = v.vocab - t.col0 < cols ? v.vocab - t.col0 : cols;
    if (grad_cols < cols || grad_cols > kMaxSize || grad_ld < grad_cols ||
        grad_ld > ((int64_t)1 << 40))
        return fail(VPA_ERR_INVALID, "grad_cols %lld (row stride %lld) for %lld valid columns",
                    (long long)grad_cols, (long long)grad_ld, (long long)cols);
    if (n_rows == 0 || grad_cols == 0)
        return ok();
    if (!logits || !aligned(logits, (size_t)esize) || !grad_logits ||
        !aligned(grad_logits, (size_t)esize))
        return fail(VPA_ERR_INVALID, "logits/grad_logits NULL or not aligned to the element size");
    if (logits == grad_logits && ld != grad_ld)
        return fail(VPA_ERR_INVALID, "a gradient in the logits' place needs grad_ld = ld");
    if ((st = check_tokens(token_ids, n_tokens)) != VPA_OK)
        return st;
    if (!row_stats || !aligned(row_stats, 4) || !aligned(grad_entropy, 4) ||
        (n_tokens > 0) != (grad_logprobs != nullptr) || !aligned(grad_logprobs, 4))
        return fail(VPA_ERR_INVALID,
                    "row_stats is NULL, or grad_logprobs not given exactly with tokens, or a "
                    "pointer not 4-byte aligned");
    if ((st = check_dispatch(logprob_grad_threads(esize, grad_cols, n_rows),
                             "vpa_token_logprobs_backward")) != VPA_OK)
        return st;
    LogprobGradTask g{};
    g.logits = logits;
    g.ld = ld;
    g.vocab = t.vocab;
    g.col0 = t.col0;
    g.cols = (int32_t)cols;
    g.grad_cols = grad_cols;
    g.grad_ld = grad_ld;
    g.n_rows = t.n_rows;
    g.token_ids = token_ids;
    g.n_tokens = n_tokens;
    g.row_stats = row_stats;
    g.grad_logprobs = grad_logprobs;
    g.grad_entropy = grad_entropy;
    g.grad = grad_logits;
    hipError_t e = launch_logprob_grad(esize, g, (hipStream_t)stream);
    return e == hipSuccess ? ok() : hip_fail(e, "vpa_token_logprobs_backward launch");
}

size_t vpa_head_linear_workspace(vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner) {
    const int esize = esize_of(dtype_value(&dtype));
    if (!esize || rows < 1 || check_sizes("", rows, outer, inner) != VPA_OK)
        return 0;
    return linear_sizes(esize, rows, outer, inner).total();
}

size_t vpa_head_linear_backward_workspace(vpa_dtype dtype, int64_t rows, int64_t outer,
                                          int64_t inner) {
    const int esize = esize_of(dtype_value(&dtype));
    if (!esize || rows < 1 || check_sizes("", rows, outer, inner) != VPA_OK)
        return 0;
    return linear_grad_sizes(esize, rows, outer, inner, true, true, true, true).total();
}

size_t vpa_head_linear_backward_need(vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner,
                                     int32_t with_dz, int32_t need_x, int32_t need_weight,
                                     int32_t need_bias) {
    const int esize = esize_of(dtype_value(&dtype));
    if (!esize || rows < 1 || check_sizes("", rows, outer, inner) != VPA_OK)
        return 0;
    return linear_grad_sizes(esize, rows, outer, inner, with_dz != 0, need_bias != 0, need_x != 0,
                             need_weight != 0)
        .total();
}

vpa_status vpa_head_linear(const void* x, int64_t ldx, const void* weight, int64_t ldw,
                           const void* bias, const void* residual, int64_t ldr, vpa_dtype dtype,
                           int64_t rows, int64_t outer, int64_t inner, int32_t act, void* y,
                           int64_t ldy, vpa_dtype out_dtype, void* pre, int64_t ldp,
                           void* workspace, size_t workspace_bytes, void* stream) {
    const int dt = dtype_value(&dtype), odt = dtype_value(&out_dtype);
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_dtype(odt)) != VPA_OK ||
        (st = check_act(act)) != VPA_OK ||
        (st = check_sizes("vpa_head_linear", rows, outer, inner)) != VPA_OK)
        return st;
    if (odt != dt && odt != VPA_F32)
        return fail(VPA_ERR_UNSUPPORTED, "out_dtype %d: the operands' type or VPA_F32", odt);
    if (rows == 0)
        return ok();
    const int e = esize_of(dt);
    if ((st = check_matrix("x", x, e, ldx, inner)) != VPA_OK ||
        (st = check_matrix("weight", weight, e, ldw, inner)) != VPA_OK ||
        (st = check_matrix("y", y, esize_of(odt), ldy, outer)) != VPA_OK ||
        (bias && (st = check_vector("bias", bias, e)) != VPA_OK) ||
        (residual && (st = check_matrix("residual", residual, e, ldr, outer)) != VPA_OK) ||
        (pre && (st = check_matrix("pre", pre, e, ldp, outer)) != VPA_OK))
        return st;
    if (residual == y && residual && (ldr != ldy || odt != dt))
        return fail(VPA_ERR_INVALID, "y in the residual's place needs its row stride and type");
    const LinearSizes z = linear_sizes(e, rows, outer, inner);
    if ((st = check_dispatch(gemm_threads(e, rows, outer, inner, true, true),
                             "vpa_head_linear")) != VPA_OK ||
        (z.x && (st = check_dispatch(dz_threads(rows > outer ? rows : outer, inner, false),
                                     "vpa_head_linear")) != VPA_OK) ||
        (st = check_workspace("vpa_head_linear", workspace, workspace_bytes, z.total())) != VPA_OK)
        return st;
    GemmTask t{};
    t.a = x;
    t.a_m = ldx;
    t.a_k = 1;
    t.b = weight;
    t.b_n = ldw;
    t.b_k = 1;
    t.a_k1 = t.b_k1 = true;
    t.m = t.m_readable = rows;
    t.n = t.n_readable = outer;
    t.k = inner;
    t.bias = bias;
    t.residual = residual;
    t.ldr = ldr;
    t.y = y;
    t.ldy = ldy;
    t.out_f32 = odt == VPA_F32;
    t.pre = pre;
    t.ldp = ldp;
    t.act = act;
    char* ws = (char*)workspace;
    hipError_t he;
    if (z.x && !chunk_rows(e, x, ldx)) {
        if ((he = copy_rows(e, x, ldx, rows, inner, ws, (hipStream_t)stream)) != hipSuccess)
            return hip_fail(he, "vpa_head_linear (x) launch");
        t.a = ws;
        t.a_m = line_stride(e, inner);
    }
    if (z.w && !chunk_rows(e, weight, ldw)) {
        if ((he = copy_rows(e, weight, ldw, outer, inner, ws + z.x, (hipStream_t)stream)) !=
            hipSuccess)
            return hip_fail(he, "vpa_head_linear (weight) launch");
        t.b = ws + z.x;
        t.b_n = line_stride(e, inner);
    }
    t.ws = ws ? ws + z.x + z.w : nullptr;
    he = launch_gemm(e, t, (hipStream_t)stream);
    return he == hipSuccess ? ok() : hip_fail(he, "vpa_head_linear launch");
}

vpa_status vpa_head_linear_backward(const void* grad, int64_t ldg, const void* x, int64_t ldx,
                                    const void* weight, int64_t ldw, const void* pre, int64_t ldp,
                                    vpa_dtype dtype, int64_t rows, int64_t outer, int64_t inner,
                                    int32_t act, void* grad_x, int64_t ldgx, void* grad_weight,
                                    int64_t ldgw, void* grad_bias, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const int dt = dtype_value(&dtype);
    return linear_backward(grad, ldg, dt, x, ldx, weight, ldw, pre, ldp, dt, rows, outer, inner,
                           act, grad_x, ldgx, grad_weight, ldgw, grad_bias, workspace,
                           workspace_bytes, (hipStream_t)stream);
}

vpa_status vpa_head_linear_backward_typed(const void* grad, int64_t ldg, vpa_dtype grad_dtype,
                                          const void* x, int64_t ldx, const void* weight,
                                          int64_t ldw, const void* pre, int64_t ldp,
                                          vpa_dtype dtype, int64_t rows, int64_t outer,
                                          int64_t inner, int32_t act, void* grad_x, int64_t ldgx,
                                          void* grad_weight, int64_t ldgw, void* grad_bias,
                                          void* workspace, size_t workspace_bytes, void* stream) {
    return linear_backward(grad, ldg, dtype_value(&grad_dtype), x, ldx, weight, ldw, pre, ldp,
                           dtype_value(&dtype), rows, outer, inner, act, grad_x, ldgx, grad_weight,
                           ldgw, grad_bias, workspace, workspace_bytes, (hipStream_t)stream);
}

vpa_status vpa_layer_norm(const void* x, int64_t ldx, vpa_dtype dtype, const void* weight,
                          const void* bias, vpa_dtype wdtype, int64_t rows, int64_t cols,
                          float eps, void* y, int64_t ldy, float* mean, float* rstd,
                          void* stream) {
    const int dt = dtype_value(&dtype), wdt = dtype_value(&wdtype);
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_dtype(wdt)) != VPA_OK ||
        (st = check_rows("vpa_layer_norm", rows)) != VPA_OK)
        return st;
    if (wdt != dt && wdt != VPA_F32)
        return fail(VPA_ERR_UNSUPPORTED, "wdtype %d: the rows' type or VPA_F32", wdt);
    if (cols < 1 || cols > kMaxSize)
        return fail(VPA_ERR_INVALID, "cols %lld outside [1, 2^31)", (long long)cols);
    if (!(eps >= 0.0f) || !isfinite(eps))
        return fail(VPA_ERR_INVALID, "eps %g is not finite and >= 0", (double)eps);
    if (rows == 0)
        return ok();
    const int e = esize_of(dt), we = esize_of(wdt);
    if ((st = check_matrix("x", x, e, ldx, cols)) != VPA_OK ||
        (st = check_matrix("y", y, e, ldy, cols)) != VPA_OK ||
        (weight && (st = check_vector("weight", weight, we)) != VPA_OK) ||
        (bias && (st = check_vector("bias", bias, we)) != VPA_OK) ||
        (mean && (st = check_vector("mean", mean, 4)) != VPA_OK) ||
        (rstd && (st = check_vector("rstd", rstd, 4)) != VPA_OK))
        return st;
    if (x == y && ldx != ldy)
        return fail(VPA_ERR_INVALID, "y in x's place needs ldy = ldx");
    if ((st = check_dispatch(norm_threads(e, rows, cols), "vpa_layer_norm")) != VPA_OK)
        return st;
    const NormTask t = {x, ldx, weight, bias, we, rows, cols, eps, y, ldy, mean, rstd};
    hipError_t he = launch_norm(e, t, (hipStream_t)stream);
    return he == hipSuccess ? ok() : hip_fail(he, "vpa_layer_norm launch");
}

size_t vpa_layer_norm_backward_workspace(int64_t rows, int64_t cols) {
    if (rows < 0 || rows > kMaxSize || cols < 1 || cols > kMaxSize)
        return 0;
    const int32_t a = norm_splits(2, rows, cols), b = norm_splits(4, rows, cols);
    return round256((size_t)2 * (size_t)(a > b ? a : b) * (size_t)cols * 4);
}

vpa_status vpa_layer_norm_backward(const void* grad, int64_t ldg, const void* x, int64_t ldx,
                                   vpa_dtype dtype, const void* weight, vpa_dtype wdtype,
                                   const float* mean, const float* rstd, int64_t rows,
                                   int64_t cols, void* grad_x, int64_t ldgx, void* grad_weight,
                                   void* grad_bias, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    const int dt = dtype_value(&dtype), wdt = dtype_value(&wdtype);
    vpa_status st;
    if ((st = check_dtype(dt)) != VPA_OK || (st = check_dtype(wdt)) != VPA_OK ||
        (st = check_rows("vpa_layer_norm_backward", rows)) != VPA_OK)
        return st;
    if (wdt != dt && wdt != VPA_F32)
        return fail(VPA_ERR_UNSUPPORTED, "wdtype %d: the rows' type or VPA_F32", wdt);
    if (cols < 1 || cols > kMaxSize)
        return fail(VPA_ERR_INVALID, "cols %lld outside [1, 2^31)", (long long)cols);
    const int e = esize_of(dt), we = esize_of(wdt);
    if (rows > 0) {
        if ((st = check_matrix("grad", grad, e, ldg, cols)) != VPA_OK ||
            (st = check_matrix("x", x, e, ldx, cols)) != VPA_OK ||
            (st = check_vector("mean", mean, 4)) != VPA_OK ||
            (st = check_vector("rstd", rstd, 4)) != VPA_OK ||
            (weight && (st = check_vector("weight", weight, we)) != VPA_OK) ||
            (grad_x && (st = check_matrix("grad_x", grad_x, e, ldgx, cols)) != VPA_OK))
            return st;
        if (grad_x == grad && grad_x && ldgx != ldg)
            return fail(VPA_ERR_INVALID, "grad_x in grad's place needs ldgx = ldg");
        // long rows take the sums over rows after grad_x is written
        if (grad_x == grad && grad_x && (grad_weight || grad_bias))
            return fail(VPA_ERR_INVALID,
                        "grad_x in grad's place cannot be joined with grad_weight or grad_bias");
    }
    const bool sums = grad_weight || grad_bias;
    if ((grad_weight && (st = check_vector("grad_weight", grad_weight, we)) != VPA_OK) ||
        (grad_bias && (st = check_vector("grad_bias", grad_bias, we)) != VPA_OK) ||
        (st = check_dispatch(norm_grad_threads(e, rows, cols, grad_x != nullptr, sums),
                             "vpa_layer_norm_backward")) != VPA_OK)
        return st;
    if (sums && (st = check_workspace("vpa_layer_norm_backward", workspace, workspace_bytes,
                                      vpa_layer_norm_backward_workspace(rows, cols))) != VPA_OK)
        return st;
    const NormGradTask t = {grad, ldg,  x,      ldx,  weight,      we,        mean,
                            rstd, rows, cols,   grad_x, ldgx,      grad_weight, grad_bias,
                            (float*)workspace};
    hipError_t he = launch_norm_grad(e, t, (hipStream_t)stream);
    return he == hipSuccess ? ok() : hip_fail(he, "vpa_layer_norm_backward launch");
}

}  // extern "C"
