/* _vpa_head_call: CPython marshalling of the launch entry points of
 * include/vpa_head.h, by the rules of _vpa_call (pycall.c): pointers are ints
 * or None, a vpa_vocab is three ints, the stream is its handle, and each
 * function returns the vpa_status.  bind(name, address) installs the address
 * of an entry point of the loaded libvpa.so.
 */
#include "pycall_args.h"
#include "vpa_head.h"

static __typeof__(&vpa_logprob_stats) p_logprob_stats;
static __typeof__(&vpa_combine_logprobs) p_combine_logprobs;
static __typeof__(&vpa_token_logprobs) p_token_logprobs;
static __typeof__(&vpa_token_logprobs_backward) p_token_logprobs_backward;
static __typeof__(&vpa_head_linear) p_head_linear;
static __typeof__(&vpa_head_linear_backward) p_head_linear_backward;
static __typeof__(&vpa_head_linear_backward_typed) p_head_linear_backward_typed;
static __typeof__(&vpa_head_linear_backward_need) p_head_linear_backward_need;
static __typeof__(&vpa_layer_norm) p_layer_norm;
static __typeof__(&vpa_layer_norm_backward) p_layer_norm_backward;

static const struct entry k_entries[] = {
    {"vpa_logprob_stats", (void**)&p_logprob_stats},
    {"vpa_combine_logprobs", (void**)&p_combine_logprobs},
    {"vpa_token_logprobs", (void**)&p_token_logprobs},
    {"vpa_token_logprobs_backward", (void**)&p_token_logprobs_backward},
    {"vpa_head_linear", (void**)&p_head_linear},
    {"vpa_head_linear_backward", (void**)&p_head_linear_backward},
    {"vpa_head_linear_backward_typed", (void**)&p_head_linear_backward_typed},
    {"vpa_head_linear_backward_need", (void**)&p_head_linear_backward_need},
    {"vpa_layer_norm", (void**)&p_layer_norm},
    {"vpa_layer_norm_backward", (void**)&p_layer_norm_backward},
};
#define N_ENTRIES ((int)(sizeof(k_entries) / sizeof(k_entries[0])))

static PyObject* py_logprob_stats(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *tokens, *ws, *stats, *stream;
    vpa_dtype dt;
    int64_t ld, n_rows;
    int32_t first, n_local, n_tokens, n_top;
    size_t ws_bytes;
    vpa_vocab v;
    if (!bound("vpa_logprob_stats", (const void*)p_logprob_stats) ||
        !parse("vpa_logprob_stats", args, nargs, "pdlViilpiipzpp", &logits, &dt, &ld, &v,
               &first, &n_local, &n_rows, &tokens, &n_tokens, &n_top, &ws, &ws_bytes, &stats,
               &stream))
        return NULL;
    RETURN_STATUS(p_logprob_stats(logits, dt, ld, v, first, n_local, n_rows, tokens, n_tokens,
                  n_top, ws, ws_bytes, stats, stream));
}

static PyObject* py_combine_logprobs(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *stats, *tokens, *logprobs, *lse, *row_stats, *top_ids, *top_logprobs, *stream;
    int64_t n_rows;
    int32_t n_tokens, n_top;
    vpa_vocab v;
    if (!bound("vpa_combine_logprobs", (const void*)p_combine_logprobs) ||
        !parse("vpa_combine_logprobs", args, nargs, "pVlpiipppppp", &stats, &v, &n_rows,
               &tokens, &n_tokens, &n_top, &logprobs, &lse, &row_stats, &top_ids, &top_logprobs,
               &stream))
        return NULL;
    RETURN_STATUS(p_combine_logprobs(stats, v, n_rows, tokens, n_tokens, n_top, logprobs, lse,
                  row_stats, top_ids, top_logprobs, stream));
}

static PyObject* py_token_logprobs(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *tokens, *ws, *logprobs, *lse, *row_stats, *top_ids, *top_logprobs, *stream;
    vpa_dtype dt;
    int64_t ld, n_rows;
    int32_t n_tokens, n_top;
    size_t ws_bytes;
    vpa_vocab v;
    if (!bound("vpa_token_logprobs", (const void*)p_token_logprobs) ||
        !parse("vpa_token_logprobs", args, nargs, "pdlVlpiipzpppppp", &logits, &dt, &ld, &v,
               &n_rows, &tokens, &n_tokens, &n_top, &ws, &ws_bytes, &logprobs, &lse, &row_stats,
               &top_ids, &top_logprobs, &stream))
        return NULL;
    RETURN_STATUS(p_token_logprobs(logits, dt, ld, v, n_rows, tokens, n_tokens, n_top, ws,
                  ws_bytes, logprobs, lse, row_stats, top_ids, top_logprobs, stream));
}

static PyObject* py_token_logprobs_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *tokens, *row_stats, *g_lp, *g_ent, *grad, *stream;
    vpa_dtype dt;
    int64_t ld, n_rows, grad_ld, grad_cols;
    int32_t first, n_local, n_tokens;
    vpa_vocab v;
    if (!bound("vpa_token_logprobs_backward", (const void*)p_token_logprobs_backward) ||
        !parse("vpa_token_logprobs_backward", args, nargs, "pdlViilpippppllp", &logits, &dt,
               &ld, &v, &first, &n_local, &n_rows, &tokens, &n_tokens, &row_stats, &g_lp, &g_ent,
               &grad, &grad_ld, &grad_cols, &stream))
        return NULL;
    RETURN_STATUS(p_token_logprobs_backward(logits, dt, ld, v, first, n_local, n_rows, tokens,
                  n_tokens, row_stats, g_lp, g_ent, grad, grad_ld, grad_cols, stream));
}

static PyObject* py_head_linear(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *x, *w, *bias, *res, *y, *pre, *ws, *stream;
    int64_t ldx, ldw, ldr, rows, outer, inner, ldy, ldp;
    vpa_dtype dt, odt;
    int32_t act;
    size_t ws_bytes;
    if (!bound("vpa_head_linear", (const void*)p_head_linear) ||
        !parse("vpa_head_linear", args, nargs, "plplppldlllipldplpzp", &x, &ldx, &w, &ldw,
               &bias, &res, &ldr, &dt, &rows, &outer, &inner, &act, &y, &ldy, &odt, &pre, &ldp,
               &ws, &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(p_head_linear(x, ldx, w, ldw, bias, res, ldr, dt, rows, outer, inner, act, y,
                  ldy, odt, pre, ldp, ws, ws_bytes, stream));
}

static PyObject* py_head_linear_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *grad, *x, *w, *pre, *gx, *gw, *gb, *ws, *stream;
    int64_t ldg, ldx, ldw, ldp, rows, outer, inner, ldgx, ldgw;
    vpa_dtype dt;
    int32_t act;
    size_t ws_bytes;
    if (!bound("vpa_head_linear_backward", (const void*)p_head_linear_backward) ||
        !parse("vpa_head_linear_backward", args, nargs, "plplplpldllliplplppzp", &grad,
               &ldg, &x, &ldx, &w, &ldw, &pre, &ldp, &dt, &rows, &outer, &inner, &act, &gx, &ldgx,
               &gw, &ldgw, &gb, &ws, &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(p_head_linear_backward(grad, ldg, x, ldx, w, ldw, pre, ldp, dt, rows, outer,
                  inner, act, gx, ldgx, gw, ldgw, gb, ws, ws_bytes, stream));
}

static PyObject* py_head_linear_backward_typed(PyObject* self, PyObject* const* args,
                                               Py_ssize_t nargs) {
    (void)self;
    void *grad, *x, *w, *pre, *gx, *gw, *gb, *ws, *stream;
    int64_t ldg, ldx, ldw, ldp, rows, outer, inner, ldgx, ldgw;
    vpa_dtype gdt, dt;
    int32_t act;
    size_t ws_bytes;
    if (!bound("vpa_head_linear_backward_typed", (const void*)p_head_linear_backward_typed) ||
        !parse("vpa_head_linear_backward_typed", args, nargs, "pldplplpldllliplplppzp", &grad,
               &ldg, &gdt, &x, &ldx, &w, &ldw, &pre, &ldp, &dt, &rows, &outer, &inner, &act, &gx,
               &ldgx, &gw, &ldgw, &gb, &ws, &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(p_head_linear_backward_typed(grad, ldg, gdt, x, ldx, w, ldw, pre, ldp, dt, rows,
                  outer, inner, act, gx, ldgx, gw, ldgw, gb, ws, ws_bytes, stream));
}

/* Host-only: the bytes of one call's workspace. */
static PyObject* py_head_linear_backward_need(PyObject* self, PyObject* const* args,
                                              Py_ssize_t nargs) {
    (void)self;
    vpa_dtype dt;
    int64_t rows, outer, inner;
    int32_t dz, need_x, need_w, need_b;
    if (!bound("vpa_head_linear_backward_need", (const void*)p_head_linear_backward_need) ||
        !parse("vpa_head_linear_backward_need", args, nargs, "dllliiii", &dt, &rows, &outer,
               &inner, &dz, &need_x, &need_w, &need_b))
        return NULL;
    return PyLong_FromSize_t(p_head_linear_backward_need(dt, rows, outer, inner, dz, need_x,
                                                         need_w, need_b));
}

static PyObject* py_layer_norm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *x, *w, *b, *y, *mean, *rstd, *stream;
    int64_t ldx, rows, cols, ldy;
    vpa_dtype dt, wdt;
    float eps;
    if (!bound("vpa_layer_norm", (const void*)p_layer_norm) ||
        !parse("vpa_layer_norm", args, nargs, "pldppdllfplppp", &x, &ldx, &dt, &w, &b, &wdt,
               &rows, &cols, &eps, &y, &ldy, &mean, &rstd, &stream))
        return NULL;
    RETURN_STATUS(p_layer_norm(x, ldx, dt, w, b, wdt, rows, cols, eps, y, ldy, mean, rstd,
                  stream));
}

static PyObject* py_layer_norm_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *grad, *x, *w, *mean, *rstd, *gx, *gw, *gb, *ws, *stream;
    int64_t ldg, ldx, rows, cols, ldgx;
    vpa_dtype dt, wdt;
    size_t ws_bytes;
    if (!bound("vpa_layer_norm_backward", (const void*)p_layer_norm_backward) ||
        !parse("vpa_layer_norm_backward", args, nargs, "plpldpdppllplpppzp", &grad, &ldg,
               &x, &ldx, &dt, &w, &wdt, &mean, &rstd, &rows, &cols, &gx, &ldgx, &gw, &gb, &ws,
               &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(p_layer_norm_backward(grad, ldg, x, ldx, dt, w, wdt, mean, rstd, rows, cols, gx,
                  ldgx, gw, gb, ws, ws_bytes, stream));
}

static PyObject* py_bind(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    return bind_entry(k_entries, N_ENTRIES, args, nargs);
}

static PyObject* py_entries(PyObject* self, PyObject* unused) {
    (void)self;
    (void)unused;
    return entry_names(k_entries, N_ENTRIES);
}

static PyMethodDef k_methods[] = {
    {"vpa_logprob_stats", FASTCALL(py_logprob_stats), "vpa_logprob_stats (include/vpa_head.h)"},
    {"vpa_combine_logprobs", FASTCALL(py_combine_logprobs), "vpa_combine_logprobs (include/vpa_head.h)"},
    {"vpa_token_logprobs", FASTCALL(py_token_logprobs), "vpa_token_logprobs (include/vpa_head.h)"},
    {"vpa_token_logprobs_backward", FASTCALL(py_token_logprobs_backward), "vpa_token_logprobs_backward (include/vpa_head.h)"},
    {"vpa_head_linear", FASTCALL(py_head_linear), "vpa_head_linear (include/vpa_head.h)"},
    {"vpa_head_linear_backward", FASTCALL(py_head_linear_backward), "vpa_head_linear_backward (include/vpa_head.h)"},
    {"vpa_head_linear_backward_typed", FASTCALL(py_head_linear_backward_typed), "vpa_head_linear_backward_typed (include/vpa_head.h)"},
    {"vpa_head_linear_backward_need", FASTCALL(py_head_linear_backward_need), "vpa_head_linear_backward_need (include/vpa_head.h)"},
    {"vpa_layer_norm", FASTCALL(py_layer_norm), "vpa_layer_norm (include/vpa_head.h)"},
    {"vpa_layer_norm_backward", FASTCALL(py_layer_norm_backward), "vpa_layer_norm_backward (include/vpa_head.h)"},
    {"bind", FASTCALL(py_bind), "bind(name, address): the entry point `name` is at `address`"},
    {"entries", py_entries, METH_NOARGS, "names of the entry points this module calls"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef k_module = {
    PyModuleDef_HEAD_INIT, "_vpa_head_call",
    "CPython marshalling of the head operators' launch entry points", -1, k_methods,
    NULL, NULL, NULL, NULL,
};

PyMODINIT_FUNC PyInit__vpa_head_call(void) { return PyModule_Create(&k_module); }
