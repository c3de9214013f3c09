/* _vpa_draft_call: CPython marshalling of the launch entry points of
 * include/vpa_draft.h, by the rules of _vpa_call (pycall.c): pointers are ints
 * or None, a vpa_vocab is three ints, the stream is its handle, and each
 * function returns the vpa_status.  bind(name, address) installs the address
 * of an entry point of the loaded libvpa.so.
 */
#include "pycall_args.h"
#include "vpa_draft.h"

static __typeof__(&vpa_sampled_verify) p_sampled_verify;
static __typeof__(&vpa_distill_loss) p_distill_loss;
static __typeof__(&vpa_distill_loss_backward) p_distill_loss_backward;
static __typeof__(&vpa_distill_loss_and_grad) p_distill_loss_and_grad;
static __typeof__(&vpa_rms_norm) p_rms_norm;
static __typeof__(&vpa_rms_norm_fp8) p_rms_norm_fp8;
static __typeof__(&vpa_rms_norm_backward) p_rms_norm_backward;
static __typeof__(&vpa_quantize_fp8) p_quantize_fp8;
static __typeof__(&vpa_head_linear_fp8) p_head_linear_fp8;
static __typeof__(&vpa_head_linear_fp8_fast) p_head_linear_fp8_fast;
static __typeof__(&vpa_head_linear_fp8_fast_workspace) p_head_linear_fp8_fast_workspace;

static const struct entry k_entries[] = {
    {"vpa_sampled_verify", (void**)&p_sampled_verify},
    {"vpa_distill_loss", (void**)&p_distill_loss},
    {"vpa_distill_loss_backward", (void**)&p_distill_loss_backward},
    {"vpa_distill_loss_and_grad", (void**)&p_distill_loss_and_grad},
    {"vpa_rms_norm", (void**)&p_rms_norm},
    {"vpa_rms_norm_fp8", (void**)&p_rms_norm_fp8},
    {"vpa_rms_norm_backward", (void**)&p_rms_norm_backward},
    {"vpa_quantize_fp8", (void**)&p_quantize_fp8},
    {"vpa_head_linear_fp8", (void**)&p_head_linear_fp8},
    {"vpa_head_linear_fp8_fast", (void**)&p_head_linear_fp8_fast},
    {"vpa_head_linear_fp8_fast_workspace", (void**)&p_head_linear_fp8_fast_workspace},
};
#define N_ENTRIES ((int)(sizeof(k_entries) / sizeof(k_entries[0])))

static PyObject* py_sampled_verify(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *ids, *probs, *accept_u, *sample_u, *temperature, *ws, *out, *sampled,
        *rejected, *stream;
    vpa_dtype dtype, qdtype;
    int64_t ld, n_req, ldq;
    int32_t k;
    size_t ws_bytes;
    vpa_vocab v;
    if (!bound("vpa_sampled_verify", (const void*)p_sampled_verify) ||
        !parse("vpa_sampled_verify", args, nargs, "pdlVlippdlppppzpppp", &logits, &dtype, &ld, &v,
               &n_req, &k, &ids, &probs, &qdtype, &ldq, &accept_u, &sample_u, &temperature, &ws,
               &ws_bytes, &out, &sampled, &rejected, &stream))
        return NULL;
    RETURN_STATUS(p_sampled_verify(logits, dtype, ld, v, n_req, k, ids, probs, qdtype, ldq,
                  accept_u, sample_u, temperature, ws, ws_bytes, out, sampled, rejected, stream));
}

static PyObject* py_distill_loss(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *ids, *lp, *ws, *loss, *stats, *stream;
    vpa_dtype dtype;
    int64_t ld, n_rows;
    int32_t n_top, tail;
    size_t ws_bytes;
    float temperature;
    vpa_vocab v;
    if (!bound("vpa_distill_loss", (const void*)p_distill_loss) ||
        !parse("vpa_distill_loss", args, nargs, "pdlVlppiifpzppp", &logits, &dtype, &ld, &v,
               &n_rows, &ids, &lp, &n_top, &tail, &temperature, &ws, &ws_bytes, &loss, &stats, &stream))
        return NULL;
    RETURN_STATUS(p_distill_loss(logits, dtype, ld, v, n_rows, ids, lp, n_top, tail, temperature,
                  ws, ws_bytes, loss, stats, stream));
}

static PyObject* py_distill_loss_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *ids, *lp, *stats, *g, *grad, *stream;
    vpa_dtype dtype;
    int64_t ld, n_rows, grad_ld, grad_cols;
    int32_t n_top;
    float temperature;
    vpa_vocab v;
    if (!bound("vpa_distill_loss_backward", (const void*)p_distill_loss_backward) ||
        !parse("vpa_distill_loss_backward", args, nargs, "pdlVlppifpppllp", &logits, &dtype, &ld,
               &v, &n_rows, &ids, &lp, &n_top, &temperature, &stats, &g, &grad, &grad_ld, &grad_cols,
               &stream))
        return NULL;
    RETURN_STATUS(p_distill_loss_backward(logits, dtype, ld, v, n_rows, ids, lp, n_top,
                  temperature, stats, g, grad, grad_ld, grad_cols, stream));
}

static PyObject* py_distill_loss_and_grad(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *logits, *ids, *lp, *g, *ws, *loss, *stats, *grad, *stream;
    vpa_dtype dtype;
    int64_t ld, n_rows, grad_ld, grad_cols;
    int32_t n_top, tail;
    size_t ws_bytes;
    float temperature;
    vpa_vocab v;
    if (!bound("vpa_distill_loss_and_grad", (const void*)p_distill_loss_and_grad) ||
        !parse("vpa_distill_loss_and_grad", args, nargs, "pdlVlppiifppzpppllp", &logits, &dtype,
               &ld, &v, &n_rows, &ids, &lp, &n_top, &tail, &temperature, &g, &ws, &ws_bytes, &loss,
               &stats, &grad, &grad_ld, &grad_cols, &stream))
        return NULL;
    RETURN_STATUS(p_distill_loss_and_grad(logits, dtype, ld, v, n_rows, ids, lp, n_top, tail,
                  temperature, g, ws, ws_bytes, loss, stats, grad, grad_ld, grad_cols, stream));
}

static PyObject* py_rms_norm(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *x, *res, *w, *summed, *y, *rstd, *stream;
    vpa_dtype dtype, wdtype;
    int64_t ldx, ldr, rows, cols, lds, ldy;
    float eps;
    if (!bound("vpa_rms_norm", (const void*)p_rms_norm) ||
        !parse("vpa_rms_norm", args, nargs, "pldplpdllfplplpp", &x, &ldx, &dtype, &res, &ldr, &w,
               &wdtype, &rows, &cols, &eps, &summed, &lds, &y, &ldy, &rstd, &stream))
        return NULL;
    RETURN_STATUS(p_rms_norm(x, ldx, dtype, res, ldr, w, wdtype, rows, cols, eps, summed, lds, y,
                  ldy, rstd, stream));
}

static PyObject* py_rms_norm_fp8(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *x, *res, *w, *summed, *y, *scale, *stream;
    vpa_dtype dtype, wdtype;
    int64_t ldx, ldr, rows, cols, lds, ldy, ldsc;
    float eps;
    if (!bound("vpa_rms_norm_fp8", (const void*)p_rms_norm_fp8) ||
        !parse("vpa_rms_norm_fp8", args, nargs, "pldplpdllfplplplp", &x, &ldx, &dtype, &res, &ldr,
               &w, &wdtype, &rows, &cols, &eps, &summed, &lds, &y, &ldy, &scale, &ldsc, &stream))
        return NULL;
    RETURN_STATUS(p_rms_norm_fp8(x, ldx, dtype, res, ldr, w, wdtype, rows, cols, eps, summed, lds,
                  y, ldy, scale, ldsc, stream));
}

static PyObject* py_rms_norm_backward(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *grad, *summed, *w, *rstd, *gs, *gx, *gw, *ws, *stream;
    vpa_dtype dtype, wdtype;
    int64_t ldg, lds, ldgs, rows, cols, ldgx;
    size_t ws_bytes;
    if (!bound("vpa_rms_norm_backward", (const void*)p_rms_norm_backward) ||
        !parse("vpa_rms_norm_backward", args, nargs, "plpldpdpplllplppzp", &grad, &ldg, &summed,
               &lds, &dtype, &w, &wdtype, &rstd, &gs, &ldgs, &rows, &cols, &gx, &ldgx, &gw, &ws,
               &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(p_rms_norm_backward(grad, ldg, summed, lds, dtype, w, wdtype, rstd, gs, ldgs,
                  rows, cols, gx, ldgx, gw, ws, ws_bytes, stream));
}

static PyObject* py_quantize_fp8(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void *x, *y, *scale, *stream;
    vpa_dtype dtype;
    int64_t ldx, rows, cols, ldy, ldsc;
    int32_t block_rows;
    if (!bound("vpa_quantize_fp8", (const void*)p_quantize_fp8) ||
        !parse("vpa_quantize_fp8", args, nargs, "pldlliplplp", &x, &ldx, &dtype, &rows, &cols,
               &block_rows, &y, &ldy, &scale, &ldsc, &stream))
        return NULL;
    RETURN_STATUS(p_quantize_fp8(x, ldx, dtype, rows, cols, block_rows, y, ldy, scale, ldsc,
                  stream));
}

static PyObject* call_linear_fp8(const char* name, __typeof__(&vpa_head_linear_fp8) fn,
                                 PyObject* const* args, Py_ssize_t nargs) {
    void *x, *xs, *w, *ws_scale, *bias, *res, *y, *ws, *stream;
    vpa_dtype odtype;
    int64_t ldx, ldxs, ldw, ldws, ldr, rows, outer, inner, ldy;
    int32_t act;
    size_t ws_bytes;
    if (!bound(name, (const void*)fn) ||
        !parse(name, args, nargs, "plplplplppllllipldpzp", &x, &ldx, &xs, &ldxs, &w, &ldw,
               &ws_scale, &ldws, &bias, &res, &ldr, &rows, &outer, &inner, &act, &y, &ldy, &odtype,
               &ws, &ws_bytes, &stream))
        return NULL;
    RETURN_STATUS(fn(x, ldx, xs, ldxs, w, ldw, ws_scale, ldws, bias, res, ldr, rows, outer, inner,
                  act, y, ldy, odtype, ws, ws_bytes, stream));
}

static PyObject* py_head_linear_fp8(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    return call_linear_fp8("vpa_head_linear_fp8", p_head_linear_fp8, args, nargs);
}

static PyObject* py_head_linear_fp8_fast(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    return call_linear_fp8("vpa_head_linear_fp8_fast", p_head_linear_fp8_fast, args, nargs);
}

/* Host-only: the bytes of one call's workspace. */
static PyObject* py_head_linear_fp8_fast_workspace(PyObject* self, PyObject* const* args,
                                                   Py_ssize_t nargs) {
    (void)self;
    int64_t rows, outer, inner;
    const char* name = "vpa_head_linear_fp8_fast_workspace";
    if (!bound(name, (const void*)p_head_linear_fp8_fast_workspace) ||
        !parse(name, args, nargs, "lll", &rows, &outer, &inner))
        return NULL;
    return PyLong_FromSize_t(p_head_linear_fp8_fast_workspace(rows, outer, inner));
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
    {"vpa_sampled_verify", FASTCALL(py_sampled_verify), "vpa_sampled_verify (include/vpa_draft.h)"},
    {"vpa_distill_loss", FASTCALL(py_distill_loss), "vpa_distill_loss (include/vpa_draft.h)"},
    {"vpa_distill_loss_backward", FASTCALL(py_distill_loss_backward), "vpa_distill_loss_backward (include/vpa_draft.h)"},
    {"vpa_distill_loss_and_grad", FASTCALL(py_distill_loss_and_grad), "vpa_distill_loss_and_grad (include/vpa_draft.h)"},
    {"vpa_rms_norm", FASTCALL(py_rms_norm), "vpa_rms_norm (include/vpa_draft.h)"},
    {"vpa_rms_norm_fp8", FASTCALL(py_rms_norm_fp8), "vpa_rms_norm_fp8 (include/vpa_draft.h)"},
    {"vpa_rms_norm_backward", FASTCALL(py_rms_norm_backward), "vpa_rms_norm_backward (include/vpa_draft.h)"},
    {"vpa_quantize_fp8", FASTCALL(py_quantize_fp8), "vpa_quantize_fp8 (include/vpa_draft.h)"},
    {"vpa_head_linear_fp8", FASTCALL(py_head_linear_fp8), "vpa_head_linear_fp8 (include/vpa_draft.h)"},
    {"vpa_head_linear_fp8_fast", FASTCALL(py_head_linear_fp8_fast), "vpa_head_linear_fp8_fast (include/vpa_draft.h)"},
    {"vpa_head_linear_fp8_fast_workspace", FASTCALL(py_head_linear_fp8_fast_workspace), "vpa_head_linear_fp8_fast_workspace (include/vpa_draft.h)"},
    {"bind", FASTCALL(py_bind), "bind(name, address): the entry point `name` is at `address`"},
    {"entries", py_entries, METH_NOARGS, "names of the entry points this module calls"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef k_module = {
    PyModuleDef_HEAD_INIT, "_vpa_draft_call",
    "CPython marshalling of the draft head operators' launch entry points", -1, k_methods,
    NULL, NULL, NULL, NULL,
};

PyMODINIT_FUNC PyInit__vpa_draft_call(void) { return PyModule_Create(&k_module); }
