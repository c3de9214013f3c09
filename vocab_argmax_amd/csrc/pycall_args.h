/* pycall_args.h -- conversion of Python arguments to C ones, shared by the
 * marshalling modules _vpa_call (pycall.c) and _vpa_head_call (headcall.c). */
#ifndef VPA_PYCALL_ARGS_H
#define VPA_PYCALL_ARGS_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdarg.h>
#include <stdint.h>
#include <string.h>

#include "vpa.h"

_Static_assert(sizeof(vpa_dtype) == sizeof(int32_t), "vpa_dtype is passed as an int32");

static int to_i64(PyObject* o, int64_t* out) {
    long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return 0;
    *out = (int64_t)v;
    return 1;
}

static int to_i32(PyObject* o, int32_t* out) {
    long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_OverflowError, "%lld does not fit a 32-bit argument", v);
        return 0;
    }
    *out = (int32_t)v;
    return 1;
}

static int to_size(PyObject* o, size_t* out) {
    size_t v = PyLong_AsSize_t(o);
    if (v == (size_t)-1 && PyErr_Occurred()) return 0;
    *out = v;
    return 1;
}

static int to_ptr(PyObject* o, void** out) {
    if (o == Py_None) {
        *out = NULL;
        return 1;
    }
    unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) return 0;
    *out = (void*)(uintptr_t)v;
    return 1;
}

static int to_float(PyObject* o, float* out) {
    double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return 0;
    *out = (float)v;
    return 1;
}

/* Converts args[0..nargs) by `fmt`, one character per Python argument:
 *   p pointer (void**), l int64 (int64_t*), i int32 (int32_t*), z size_t
 *   (size_t*), f float (float*), d dtype (vpa_dtype*, an int32 value), V vocab (vpa_vocab*, three
 *   arguments), e epilogue (vpa_epilogue* storage, then const vpa_epilogue**
 *   set to it or to NULL). */
static int parse(const char* name, PyObject* const* args, Py_ssize_t nargs, const char* fmt,
                 ...) {
    Py_ssize_t want = 0;
    for (const char* f = fmt; *f; ++f) want += (*f == 'V') ? 3 : 1;
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, nargs);
        return 0;
    }
    va_list ap;
    va_start(ap, fmt);
    int ok = 1;
    Py_ssize_t a = 0;
    for (const char* f = fmt; ok && *f; ++f) {
        switch (*f) {
        case 'p':
            ok = to_ptr(args[a++], va_arg(ap, void**));
            break;
        case 'l':
            ok = to_i64(args[a++], va_arg(ap, int64_t*));
            break;
        case 'i':
            ok = to_i32(args[a++], va_arg(ap, int32_t*));
            break;
        case 'f':
            ok = to_float(args[a++], va_arg(ap, float*));
            break;
        case 'z':
            ok = to_size(args[a++], va_arg(ap, size_t*));
            break;
        case 'd': {
            int32_t v = 0;
            vpa_dtype* out = va_arg(ap, vpa_dtype*);
            ok = to_i32(args[a++], &v);
            /* the library reads the argument's bytes as an int, so any int32
             * reaches its own range check */
            if (ok) memcpy(out, &v, sizeof(v));
            break;
        }
        case 'V': {
            vpa_vocab* v = va_arg(ap, vpa_vocab*);
            ok = to_i64(args[a], &v->vocab) && to_i64(args[a + 1], &v->shard_width) &&
                 to_i32(args[a + 2], &v->n_shards);
            a += 3;
            break;
        }
        case 'e': {
            vpa_epilogue* e = va_arg(ap, vpa_epilogue*);
            const vpa_epilogue** pe = va_arg(ap, const vpa_epilogue**);
            PyObject* o = args[a++];
            if (o == Py_None) {
                *pe = NULL;
                break;
            }
            if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
                PyErr_SetString(PyExc_TypeError,
                                "an epilogue is None or a tuple (d2t, d2t_len, scale)");
                ok = 0;
                break;
            }
            void* d2t = NULL;
            double scale = 0.0;
            ok = to_ptr(PyTuple_GET_ITEM(o, 0), &d2t) &&
                 to_i64(PyTuple_GET_ITEM(o, 1), &e->d2t_len);
            if (ok) {
                scale = PyFloat_AsDouble(PyTuple_GET_ITEM(o, 2));
                ok = !(scale == -1.0 && PyErr_Occurred());
            }
            e->d2t = (const int64_t*)d2t;
            e->scale = (float)scale;
            *pe = e;
            break;
        }
        default:
            PyErr_Format(PyExc_SystemError, "%s: bad format character", name);
            ok = 0;
        }
    }
    va_end(ap);
    return ok;
}

static int bound(const char* name, const void* fn) {
    if (fn) return 1;
    PyErr_Format(PyExc_RuntimeError, "%s is not bound: call bind() with its address first", name);
    return 0;
}

#define RETURN_STATUS(call)                                                                     \
    do {                                                                                        \
        vpa_status st_;                                                                         \
        Py_BEGIN_ALLOW_THREADS st_ = (call);                                                    \
        Py_END_ALLOW_THREADS return PyLong_FromLong((long)st_);                                 \
    } while (0)

/* A module's entry points: name and where its bound address goes. */
struct entry {
    const char* name;
    void** slot;
};

static PyObject* bind_entry(const struct entry* entries, int n, PyObject* const* args,
                            Py_ssize_t nargs) {
    if (nargs != 2 || !PyUnicode_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "bind(name: str, address: int)");
        return NULL;
    }
    const char* name = PyUnicode_AsUTF8(args[0]);
    void* addr = NULL;
    if (!name || !to_ptr(args[1], &addr)) return NULL;
    if (!addr) {
        PyErr_Format(PyExc_ValueError, "bind(%s): null address", name);
        return NULL;
    }
    for (int i = 0; i < n; ++i) {
        if (strcmp(entries[i].name, name) == 0) {
            *entries[i].slot = addr;
            Py_RETURN_NONE;
        }
    }
    PyErr_Format(PyExc_KeyError, "%s is not an entry point this module calls", name);
    return NULL;
}

static PyObject* entry_names(const struct entry* entries, int n) {
    PyObject* t = PyTuple_New(n);
    if (!t) return NULL;
    for (int i = 0; i < n; ++i) {
        PyObject* s = PyUnicode_FromString(entries[i].name);
        if (!s) {
            Py_DECREF(t);
            return NULL;
        }
        PyTuple_SET_ITEM(t, i, s);
    }
    return t;
}

#define FASTCALL(f) (PyCFunction)(void (*)(void))(f), METH_FASTCALL

#endif /* VPA_PYCALL_ARGS_H */
