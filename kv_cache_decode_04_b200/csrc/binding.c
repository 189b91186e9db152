/*
 * binding.c -- the CPython side of the short calls: cache rows, page pool,
 * draft trees and packed prompts.
 *
 * These calls take their kernels 3 to 10 us, and through ctypes the host spent
 * as long on them again: a third in converting arguments, a third in asking
 * each tensor three things from bytecode.  Here one function per call asks the
 * tensors (device, contiguity, address), finds the stream and calls the C ABI.
 * No torch headers: a tensor is asked through its Python methods.  Shapes and
 * types are checked in __init__.py, values in the library.
 *
 * Every function takes (stream or None, tensors or None ..., numbers ...) and
 * returns the library's status code, or None when a tensor is not a contiguous
 * one on the current CUDA device (the caller then says which).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "gqa.h"

enum { MAX_TENSORS = 10, MAX_NUMBERS = 12 };

static PyObject *s_get_device, *s_is_contiguous, *s_data_ptr, *s_cuda_stream;
static PyObject *f_current_device, *f_current_stream; /* of torch, given to bind() */

/* The C ABI, by address: the library may be the release or the debug build. */
static struct {
    int (*prefill_packed)(const void *, const void *, const void *, const int32_t *, void *, int, int, int, int, int,
                          float, int, gqa_dtype, gqa_stream_t);
    int (*decode_tree)(const void *, const void *, const void *, const int32_t *, const int32_t *, const int64_t *,
                       const int32_t *, float, void *, int, int, int, int, int, int, int, int, gqa_dtype, void *,
                       size_t, gqa_stream_t);
    int (*cache_append)(const void *, const void *, const int32_t *, const int32_t *, int32_t *, void *, void *,
                        const int32_t *, int, int, int, int, int, int, int, gqa_dtype, gqa_stream_t);
    int (*cache_compact)(void *, void *, const int32_t *, const int32_t *, const int32_t *, const int32_t *, int32_t *,
                         int, int, int, int, int, int, int, gqa_dtype, gqa_stream_t);
    int (*pages_reserve)(int32_t *, int32_t *, const int32_t *, const int32_t *, void *, void *, int, int, int, int,
                         int, int, gqa_dtype, void *, size_t, gqa_stream_t);
    int (*pages_fork)(int32_t *, int32_t *, int32_t *, const int32_t *, const int32_t *, int, int, int, int, int,
                      gqa_stream_t);
    int (*pages_release)(int32_t *, int32_t *, const int32_t *, int, int, int, int, gqa_stream_t);
} abi;

typedef struct {
    void *p[MAX_TENSORS];       /* addresses, NULL for None */
    long long n[MAX_NUMBERS];   /* the numbers behind the tensors */
    double scale;               /* the number behind those, where a call has one */
    gqa_stream_t stream;
} Args;

static int ask_long(PyObject *o, PyObject *method, long long *v) {
    PyObject *r = PyObject_CallMethodNoArgs(o, method);
    if (!r) return -1;
    *v = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

/* wide: the last number is a size_t; the others are C ints.
   1: `a` is filled; 0: a tensor is not ready; -1: a Python error is set. */
static int take(PyObject *const *args, Py_ssize_t nargs, int tensors, int numbers, int wide, int scale, Args *a) {
    if (nargs != 1 + tensors + numbers + scale) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, %zd given", 1 + tensors + numbers + scale, nargs);
        return -1;
    }
    long long index = -1;
    for (int i = 0; i < tensors; ++i) {
        PyObject *t = args[1 + i];
        a->p[i] = NULL;
        if (t == Py_None) continue;
        long long device;
        if (ask_long(t, s_get_device, &device)) return -1;
        if (i == 0) index = device;
        if (device < 0 || device != index) return 0;
        PyObject *dense = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!dense) return -1;
        const int ok = PyObject_IsTrue(dense);
        Py_DECREF(dense);
        if (ok <= 0) return ok;
        PyObject *r = PyObject_CallMethodNoArgs(t, s_data_ptr);
        if (!r) return -1;
        a->p[i] = PyLong_AsVoidPtr(r);
        Py_DECREF(r);
        if (!a->p[i] && PyErr_Occurred()) return -1;
    }
    for (int i = 0; i < numbers; ++i) {
        a->n[i] = PyLong_AsLongLong(args[1 + tensors + i]);
        if (a->n[i] == -1 && PyErr_Occurred()) return -1;
        if (!(wide && i + 1 == numbers) && (a->n[i] > 0x7fffffffll || a->n[i] < -0x80000000ll)) {
            PyErr_SetString(PyExc_OverflowError, "a number does not fit a C int");
            return -1;
        }
    }
    if (scale) {
        a->scale = PyFloat_AsDouble(args[nargs - 1]);
        if (a->scale == -1.0 && PyErr_Occurred()) return -1;
    }
    /* the tensors' device is the current one */
    PyObject *d = PyObject_CallNoArgs(f_current_device);
    if (!d) return -1;
    const long long current = PyLong_AsLongLong(d);
    if (current == -1 && PyErr_Occurred()) {
        Py_DECREF(d);
        return -1;
    }
    PyObject *h = NULL;
    if (current == index) h = args[0] == Py_None ? PyObject_CallOneArg(f_current_stream, d)
                                                 : PyObject_GetAttr(args[0], s_cuda_stream);
    Py_DECREF(d);
    if (current != index) return 0;
    if (!h) return -1;
    a->stream = (gqa_stream_t)PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    return !a->stream && PyErr_Occurred() ? -1 : 1;
}

/* Runs `call` (which sets rc) without the interpreter lock, as ctypes does. */
#define CALL(tensors, numbers, wide, scale, call)                                  \
    Args a;                                                                   \
    int rc = take(args, nargs, tensors, numbers, wide, scale, &a);            \
    if (rc < 0) return NULL;                                                  \
    if (rc == 0) Py_RETURN_NONE;                                              \
    Py_BEGIN_ALLOW_THREADS;                                                   \
    rc = call;                                                                \
    Py_END_ALLOW_THREADS;                                                     \
    return PyLong_FromLong(rc)
#define N(i) ((int)a.n[i])

/* q k v cu_seqlens out | B N H G d_h window dtype | scale */
static PyObject *prefill_packed(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(5, 7, 0, 1, abi.prefill_packed(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], N(0), N(1), N(2), N(3), N(4),
                                     (float)a.scale, N(5), (gqa_dtype)N(6), a.stream));
}

/* q k_cache v_cache block_table seqlens tree_mask n_draft out workspace |
   B n H G d_h page P M dtype workspace_bytes | scale */
static PyObject *decode_tree(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(9, 10, 1, 1, abi.decode_tree(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], (float)a.scale, a.p[7],
                                   N(0), N(1), N(2), N(3), N(4), N(5), N(6), N(7), (gqa_dtype)N(8), a.p[8],
                                   (size_t)a.n[9], a.stream));
}

/* k_cache v_cache k_new v_new cu_seqlens seqlens seqlens_out block_table | B N G d_h page P M dtype */
static PyObject *cache_append(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(8, 8, 0, 0, abi.cache_append(a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], a.p[0], a.p[1], a.p[7], N(0), N(1), N(2),
                                   N(3), N(4), N(5), N(6), (gqa_dtype)N(7), a.stream));
}

/* k_cache v_cache block_table seqlens keep n_keep seqlens_out | B m G d_h page P M dtype */
static PyObject *cache_compact(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(7, 8, 0, 0, abi.cache_compact(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], a.p[6], N(0), N(1), N(2), N(3),
                                    N(4), N(5), N(6), (gqa_dtype)N(7), a.stream));
}

/* block_table refcount seqlens n_new k_pages v_pages workspace | B G d_h page P M dtype workspace_bytes */
static PyObject *pages_reserve(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(7, 8, 1, 0, abi.pages_reserve(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], a.p[5], N(0), N(1), N(2), N(3), N(4), N(5),
                                    (gqa_dtype)N(6), a.p[6], (size_t)a.n[7], a.stream));
}

/* block_table refcount seqlens src dst | n B page P M */
static PyObject *pages_fork(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(5, 5, 0, 0, abi.pages_fork(a.p[0], a.p[1], a.p[2], a.p[3], a.p[4], N(0), N(1), N(2), N(3), N(4), a.stream));
}

/* block_table refcount lengths | B page P M */
static PyObject *pages_release(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    CALL(3, 4, 0, 0, abi.pages_release(a.p[0], a.p[1], a.p[2], N(0), N(1), N(2), N(3), a.stream));
}

/* bind(addresses of the seven entry points in abi's order, torch's current device, current stream) */
static PyObject *bind(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
    (void)self;
    void **slot = (void **)&abi;
    const Py_ssize_t entries = sizeof abi / sizeof(void *);
    if (nargs != entries + 2) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected", entries + 2);
        return NULL;
    }
    for (Py_ssize_t i = 0; i < entries; ++i) {
        slot[i] = PyLong_AsVoidPtr(args[i]);
        if (!slot[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
            return NULL;
        }
    }
    Py_XSETREF(f_current_device, Py_NewRef(args[entries]));
    Py_XSETREF(f_current_stream, Py_NewRef(args[entries + 1]));
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind),          METHOD(prefill_packed), METHOD(decode_tree),
                                METHOD(cache_append),  METHOD(cache_compact),  METHOD(pages_reserve),
                                METHOD(pages_fork),    METHOD(pages_release),  {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_get_device || !s_is_contiguous || !s_data_ptr || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
