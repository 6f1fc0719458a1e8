/* _qmm_call -- the per-call hand-off of qmm() and the K/V cache calls from Python to the C ABI, in C.
 *
 * A ctypes call converts every argument through Python-level descriptors, which costs
 * several microseconds per call: as much as a whole small-M matmul on the GPU.  This module
 * takes the same plain integers (device pointers, sizes, format, plan address, stream
 * handle) as a vectorcall and forwards them to the library's qmm_ex, whose address the
 * Python side binds once from the loaded libqmm_b200.so (the K/V cache's functions likewise).  It
 * does no arithmetic and holds no state beyond those function pointers; all argument checks stay
 * in the library.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../include/qmm.h"

typedef int (*qmm_ex_fn)(const void* x, const uint32_t* packed, const uint16_t* scales,
                         const uint16_t* biases, void* y, int64_t M, int64_t N, int64_t K,
                         int bits, int group, int dtype, const void* plan, void* stream);

static qmm_ex_fn g_qmm_ex = NULL;

static PyObject* bind(PyObject* self, PyObject* arg) {
    (void)self;
    void* p = PyLong_AsVoidPtr(arg);
    if (p == NULL) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "qmm_ex address is null");
        return NULL;
    }
    g_qmm_ex = (qmm_ex_fn)p;
    Py_RETURN_NONE;
}

/* qmm_ex(x, packed, scales, biases, y, M, N, K, bits, group, dtype, plan, stream) -> status
 * Pointers, the plan address (0 = default plan) and the stream handle are Python ints. */
static PyObject* call(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    if (nargs != 13) {
        PyErr_SetString(PyExc_TypeError, "qmm_ex takes 13 arguments");
        return NULL;
    }
    if (g_qmm_ex == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "qmm_ex is not bound");
        return NULL;
    }
    void* ptr[5];
    for (int i = 0; i < 5; ++i) ptr[i] = PyLong_AsVoidPtr(args[i]);
    const long long M = PyLong_AsLongLong(args[5]);
    const long long N = PyLong_AsLongLong(args[6]);
    const long long K = PyLong_AsLongLong(args[7]);
    const long bits = PyLong_AsLong(args[8]);
    const long group = PyLong_AsLong(args[9]);
    const long dtype = PyLong_AsLong(args[10]);
    void* plan = PyLong_AsVoidPtr(args[11]);
    void* stream = PyLong_AsVoidPtr(args[12]);
    if (PyErr_Occurred()) return NULL;
    const int st = g_qmm_ex(ptr[0], (const uint32_t*)ptr[1], (const uint16_t*)ptr[2],
                            (const uint16_t*)ptr[3], ptr[4], (int64_t)M, (int64_t)N, (int64_t)K,
                            (int)bits, (int)group, (int)dtype, plan, stream);
    return PyLong_FromLong(st);
}

/* ---- the K/V cache: five functions of the ABI, bound together ---- */
static struct {
    qmm_status (*append)(const qmm_kv_cache*, const void*, int64_t, int64_t, const void*, int64_t, int64_t,
                         const qmm_kv_seqs*, const int32_t*, int64_t, qmm_dtype, void*);
    qmm_status (*gather)(const qmm_kv_cache*, const qmm_kv_seqs*, const int32_t*, int64_t, void*, int64_t, int64_t,
                         void*, int64_t, int64_t, qmm_dtype, void*);
    qmm_status (*copy_pages)(const qmm_kv_cache*, const int32_t*, const int32_t*, int64_t, void*);
    qmm_status (*compact)(const qmm_kv_cache*, const qmm_kv_seqs*, const int32_t*, const int32_t*, int64_t, void*);
    qmm_status (*attention)(const qmm_kv_cache*, const void*, int64_t, int64_t, void*, int64_t, int64_t, float*,
                            const qmm_kv_seqs*, const int32_t*, int64_t, int, float, int64_t, const int64_t*,
                            qmm_dtype, void*);
} g_kv;

/* The first n arguments as 64-bit integers (addresses too); 0 and an exception if one is none. */
static int ints(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want, Py_ssize_t n, int64_t* v) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
        return 0;
    }
    if (g_kv.append == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "the K/V cache functions are not bound");
        return 0;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        v[i] = (int64_t)PyLong_AsLongLong(args[i]);
        if (v[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}
#define PTR(type, x) ((type)(uintptr_t)(x))
/* table, its row stride, columns, sequences, offsets */
static qmm_kv_seqs seqs_of(const int64_t* v) {
    qmm_kv_seqs s = {PTR(const int32_t*, v[0]), PTR(const int32_t*, v[4]), v[3], v[1], v[2]};
    return s;
}

/* bind_kv(append, gather, copy_pages, compact, attention): the functions' addresses */
static PyObject* bind_kv(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void* p[5];
    if (nargs != 5) {
        PyErr_SetString(PyExc_TypeError, "bind_kv takes 5 addresses");
        return NULL;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (p[i] == NULL) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is null");
            return NULL;
        }
    }
    *(void**)&g_kv.append = p[0];
    *(void**)&g_kv.gather = p[1];
    *(void**)&g_kv.copy_pages = p[2];
    *(void**)&g_kv.compact = p[3];
    *(void**)&g_kv.attention = p[4];
    Py_RETURN_NONE;
}

/* cache, k, strides (token, head), v, strides, seqs (5), lens, tokens, dtype, stream */
static PyObject* kv_append(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    int64_t v[16];
    if (!ints(args, nargs, 16, 16, v)) return NULL;
    const qmm_kv_seqs s = seqs_of(v + 7);
    return PyLong_FromLong(g_kv.append(PTR(const qmm_kv_cache*, v[0]), PTR(void*, v[1]), v[2], v[3], PTR(void*, v[4]), v[5],
                                       v[6], &s, PTR(const int32_t*, v[12]), v[13], (qmm_dtype)v[14], PTR(void*, v[15])));
}

/* cache, seqs (5), starts, tokens, k, strides, v, strides, dtype, stream */
static PyObject* kv_gather(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    int64_t v[16];
    if (!ints(args, nargs, 16, 16, v)) return NULL;
    const qmm_kv_seqs s = seqs_of(v + 1);
    return PyLong_FromLong(g_kv.gather(PTR(const qmm_kv_cache*, v[0]), &s, PTR(const int32_t*, v[6]), v[7], PTR(void*, v[8]),
                                       v[9], v[10], PTR(void*, v[11]), v[12], v[13], (qmm_dtype)v[14], PTR(void*, v[15])));
}

/* cache, src, dst, pairs, stream */
static PyObject* kv_copy_pages(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    int64_t v[5];
    if (!ints(args, nargs, 5, 5, v)) return NULL;
    return PyLong_FromLong(g_kv.copy_pages(PTR(const qmm_kv_cache*, v[0]), PTR(const int32_t*, v[1]),
                                           PTR(const int32_t*, v[2]), v[3], PTR(void*, v[4])));
}

/* cache, seqs (5), starts, keep, kept, stream */
static PyObject* kv_compact(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    int64_t v[10];
    if (!ints(args, nargs, 10, 10, v)) return NULL;
    const qmm_kv_seqs s = seqs_of(v + 1);
    return PyLong_FromLong(g_kv.compact(PTR(const qmm_kv_cache*, v[0]), &s, PTR(const int32_t*, v[6]),
                                        PTR(const int32_t*, v[7]), v[8], PTR(void*, v[9])));
}

/* cache, q, strides, o, strides, lse, seqs (5), lens, tokens, heads, window, tree, dtype, stream, scale */
static PyObject* kv_attention(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    int64_t v[20];
    if (!ints(args, nargs, 21, 20, v)) return NULL;
    const double scale = PyFloat_AsDouble(args[20]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    const qmm_kv_seqs s = seqs_of(v + 8);
    return PyLong_FromLong(g_kv.attention(PTR(const qmm_kv_cache*, v[0]), PTR(void*, v[1]), v[2], v[3], PTR(void*, v[4]), v[5],
                                          v[6], PTR(float*, v[7]), &s, PTR(const int32_t*, v[13]), v[14], (int)v[15],
                                          (float)scale, v[16], PTR(const int64_t*, v[17]), (qmm_dtype)v[18],
                                          PTR(void*, v[19])));
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_O, "bind(address of qmm_ex)"},
    {"qmm_ex", (PyCFunction)(void (*)(void))call, METH_FASTCALL,
     "qmm_ex(x, packed, scales, biases, y, M, N, K, bits, group, dtype, plan, stream) -> status"},
    {"bind_kv", (PyCFunction)(void (*)(void))bind_kv, METH_FASTCALL, "addresses of the five K/V cache functions"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, "qmm_kv_append -> status"},
    {"kv_gather", (PyCFunction)(void (*)(void))kv_gather, METH_FASTCALL, "qmm_kv_gather -> status"},
    {"kv_copy_pages", (PyCFunction)(void (*)(void))kv_copy_pages, METH_FASTCALL, "qmm_kv_copy_pages -> status"},
    {"kv_compact", (PyCFunction)(void (*)(void))kv_compact, METH_FASTCALL, "qmm_kv_compact -> status"},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, "qmm_kv_attention -> status"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qmm_call(void) { return PyModule_Create(&module); }
