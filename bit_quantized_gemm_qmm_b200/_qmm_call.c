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

/* torch's copy of the exchange format: plain C.  A torch without the exchange functions gets the module without the
 * K/V cache's calls. */
#if defined(__has_include)
#if __has_include(<ATen/dlpack.h>)
#include <ATen/dlpack.h>
#endif
#endif
#if defined(DLPACK_MAJOR_VERSION) && DLPACK_MAJOR_VERSION == 1 && DLPACK_MINOR_VERSION >= 3
#define WITH_KV 1
#else
#define WITH_KV 0
#endif

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

#if WITH_KV
/* ---- the K/V cache: five functions of the ABI, bound together.  They take tensors, read through
 * torch's DLPack exchange functions (a view of a tensor's pointer, sizes and strides in about the
 * time of one attribute look-up), and check what the ABI cannot see. ---- */
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
static const DLPackExchangeAPI* g_dl = NULL;
static PyTypeObject* g_tensor = NULL;

/* A call's cache: the address of its descriptor and its device. */
typedef struct {
    const qmm_kv_cache* cache;
    int device;
    void* stream;
} ctx;

static int is_type(const DLTensor* t, int code, int bits) {
    return t->dtype.code == code && t->dtype.bits == bits && t->dtype.lanes == 1;
}

/* View of a tensor of `dims` dimensions on the call's device; 0 and an exception if it is none. */
static int view(const ctx* x, PyObject* obj, const char* what, int dims, DLTensor* t) {
    if (!PyObject_TypeCheck(obj, g_tensor)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
        return 0;
    }
    if (g_dl->dltensor_from_py_object_no_sync(obj, t) != 0) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s cannot be read", what);
        return 0;
    }
    if (t->device.device_type != kDLCUDA || t->device.device_id != x->device || t->ndim != dims) {
        PyErr_Format(PyExc_ValueError, "%s must be a tensor of %d dimension%s on the cache's CUDA device", what, dims,
                     dims == 1 ? "" : "s");
        return 0;
    }
    return 1;
}
static void* data(const DLTensor* t) { return (char*)t->data + t->byte_offset; }

/* A contiguous vector of n values (n < 0: any number) of a type. */
static int vec(const ctx* x, PyObject* obj, const char* what, int64_t n, int code, int bits, DLTensor* t) {
    if (!view(x, obj, what, 1, t)) return 0;
    if (!is_type(t, code, bits) || (n >= 0 && t->shape[0] != n) || (t->shape[0] > 1 && t->strides && t->strides[0] != 1)) {
        PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s%d vector of %s%lld values", what,
                     code == kDLInt ? "int" : "float", bits, n < 0 ? "any number, not " : "", (long long)(n < 0 ? t->shape[0] : n));
        return 0;
    }
    return 1;
}

/* [tokens, heads, head_dim] rows with a contiguous last dimension. */
typedef struct {
    void* p;
    int64_t ts, hs, tokens, heads;
    int dtype;
} rows;
static int rows_of(const ctx* x, PyObject* obj, const char* what, rows* r) {
    DLTensor t;
    if (!view(x, obj, what, 3, &t)) return 0;
    r->dtype = is_type(&t, kDLFloat, 16) ? QMM_F16 : is_type(&t, kDLBfloat, 16) ? QMM_BF16 : -1;
    if (r->dtype < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be fp16 or bf16", what);
        return 0;
    }
    r->tokens = t.shape[0], r->heads = t.shape[1];
    const int64_t dim = t.shape[2];
    const int64_t s0 = t.strides ? t.strides[0] : t.shape[1] * dim, s1 = t.strides ? t.strides[1] : dim;
    if (dim != x->cache->head_dim || (t.strides && t.strides[2] != 1)) {
        PyErr_Format(PyExc_ValueError, "%s must have contiguous rows of head_dim=%d values", what, (int)x->cache->head_dim);
        return 0;
    }
    r->p = data(&t), r->ts = r->tokens > 1 ? s0 : 0, r->hs = r->heads > 1 ? s1 : 0;
    return 1;
}

/* The cache's descriptor address and device, and the device's current stream. */
static int begin(PyObject* const* args, Py_ssize_t nargs, Py_ssize_t want, ctx* x) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, nargs);
        return 0;
    }
    if (g_dl == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "the K/V cache functions are not bound");
        return 0;
    }
    x->cache = (const qmm_kv_cache*)PyLong_AsVoidPtr(args[0]);
    x->device = (int)PyLong_AsLong(args[1]);
    x->stream = NULL;
    if (PyErr_Occurred()) return 0;
    if (x->cache == NULL) {
        PyErr_SetString(PyExc_ValueError, "the cache's address is null");
        return 0;
    }
    return 1;
}
static int stream_of(ctx* x) {
    if (g_dl->current_work_stream(kDLCUDA, x->device, &x->stream) == 0) return 1;
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "no current stream");
    return 0;
}

/* Page table, offsets and one value a sequence (`at`). */
static int seqs_of(const ctx* x, PyObject* table, PyObject* at, const char* at_name, PyObject* cu, const char* cu_name,
                   qmm_kv_seqs* s, const int32_t** at_out) {
    DLTensor t, c, v;
    if (!view(x, table, "page_table", 2, &t)) return 0;
    if (!is_type(&t, kDLInt, 32) || (t.shape[1] > 1 && t.strides && t.strides[1] != 1)) {
        PyErr_SetString(PyExc_ValueError, "page_table must be int32 [seqs, pages] with contiguous rows");
        return 0;
    }
    if (!vec(x, at, at_name, t.shape[0], kDLInt, 32, &v) || !vec(x, cu, cu_name, t.shape[0] + 1, kDLInt, 32, &c)) return 0;
    s->page_table = (const int32_t*)data(&t);
    s->cu_tokens = (const int32_t*)data(&c);
    s->seqs = t.shape[0];
    s->max_pages = t.shape[1];
    s->table_stride = t.shape[0] > 1 && t.strides ? t.strides[0] : t.shape[1];
    *at_out = (const int32_t*)data(&v);
    return 1;
}

static int same_rows(const rows* a, const rows* b, const char* what) {
    if (a->tokens == b->tokens && a->heads == b->heads && a->dtype == b->dtype) return 1;
    PyErr_SetString(PyExc_ValueError, what);
    return 0;
}

/* bind_kv(append, gather, copy_pages, compact, attention, tensor type): the functions' addresses */
static PyObject* bind_kv(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    void* p[5];
    if (nargs != 6) {
        PyErr_SetString(PyExc_TypeError, "bind_kv takes 5 addresses and the tensor type");
        return NULL;
    }
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (p[i] == NULL) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "a function's address is null");
            return NULL;
        }
    }
    if (!PyType_Check(args[5])) {
        PyErr_SetString(PyExc_TypeError, "the tensor type expected");
        return NULL;
    }
    PyObject* capsule = PyObject_GetAttrString(args[5], "__dlpack_c_exchange_api__");
    if (capsule == NULL) return NULL;
    const DLPackExchangeAPI* api = (const DLPackExchangeAPI*)PyCapsule_GetPointer(capsule, "dlpack_exchange_api");
    Py_DECREF(capsule); /* the functions live as long as the process */
    if (api == NULL) return NULL;
    if (api->header.version.major != DLPACK_MAJOR_VERSION || api->dltensor_from_py_object_no_sync == NULL ||
        api->current_work_stream == NULL) {
        PyErr_SetString(PyExc_RuntimeError, "this torch's DLPack exchange functions are of another version");
        return NULL;
    }
    *(void**)&g_kv.append = p[0];
    *(void**)&g_kv.gather = p[1];
    *(void**)&g_kv.copy_pages = p[2];
    *(void**)&g_kv.compact = p[3];
    *(void**)&g_kv.attention = p[4];
    Py_INCREF(args[5]);
    Py_XDECREF((PyObject*)g_tensor);
    g_tensor = (PyTypeObject*)args[5];
    g_dl = api;
    Py_RETURN_NONE;
}

/* cache, device, k, v, page_table, lens, cu_tokens */
static PyObject* kv_append(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    ctx x;
    rows k, v;
    qmm_kv_seqs s;
    const int32_t* lens;
    if (!begin(args, nargs, 7, &x) || !rows_of(&x, args[2], "k", &k) || !rows_of(&x, args[3], "v", &v)) return NULL;
    if (!same_rows(&k, &v, "k and v must have one shape and dtype")) return NULL;
    if (k.heads != x.cache->kv_heads) {
        PyErr_Format(PyExc_ValueError, "k and v must have kv_heads=%d heads", (int)x.cache->kv_heads);
        return NULL;
    }
    if (!seqs_of(&x, args[4], args[5], "lens", args[6], "cu_tokens", &s, &lens) || !stream_of(&x)) return NULL;
    return PyLong_FromLong(g_kv.append(x.cache, k.p, k.ts, k.hs, v.p, v.ts, v.hs, &s, lens, k.tokens, (qmm_dtype)k.dtype, x.stream));
}

/* cache, device, k, v, page_table, starts, cu_tokens */
static PyObject* kv_gather(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    ctx x;
    rows k, v;
    qmm_kv_seqs s;
    const int32_t* starts;
    if (!begin(args, nargs, 7, &x) || !rows_of(&x, args[2], "out[0]", &k) || !rows_of(&x, args[3], "out[1]", &v)) return NULL;
    if (!same_rows(&k, &v, "the outputs must have one shape and dtype")) return NULL;
    if (k.heads != x.cache->kv_heads) {
        PyErr_Format(PyExc_ValueError, "the outputs must have kv_heads=%d heads", (int)x.cache->kv_heads);
        return NULL;
    }
    if (!seqs_of(&x, args[4], args[5], "starts", args[6], "cu_tokens", &s, &starts) || !stream_of(&x)) return NULL;
    return PyLong_FromLong(g_kv.gather(x.cache, &s, starts, k.tokens, k.p, k.ts, k.hs, v.p, v.ts, v.hs, (qmm_dtype)k.dtype, x.stream));
}

/* cache, device, src, dst */
static PyObject* kv_copy_pages(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    ctx x;
    DLTensor a, b;
    if (!begin(args, nargs, 4, &x) || !vec(&x, args[2], "src", -1, kDLInt, 32, &a) ||
        !vec(&x, args[3], "dst", a.shape[0], kDLInt, 32, &b) || !stream_of(&x))
        return NULL;
    return PyLong_FromLong(g_kv.copy_pages(x.cache, (const int32_t*)data(&a), (const int32_t*)data(&b), a.shape[0], x.stream));
}

/* cache, device, page_table, starts, keep, cu_keep */
static PyObject* kv_compact(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    ctx x;
    DLTensor k;
    qmm_kv_seqs s;
    const int32_t* starts;
    if (!begin(args, nargs, 6, &x) || !seqs_of(&x, args[2], args[3], "starts", args[5], "cu_keep", &s, &starts) ||
        !vec(&x, args[4], "keep", -1, kDLInt, 32, &k) || !stream_of(&x))
        return NULL;
    return PyLong_FromLong(g_kv.compact(x.cache, &s, starts, (const int32_t*)data(&k), k.shape[0], x.stream));
}

/* cache, device, q, page_table, lens, cu_tokens, o, lse, tree or None, window, scale */
static PyObject* kv_attention(PyObject* self, PyObject* const* args, Py_ssize_t nargs) {
    (void)self;
    ctx x;
    rows q, o;
    DLTensor l, tree;
    qmm_kv_seqs s;
    const int32_t* lens;
    if (!begin(args, nargs, 11, &x) || !rows_of(&x, args[2], "q", &q) || !rows_of(&x, args[6], "out", &o)) return NULL;
    if (!same_rows(&q, &o, "out must have q's shape and dtype")) return NULL;
    if (!seqs_of(&x, args[3], args[4], "lens", args[5], "cu_tokens", &s, &lens) || !view(&x, args[7], "lse", 2, &l)) return NULL;
    if (!is_type(&l, kDLFloat, 32) || l.shape[0] != q.tokens || l.shape[1] != q.heads ||
        (l.strides && ((l.shape[1] > 1 && l.strides[1] != 1) || (l.shape[0] > 1 && l.strides[0] != l.shape[1])))) {
        PyErr_SetString(PyExc_ValueError, "lse must be contiguous fp32 [tokens, heads]");
        return NULL;
    }
    if (args[8] != Py_None && !vec(&x, args[8], "tree", q.tokens, kDLInt, 64, &tree)) return NULL;
    const int64_t window = (int64_t)PyLong_AsLongLong(args[9]);
    const double scale = PyFloat_AsDouble(args[10]);
    if (PyErr_Occurred() || !stream_of(&x)) return NULL;
    return PyLong_FromLong(g_kv.attention(x.cache, q.p, q.ts, q.hs, o.p, o.ts, o.hs, (float*)data(&l), &s, lens, q.tokens,
                                          (int)q.heads, (float)scale, window,
                                          args[8] == Py_None ? NULL : (const int64_t*)data(&tree), (qmm_dtype)q.dtype, x.stream));
}

#endif /* WITH_KV */

static PyMethodDef methods[] = {
    {"bind", bind, METH_O, "bind(address of qmm_ex)"},
    {"qmm_ex", (PyCFunction)(void (*)(void))call, METH_FASTCALL,
     "qmm_ex(x, packed, scales, biases, y, M, N, K, bits, group, dtype, plan, stream) -> status"},
#if WITH_KV
    {"bind_kv", (PyCFunction)(void (*)(void))bind_kv, METH_FASTCALL, "addresses of the five K/V cache functions, and the tensor type"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, "qmm_kv_append -> status"},
    {"kv_gather", (PyCFunction)(void (*)(void))kv_gather, METH_FASTCALL, "qmm_kv_gather -> status"},
    {"kv_copy_pages", (PyCFunction)(void (*)(void))kv_copy_pages, METH_FASTCALL, "qmm_kv_copy_pages -> status"},
    {"kv_compact", (PyCFunction)(void (*)(void))kv_compact, METH_FASTCALL, "qmm_kv_compact -> status"},
    {"kv_attention", (PyCFunction)(void (*)(void))kv_attention, METH_FASTCALL, "qmm_kv_attention -> status"},
#endif
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_call", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qmm_call(void) { return PyModule_Create(&module); }
