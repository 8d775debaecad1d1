/* pyfast.c -- a CPython extension that calls the library's 14-argument
 * matmul entry points (qmm_gemv, qmm_gemm, qmm_gemv_tile16: same signature) and
 * the paged cache calls (qmm_kv_append, qmm_paged_attn)
 * through a function address, so that the Python binding's hot calls skip
 * ctypes' per-argument conversion.  It does no arithmetic and no checks
 * beyond argument parsing; the binding falls back to ctypes when this module
 * is not built.  Built by build.py next to libqmm.so. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>

/* The host struct of the paged cache calls, as in include/qmm.h (which needs the
 * CUDA headers; this file does not). */
typedef struct {
    void *k, *v;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *block_table, *cu_q, *kv_len;
    int num_pages, page_size, blocks;
    int batch, tokens;
    int kv_heads, head_dim;
    int dtype;
} qmm_paged_kv;

typedef int (*qmm_call14)(const void *, int, const uint8_t *, int, int, const void *, const uint8_t *,
                          int, void *, int, int, int, int, void *);

static int as_u64(PyObject *o, unsigned long long *v)
{
    if (o == Py_None) {
        *v = 0;
        return 0;
    }
    *v = PyLong_AsUnsignedLongLong(o);
    return (*v == (unsigned long long)-1 && PyErr_Occurred()) ? -1 : 0;
}

static int as_int(PyObject *o, int *v)
{
    long t = PyLong_AsLong(o);
    if (t == -1 && PyErr_Occurred())
        return -1;
    if (t < INT32_MIN || t > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "argument does not fit in a C int");
        return -1;
    }
    *v = (int)t;
    return 0;
}

/* call14(fn, x, x_dtype, packed, bits, group, scales, zeros, zero_const, y,
 *        y_dtype, M, N, K, stream) -> status.  Pointers are ints or None. */
static PyObject *call14(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    if (nargs != 15) {
        PyErr_SetString(PyExc_TypeError, "call14 takes 15 arguments");
        return NULL;
    }
    unsigned long long fn, x, packed, scales, zeros, y, stream;
    int xdt, bits, group, zc, ydt, M, N, K;
    if (as_u64(args[0], &fn) || as_u64(args[1], &x) || as_int(args[2], &xdt) || as_u64(args[3], &packed) ||
        as_int(args[4], &bits) || as_int(args[5], &group) || as_u64(args[6], &scales) ||
        as_u64(args[7], &zeros) || as_int(args[8], &zc) || as_u64(args[9], &y) || as_int(args[10], &ydt) ||
        as_int(args[11], &M) || as_int(args[12], &N) || as_int(args[13], &K) || as_u64(args[14], &stream))
        return NULL;
    if (!fn) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return NULL;
    }
    const int st = ((qmm_call14)(uintptr_t)fn)((const void *)(uintptr_t)x, xdt, (const uint8_t *)(uintptr_t)packed,
                                               bits, group, (const void *)(uintptr_t)scales,
                                               (const uint8_t *)(uintptr_t)zeros, zc, (void *)(uintptr_t)y, ydt, M,
                                               N, K, (void *)(uintptr_t)stream);
    return PyLong_FromLong(st);
}

static int as_i64(PyObject *o, int64_t *v)
{
    *v = PyLong_AsLongLong(o);
    return (*v == -1 && PyErr_Occurred()) ? -1 : 0;
}

static int as_ptr(PyObject *o, void **p)
{
    unsigned long long v;
    if (as_u64(o, &v))
        return -1;
    *p = (void *)(uintptr_t)v;
    return 0;
}

/* The 16 fields of a qmm_paged_kv, in order. */
#define PAGED_FIELDS 16
static int as_paged(PyObject *const *a, qmm_paged_kv *kv)
{
    void *table, *cu, *len;
    if (as_ptr(a[0], &kv->k) || as_ptr(a[1], &kv->v) || as_i64(a[2], &kv->page_stride) ||
        as_i64(a[3], &kv->slot_stride) || as_i64(a[4], &kv->head_stride) || as_ptr(a[5], &table) ||
        as_ptr(a[6], &cu) || as_ptr(a[7], &len) || as_int(a[8], &kv->num_pages) || as_int(a[9], &kv->page_size) ||
        as_int(a[10], &kv->blocks) || as_int(a[11], &kv->batch) || as_int(a[12], &kv->tokens) ||
        as_int(a[13], &kv->kv_heads) || as_int(a[14], &kv->head_dim) || as_int(a[15], &kv->dtype))
        return -1;
    kv->block_table = (const int32_t *)table;
    kv->cu_q = (const int32_t *)cu;
    kv->kv_len = (const int32_t *)len;
    return 0;
}

typedef int (*append_fn)(const qmm_paged_kv *, const void *, int64_t, const void *, int64_t, const void *, int64_t,
                         void *, int, const void *, int, int, int, void *);

/* kv_append(fn, <16 fields>, k, k_stride, v, v_stride, q, q_stride, q_out,
 *           q_heads, cos_sin, rot, rope_len, interleaved, stream) -> status */
static PyObject *kv_append(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    if (nargs != 1 + PAGED_FIELDS + 13) {
        PyErr_SetString(PyExc_TypeError, "kv_append takes 30 arguments");
        return NULL;
    }
    qmm_paged_kv kv;
    void *fn, *k, *v, *q, *q_out, *cs, *stream;
    int64_t ks, vs, qs;
    int heads, rot, len, inter;
    PyObject *const *a = args + 1 + PAGED_FIELDS;
    if (as_ptr(args[0], &fn) || as_paged(args + 1, &kv) || as_ptr(a[0], &k) || as_i64(a[1], &ks) || as_ptr(a[2], &v) ||
        as_i64(a[3], &vs) || as_ptr(a[4], &q) || as_i64(a[5], &qs) || as_ptr(a[6], &q_out) || as_int(a[7], &heads) ||
        as_ptr(a[8], &cs) || as_int(a[9], &rot) || as_int(a[10], &len) || as_int(a[11], &inter) ||
        as_ptr(a[12], &stream))
        return NULL;
    if (!fn) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return NULL;
    }
    return PyLong_FromLong(
        ((append_fn)(uintptr_t)fn)(&kv, k, ks, v, vs, q, qs, q_out, heads, cs, rot, len, inter, stream));
}

typedef int (*attn_fn)(const qmm_paged_kv *, const void *, int64_t, int, float, int, int, void *, void *, int, int,
                       void *, size_t, void *);

/* paged_attn(fn, <16 fields>, q, q_stride, q_heads, scale, causal, window, out,
 *            lse, max_q, max_kv, workspace, workspace_bytes, stream) -> status */
static PyObject *paged_attn(PyObject *self, PyObject *const *args, Py_ssize_t nargs)
{
    (void)self;
    if (nargs != 1 + PAGED_FIELDS + 13) {
        PyErr_SetString(PyExc_TypeError, "paged_attn takes 30 arguments");
        return NULL;
    }
    qmm_paged_kv kv;
    void *fn, *q, *out, *lse, *ws, *stream;
    int64_t qs;
    int heads, causal, window, max_q, max_kv;
    unsigned long long bytes;
    PyObject *const *a = args + 1 + PAGED_FIELDS;
    if (as_ptr(args[0], &fn) || as_paged(args + 1, &kv) || as_ptr(a[0], &q) || as_i64(a[1], &qs) ||
        as_int(a[2], &heads))
        return NULL;
    const double scale = PyFloat_AsDouble(a[3]);
    if ((scale == -1.0 && PyErr_Occurred()) || as_int(a[4], &causal) || as_int(a[5], &window) || as_ptr(a[6], &out) ||
        as_ptr(a[7], &lse) || as_int(a[8], &max_q) || as_int(a[9], &max_kv) || as_ptr(a[10], &ws) ||
        as_u64(a[11], &bytes) || as_ptr(a[12], &stream))
        return NULL;
    if (!fn) {
        PyErr_SetString(PyExc_ValueError, "null function address");
        return NULL;
    }
    return PyLong_FromLong(((attn_fn)(uintptr_t)fn)(&kv, q, qs, heads, (float)scale, causal, window, out, lse, max_q,
                                                     max_kv, ws, (size_t)bytes, stream));
}

static PyMethodDef methods[] = {
    {"call14", (PyCFunction)(void (*)(void))call14, METH_FASTCALL,
     "call14(fn, x, x_dtype, packed, bits, group, scales, zeros, zero_const, y, y_dtype, M, N, K, stream)"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL,
     "kv_append(fn, <qmm_paged_kv fields>, k, k_stride, v, v_stride, q, q_stride, q_out, q_heads, cos_sin, rot, "
     "rope_len, interleaved, stream)"},
    {"paged_attn", (PyCFunction)(void (*)(void))paged_attn, METH_FASTCALL,
     "paged_attn(fn, <qmm_paged_kv fields>, q, q_stride, q_heads, scale, causal, window, out, lse, max_q, max_kv, "
     "workspace, workspace_bytes, stream)"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmmfast", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qmmfast(void) { return PyModule_Create(&module); }
