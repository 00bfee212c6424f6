/*
 * Argument marshalling of the cs_qcache_* calls for Python: tensors' shapes,
 * strides and addresses into the C ABI's arguments, and nothing else.  A
 * decode step's kernels take a few microseconds, and reading the same
 * attributes one by one in Python took longer than launching them.
 *
 * The module knows nothing of torch: a tensor is whatever has shape, stride(),
 * dtype, is_cuda, is_contiguous() and data_ptr().  init() is given the dtypes
 * and the addresses of libcs.so's functions.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "cs.h"

static PyObject *n_shape, *n_stride, *n_dtype, *n_is_cuda, *n_contig, *n_data_ptr;
static PyObject *dt_f32, *dt_f16, *dt_bf16, *dt_i32;

typedef cs_status (*append_fn)(const cs_qcache *, const cs_head_rows *, const cs_head_rows *, int, const int32_t *,
                               const int32_t *, const int32_t *, const int32_t *, void *, size_t, cs_stream_t);
typedef cs_status (*read_fn)(const cs_qcache *, const cs_head_rows *, const cs_head_rows *, int, const int32_t *,
                             const int32_t *, void *, size_t, cs_stream_t);
typedef cs_status (*attention_fn)(const cs_qcache *, const cs_head_rows *, int, int, const int32_t *, const int32_t *,
                                  const uint32_t *, float, float, float *, const cs_head_rows *, void *, size_t,
                                  cs_stream_t);
typedef cs_status (*evict_fn)(const cs_qcache *, const int32_t *, int, int, const int32_t *, int, int, int32_t *,
                              void *, size_t, cs_stream_t);
typedef cs_status (*trim_fn)(const cs_qcache *, const int32_t *, int, const int32_t *, int, int, const cs_qcache *,
                             void *, size_t, cs_stream_t);
static append_fn f_append;
static read_fn f_read;
static attention_fn f_attention;
static evict_fn f_evict;
static trim_fn f_trim;

#define MAX_DIMS 4

/* shape or strides, as a tuple of ints; -1 if it has another length than nd */
static int tuple_of(PyObject *t, int nd, int64_t *out) {
    if (!t) return -1;
    int ok = PyTuple_Check(t) && PyTuple_GET_SIZE(t) == nd;
    for (int i = 0; ok && i < nd; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (out[i] == -1 && PyErr_Occurred()) ok = 0;
    }
    Py_DECREF(t);
    return ok ? 0 : -1;
}

static int truth(PyObject *o) {
    if (!o) return -1;
    const int r = PyObject_IsTrue(o);
    Py_DECREF(o);
    return r;
}

static void *address(PyObject *t, const char *what) {
    const int cuda = truth(PyObject_GetAttr(t, n_is_cuda));
    if (cuda < 0) return NULL;
    if (!cuda) {
        PyErr_Format(PyExc_ValueError, "%s: expected a CUDA tensor", what);
        return NULL;
    }
    PyObject *p = PyObject_CallMethodNoArgs(t, n_data_ptr);
    if (!p) return NULL;
    void *a = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return a;
}

/* cs_head_rows of a [batch, tokens, heads, d] tensor; heads < 0: any number, stored in *heads_out */
static int rows_of(PyObject *t, const cs_qcache *c, int64_t heads, const char *what, cs_head_rows *r, int64_t *tokens,
                   int64_t *heads_out) {
    int64_t shape[MAX_DIMS], st[MAX_DIMS];
    if (tuple_of(PyObject_GetAttr(t, n_shape), 4, shape) || tuple_of(PyObject_CallMethodNoArgs(t, n_stride), 4, st) ||
        shape[0] != c->batch || (heads >= 0 && shape[2] != heads) || shape[3] != c->d_head || st[3] != 1 ||
        shape[1] > INT32_MAX || shape[2] > INT32_MAX) {
        if (!PyErr_Occurred())
            PyErr_Format(PyExc_ValueError, "%s: expected [%d, tokens, heads, %d] with contiguous rows, and the heads "
                         "that the call has", what, c->batch, c->d_head);
        return -1;
    }
    PyObject *dt = PyObject_GetAttr(t, n_dtype);
    if (!dt) return -1;
    Py_DECREF(dt); /* dtypes are never freed: init() holds them */
    if (dt == dt_f32) r->dtype = CS_F32;
    else if (dt == dt_f16) r->dtype = CS_F16;
    else if (dt == dt_bf16) r->dtype = CS_BF16;
    else {
        PyErr_Format(PyExc_ValueError, "%s: its dtype is not fp32, fp16 or bf16", what);
        return -1;
    }
    r->data = address(t, what);
    if (PyErr_Occurred()) return -1;
    r->ld_batch = st[0];
    r->ld_token = st[1];
    r->ld_head = st[2];
    *tokens = shape[1];
    if (heads_out) *heads_out = shape[2];
    return 0;
}

/* the address of a contiguous int32 tensor of nd dimensions (its sizes in want, -1 for any, read into want), NULL for None */
static int ints_of(PyObject *t, int nd, int64_t *want, const char *what, void **out) {
    *out = NULL;
    if (t == Py_None) return 0;
    int64_t shape[MAX_DIMS];
    PyObject *dt = PyObject_GetAttr(t, n_dtype);
    if (!dt) return -1;
    Py_DECREF(dt);
    int ok = dt == dt_i32 && tuple_of(PyObject_GetAttr(t, n_shape), nd, shape) == 0;
    for (int i = 0; ok && i < nd; ++i) {
        ok = want[i] < 0 ? shape[i] <= INT32_MAX : shape[i] == want[i];
        want[i] = shape[i];
    }
    if (ok) ok = truth(PyObject_CallMethodNoArgs(t, n_contig)) == 1;
    if (!ok) {
        if (!PyErr_Occurred())
            PyErr_Format(PyExc_ValueError, "%s: expected a contiguous int32 tensor of the call's sizes", what);
        return -1;
    }
    *out = address(t, what);
    return PyErr_Occurred() ? -1 : 0;
}

static int batch_ints(PyObject *t, const cs_qcache *c, const char *what, const int32_t **out) {
    int64_t want[1] = {c->batch};
    return ints_of(t, 1, want, what, (void **)out);
}

static int as_int(PyObject *o, int *out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v > INT32_MAX || v < INT32_MIN) {
        PyErr_SetString(PyExc_ValueError, "a number is out of range");
        return -1;
    }
    *out = (int)v;
    return 0;
}

typedef struct tail { void *ws; size_t bytes; cs_stream_t stream; } tail;
static int tail_of(PyObject *const *a, tail *t) {
    t->ws = PyLong_AsVoidPtr(a[0]);
    t->bytes = PyLong_AsSize_t(a[1]);
    t->stream = (cs_stream_t)PyLong_AsVoidPtr(a[2]);
    return PyErr_Occurred() ? -1 : 0;
}

#define COUNT(n)                                                                  \
    if (nargs != (n)) {                                                           \
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", (n), nargs); \
        return NULL;                                                              \
    }                                                                             \
    const cs_qcache *c = (const cs_qcache *)PyLong_AsVoidPtr(a[0]);               \
    if (!c) return NULL
#define CALL(expr)                \
    cs_status st;                 \
    Py_BEGIN_ALLOW_THREADS        \
    st = (expr);                  \
    Py_END_ALLOW_THREADS          \
    return PyLong_FromLong((long)st)

/* cache, k, v, start, slots[, n_new, pos], ws, bytes, stream */
static PyObject *rows_call(PyObject *const *a, Py_ssize_t nargs, int append) {
    COUNT(append ? 10 : 8);
    cs_head_rows k, v;
    int64_t n, nv;
    const int32_t *start, *slots, *n_new = NULL, *pos = NULL;
    tail t;
    if (rows_of(a[1], c, c->n_heads, "k", &k, &n, NULL) || rows_of(a[2], c, c->n_heads, "v", &v, &nv, NULL)) return NULL;
    if (n != nv) {
        PyErr_SetString(PyExc_ValueError, "k and v differ in their number of tokens");
        return NULL;
    }
    int64_t want[3] = {c->batch, c->n_heads, n};
    if (batch_ints(a[3], c, "start", &start) || ints_of(a[4], 3, want, "slots", (void **)&slots) ||
        (append && (batch_ints(a[5], c, "n_new", &n_new) || batch_ints(a[6], c, "pos", &pos))) ||
        tail_of(a + (append ? 7 : 5), &t))
        return NULL;
    if (append) {
        CALL(f_append(c, &k, &v, (int)n, start, slots, n_new, pos, t.ws, t.bytes, t.stream));
    } else {
        CALL(f_read(c, &k, &v, (int)n, start, slots, t.ws, t.bytes, t.stream));
    }
}
static PyObject *py_append(PyObject *self, PyObject *const *a, Py_ssize_t nargs) { return rows_call(a, nargs, 1); }
static PyObject *py_read(PyObject *self, PyObject *const *a, Py_ssize_t nargs) { return rows_call(a, nargs, 0); }

/* cache, q, length, out, q_pos, mask (an address or 0), scale, weight (likewise), decay, ws, bytes, stream */
static PyObject *py_attention(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    COUNT(12);
    cs_head_rows q, out;
    int64_t n, no, heads;
    const int32_t *length, *q_pos;
    tail t;
    if (rows_of(a[1], c, -1, "q", &q, &n, &heads) || rows_of(a[3], c, heads, "out", &out, &no, NULL)) return NULL;
    if (n != no) {
        PyErr_SetString(PyExc_ValueError, "q and out differ in their number of tokens");
        return NULL;
    }
    const uint32_t *mask = (const uint32_t *)PyLong_AsVoidPtr(a[5]);
    float *weight = (float *)PyLong_AsVoidPtr(a[7]);
    const double scale = PyFloat_AsDouble(a[6]), decay = PyFloat_AsDouble(a[8]);
    if (PyErr_Occurred() || batch_ints(a[2], c, "length", &length) || batch_ints(a[4], c, "q_pos", &q_pos) || tail_of(a + 9, &t))
        return NULL;
    CALL(f_attention(c, &q, (int)heads, (int)n, length, q_pos, mask, (float)scale, (float)decay, weight, &out, t.ws, t.bytes,
                     t.stream));
}

/* cache, length, limit, slots, next_pos, sinks, recent, ws, bytes, stream */
static PyObject *py_evict(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    COUNT(10);
    const int32_t *length, *next_pos;
    int32_t *slots;
    int limit, sinks, recent;
    int64_t want[3] = {c->batch, c->n_heads, -1};
    tail t;
    if (batch_ints(a[1], c, "length", &length) || as_int(a[2], &limit) || ints_of(a[3], 3, want, "slots", (void **)&slots) ||
        batch_ints(a[4], c, "next_pos", &next_pos) || as_int(a[5], &sinks) || as_int(a[6], &recent) || tail_of(a + 7, &t))
        return NULL;
    CALL(f_evict(c, length, limit, slots ? (int)want[2] : 0, next_pos, sinks, recent, slots, t.ws, t.bytes, t.stream));
}

/* cache, length, keep, dst cache, next_pos, sinks, recent, ws, bytes, stream */
static PyObject *py_trim(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    COUNT(10);
    const cs_qcache *dst = (const cs_qcache *)PyLong_AsVoidPtr(a[3]);
    const int32_t *length, *next_pos;
    int keep, sinks, recent;
    tail t;
    if (!dst || batch_ints(a[1], c, "length", &length) || as_int(a[2], &keep) || batch_ints(a[4], c, "next_pos", &next_pos) ||
        as_int(a[5], &sinks) || as_int(a[6], &recent) || tail_of(a + 7, &t))
        return NULL;
    CALL(f_trim(c, length, keep, next_pos, sinks, recent, dst, t.ws, t.bytes, t.stream));
}

/* float32, float16, bfloat16, int32, then the five functions' addresses */
static PyObject *py_init(PyObject *self, PyObject *const *a, Py_ssize_t nargs) {
    if (nargs != 9) {
        PyErr_SetString(PyExc_TypeError, "expected 9 arguments");
        return NULL;
    }
    PyObject **dts[4] = {&dt_f32, &dt_f16, &dt_bf16, &dt_i32};
    for (int i = 0; i < 4; ++i) {
        Py_INCREF(a[i]);
        *dts[i] = a[i];
    }
    f_append = (append_fn)PyLong_AsVoidPtr(a[4]);
    f_read = (read_fn)PyLong_AsVoidPtr(a[5]);
    f_attention = (attention_fn)PyLong_AsVoidPtr(a[6]);
    f_evict = (evict_fn)PyLong_AsVoidPtr(a[7]);
    f_trim = (trim_fn)PyLong_AsVoidPtr(a[8]);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

#define FN(f) (PyCFunction)(void (*)(void))f
static PyMethodDef methods[] = {
    {"init", FN(py_init), METH_FASTCALL, NULL},           {"append", FN(py_append), METH_FASTCALL, NULL},
    {"read", FN(py_read), METH_FASTCALL, NULL},           {"attention", FN(py_attention), METH_FASTCALL, NULL},
    {"evict", FN(py_evict), METH_FASTCALL, NULL},         {"trim", FN(py_trim), METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__qcall(void) {
    n_shape = PyUnicode_InternFromString("shape");
    n_stride = PyUnicode_InternFromString("stride");
    n_dtype = PyUnicode_InternFromString("dtype");
    n_is_cuda = PyUnicode_InternFromString("is_cuda");
    n_contig = PyUnicode_InternFromString("is_contiguous");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    return PyModule_Create(&module);
}
