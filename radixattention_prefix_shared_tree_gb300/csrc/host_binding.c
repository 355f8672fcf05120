/* Argument marshalling of kv_store_rope for Python, in C.
 *
 * An append is one launch of about two microseconds of GPU time for a single
 * token, and checking and passing its eight tensors from Python took five
 * microseconds of host time on top of the launch; here it takes about one.
 * The module knows tensors by their Python attributes only (data_ptr, shape,
 * stride, dtype, get_device), so it is built without torch's headers.  Nothing
 * is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "radixattn.h"

typedef rc_status (*store_rope_fn)(const rc_pool_desc*, const rc_rope_desc*, const int32_t*, const int32_t*, const void*,
                                   int64_t, const void*, int64_t, int32_t, const void*, int64_t, int32_t, void*, int64_t,
                                   int32_t*, const int32_t*, rc_stream_t);

static store_rope_fn fn_store_rope;
static PyObject *o_bf16, *o_i32, *o_get_device, *o_get_stream;                      /* set by bind() */
static PyObject *s_data_ptr, *s_shape, *s_stride, *s_dtype, *s_get_device, *s_is_contiguous, *s_cuda_stream;

/* The whole number that a call or attribute gave (steals `v`); -1 with an error set otherwise. */
static long long as_int(PyObject* v) {
    if (!v) return -1;
    const long long x = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return x;
}

/* Up to four sizes of a tuple (steals `v`); the tuple's length, -1 on error. */
static Py_ssize_t as_sizes(PyObject* v, long long out[4]) {
    if (!v) return -1;
    if (!PyTuple_Check(v)) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor");
        Py_DECREF(v);
        return -1;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(v);
    for (Py_ssize_t i = 0; i < n && i < 4; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v, i));
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : n;
}

static int has_dtype(PyObject* t, PyObject* want) {
    PyObject* d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    const int same = d == want;
    Py_DECREF(d);
    return same;
}

/* The tensor's address, on the current device `dev`. */
static int address(PyObject* t, const char* name, long long dev, void** ptr) {
    const long long d = as_int(PyObject_CallMethodNoArgs(t, s_get_device));
    if (PyErr_Occurred()) return -1;
    if (d != dev) {
        PyErr_Format(PyExc_ValueError, "kv_store_rope: %s is on device %lld (-1: the host), the current device is %lld",
                     name, d, dev);
        return -1;
    }
    PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return -1;
    *ptr = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/* bf16 rows [n, heads, dim] with dense rows per token (heads < 0: any); the
 * elements between tokens, which may be more (a slice of a projection's
 * output), go to *stride, the heads to *heads_out. */
static int rows(PyObject* t, const char* name, long long n, long long heads, long long dim, int write, int64_t* stride,
                long long* heads_out) {
    long long sh[4] = {0}, st[4] = {0};
    const Py_ssize_t nd = as_sizes(PyObject_GetAttr(t, s_shape), sh);
    if (nd < 0) return -1;
    if (nd != 3 || sh[0] != n || sh[2] != dim || (heads >= 0 && sh[1] != heads) || sh[1] <= 0) {
        if (heads >= 0)
            PyErr_Format(PyExc_ValueError, "%s: expected [%lld, %lld, %lld]", name, n, heads, dim);
        else
            PyErr_Format(PyExc_ValueError, "%s: expected [%lld, heads, %lld]", name, n, dim);
        return -1;
    }
    const int ok = has_dtype(t, o_bf16);
    if (ok <= 0) {
        if (ok == 0) PyErr_Format(PyExc_ValueError, "%s: expected bf16", name);
        return -1;
    }
    if (as_sizes(PyObject_CallMethodNoArgs(t, s_stride), st) != 3) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: expected three strides", name);
        return -1;
    }
    if (st[2] != 1 || (sh[1] > 1 && st[1] != dim)) {
        PyErr_Format(PyExc_ValueError, "%s: each token's rows must be dense, got strides (%lld, %lld, %lld)", name, st[0],
                     st[1], st[2]);
        return -1;
    }
    if (n <= 1) st[0] = sh[1] * dim;
    if (write && st[0] < sh[1] * dim) {
        PyErr_Format(PyExc_ValueError, "%s: overlapping rows, %lld elements apart", name, st[0]);
        return -1;
    }
    *stride = st[0];
    if (heads_out) *heads_out = sh[1];
    return 0;
}

/* A contiguous int32 tensor of n entries (n < 0: any); its entries, -1 on error. */
static long long ids(PyObject* t, const char* name, long long n) {
    const int ok = has_dtype(t, o_i32);
    if (ok < 0) return -1;
    long long sh[4] = {1, 1, 1, 1};
    const Py_ssize_t nd = as_sizes(PyObject_GetAttr(t, s_shape), sh);
    if (nd < 0) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    const int dense = c == Py_True;
    Py_DECREF(c);
    if (!ok || !dense || nd != 1 || (n >= 0 && sh[0] != n)) {
        if (n >= 0)
            PyErr_Format(PyExc_ValueError, "%s: expected a contiguous int32 tensor of %lld entries", name, n);
        else
            PyErr_Format(PyExc_ValueError, "%s: expected a contiguous one-dimensional int32 tensor", name);
        return -1;
    }
    return sh[0];
}

/* kv_store_rope(pool, rope, slots, positions, k_new, v_new, q, q_out, table, table_pos, stream, pool's device,
 * rope's device) -> status.  pool, rope: addresses of the descriptors; stream: None for the current one; devices:
 * None where they are not known. */
static PyObject* store_rope(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 13 || !fn_store_rope) {
        PyErr_SetString(PyExc_TypeError, "kv_store_rope: bind() first, then 13 arguments");
        return NULL;
    }
    const rc_pool_desc* pool = (const rc_pool_desc*)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    const rc_rope_desc* rope = (const rc_rope_desc*)(uintptr_t)PyLong_AsUnsignedLongLong(a[1]);
    if (PyErr_Occurred()) return NULL;
    PyObject *slots = a[2], *positions = a[3], *k = a[4], *v = a[5], *q = a[6], *q_out = a[7], *table = a[8], *tpos = a[9];
    const long long hkv = pool->kv_heads, d = pool->head_dim_k;
    const long long n = ids(slots, "slots", -1);
    if (n < 0 || ids(positions, "positions", n) < 0) return NULL;
    if (n > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "kv_store_rope: too many tokens");
        return NULL;
    }
    int64_t ks = 0, vs = 0, qs = 0, os = 0;
    long long hq = 0;
    if (rows(k, "k_new", n, hkv, d, 0, &ks, NULL)) return NULL;
    if (v != Py_None && rows(v, "v_new", n, hkv, d, 0, &vs, NULL)) return NULL;
    if (q == Py_None && q_out != Py_None) {
        PyErr_SetString(PyExc_ValueError, "kv_store_rope: q_out without q");
        return NULL;
    }
    if (q != Py_None) {
        if (rows(q, "q", n, -1, d, q_out == Py_None, &qs, &hq)) return NULL;
        if (q_out == Py_None) {
            q_out = q;
            os = qs;
        } else if (rows(q_out, "q_out", n, hq, d, 1, &os, NULL)) {
            return NULL;
        }
    }
    if (tpos != Py_None && ids(tpos, "table_pos", n) < 0) return NULL;
    if (table != Py_None && ids(table, "table", -1) < 0) return NULL;
    const long long dev = as_int(PyObject_CallNoArgs(o_get_device));
    if (PyErr_Occurred()) return NULL;
    void *p[8] = {0};
    PyObject* t[8] = {slots, positions, k, v, q, q_out, table, tpos};
    static const char* const names[8] = {"slots", "positions", "k_new", "v_new", "q", "q_out", "table", "table_pos"};
    for (int i = 0; i < 8; ++i)
        if (t[i] != Py_None && address(t[i], names[i], dev, &p[i])) return NULL;
    for (int i = 11; i < 13; ++i) {
        if (a[i] == Py_None) continue;
        const long long d_dev = PyLong_AsLongLong(a[i]);
        if (PyErr_Occurred()) return NULL;
        if (d_dev != dev) {
            PyErr_Format(PyExc_ValueError,
                         "kv_store_rope: the %s on device %lld (-1: the host, -2: several), the current device is %lld",
                         i == 11 ? "pool's arrays are" : "rotation table is", d_dev, dev);
            return NULL;
        }
    }
    unsigned long long stream;
    PyObject* s = a[10] != Py_None ? PyObject_GetAttr(a[10], s_cuda_stream) : NULL;
    if (a[10] == Py_None) {
        PyObject* dv = PyLong_FromLongLong(dev);
        if (!dv) return NULL;
        s = PyObject_CallOneArg(o_get_stream, dv);
        Py_DECREF(dv);
    }
    if (!s) return NULL;
    stream = PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_store_rope(pool, rope, (const int32_t*)p[0], (const int32_t*)p[1], p[2], ks, p[3], vs, (int32_t)n, p[4], qs,
                       (int32_t)hq, p[5], os, (int32_t*)p[6], (const int32_t*)p[7], (rc_stream_t)(uintptr_t)stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* bind(address of kv_store_rope, torch.bfloat16, torch.int32, current device, current stream of a device) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 5) {
        PyErr_SetString(PyExc_TypeError, "bind: 5 arguments");
        return NULL;
    }
    const unsigned long long f = PyLong_AsUnsignedLongLong(a[0]);
    if (PyErr_Occurred()) return NULL;
    PyObject** const to[4] = {&o_bf16, &o_i32, &o_get_device, &o_get_stream};
    for (int i = 0; i < 4; ++i) {
        Py_INCREF(a[i + 1]);
        Py_XDECREF(*to[i]);
        *to[i] = a[i + 1];
    }
    fn_store_rope = (store_rope_fn)(uintptr_t)f;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"kv_store_rope", (PyCFunction)(void (*)(void))store_rope, METH_FASTCALL, NULL},
                                {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "radixattn_host", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_radixattn_host(void) {
    static const char* const names[] = {"data_ptr", "shape", "stride", "dtype", "get_device", "is_contiguous", "cuda_stream"};
    PyObject** const to[] = {&s_data_ptr, &s_shape, &s_stride, &s_dtype, &s_get_device, &s_is_contiguous, &s_cuda_stream};
    for (int i = 0; i < 7; ++i)
        if (!(*to[i] = PyUnicode_InternFromString(names[i]))) return NULL;
    return PyModule_Create(&module);
}
