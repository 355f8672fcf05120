/* Argument marshalling of the per-step calls for Python, in C: kv_store_rope,
 * attn_prompt, kv_load, beam_select and beam_reorder.
 *
 * An append is one launch of about two microseconds of GPU time for a single
 * token, and checking and passing its eight tensors from Python took five
 * microseconds of host time on top of the launch; here it takes about one.
 * Host time of a whole call, from Python before and now: attn_prompt (with its
 * three tensor maps) 14.2 and 5.8 us, kv_load 10.0 and 4.4, beam_select 13.4 and
 * 5.7.
 * The module knows tensors by their Python attributes only (data_ptr, shape,
 * stride, dtype, get_device), so it is built without torch's headers.  Nothing
 * is kept between calls.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>
#include <stdio.h>

#include "radixattn.h"

typedef rc_status (*store_rope_fn)(const rc_pool_desc*, const rc_rope_desc*, const int32_t*, const int32_t*, const void*,
                                   int64_t, const void*, int64_t, int32_t, const void*, int64_t, int32_t, void*, int64_t,
                                   int32_t*, const int32_t*, rc_stream_t);

typedef rc_status (*prompt_fn)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const int32_t*, int32_t,
                               int64_t, int32_t, int32_t, int32_t, float, void*, float*, int32_t*, rc_stream_t);
typedef rc_status (*load_fn)(const rc_pool_desc*, const int32_t*, int32_t, void*, int64_t, void*, int64_t, rc_stream_t);
typedef rc_status (*select_fn)(const void*, int32_t, int64_t, int32_t, int32_t, int32_t, const float*, const uint8_t*,
                               int32_t, int32_t, float*, int32_t*, int32_t*, uint8_t*, int32_t*, rc_stream_t);
typedef rc_status (*reorder_fn)(const int32_t*, int32_t*, int64_t, const int32_t*, const int32_t*, const int32_t*,
                                const int32_t*, int32_t, int32_t, int32_t, int32_t*, rc_stream_t);

/* set by bind() */
static store_rope_fn fn_store_rope;
static prompt_fn fn_prompt;
static load_fn fn_load;
static select_fn fn_select;
static reorder_fn fn_reorder;
static PyObject *o_bf16, *o_i32, *o_f32, *o_u8, *o_bool, *o_get_device, *o_get_stream;
static PyObject *s_data_ptr, *s_shape, *s_stride, *s_dtype, *s_get_device, *s_is_contiguous, *s_cuda_stream, *s_numel,
    *s_device;

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

/* Positions on several axes: a contiguous int32 tensor [axes, n], or with rows for further axes (up to 4 in all) behind
 * them, which no pair turns by. */
static int axis_ids(PyObject* t, const char* name, long long axes, long long n) {
    const int ok = has_dtype(t, o_i32);
    if (ok < 0) return -1;
    long long sh[4] = {0};
    const Py_ssize_t nd = as_sizes(PyObject_GetAttr(t, s_shape), sh);
    if (nd < 0) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    const int dense = c == Py_True;
    Py_DECREF(c);
    if (!ok || !dense || nd != 2 || sh[0] < axes || sh[0] > 4 || sh[1] != n) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous int32 tensor [%lld, %lld] (or of up to 4 axes)", name, axes, n);
        return -1;
    }
    return 0;
}

/* The stream's handle; None: the current one of device `dev`. */
static int stream_of(PyObject* stream, long long dev, rc_stream_t* out) {
    PyObject* s = NULL;
    if (stream != Py_None) {
        s = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        PyObject* dv = PyLong_FromLongLong(dev);
        if (!dv) return -1;
        s = PyObject_CallOneArg(o_get_stream, dv);
        Py_DECREF(dv);
    }
    if (!s) return -1;
    *out = (rc_stream_t)(uintptr_t)PyLong_AsUnsignedLongLong(s);
    Py_DECREF(s);
    return PyErr_Occurred() ? -1 : 0;
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
    if (n < 0) return NULL;
    int axes = rope->n_axes > 1;
    if (!axes && rope->pair_axis) { /* all pairs turn by axis 0: [n], or that axis and others */
        long long sh[4] = {0};
        const Py_ssize_t nd = as_sizes(PyObject_GetAttr(positions, s_shape), sh);
        if (nd < 0) return NULL;
        axes = nd == 2;
    }
    if (axes ? axis_ids(positions, "positions", rope->n_axes, n) < 0 : ids(positions, "positions", n) < 0) return NULL;
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
    rc_stream_t stream;
    if (stream_of(a[10], dev, &stream)) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_store_rope(pool, rope, (const int32_t*)p[0], (const int32_t*)p[1], p[2], ks, p[3], vs, (int32_t)n, p[4], qs,
                       (int32_t)hq, p[5], os, (int32_t*)p[6], (const int32_t*)p[7], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* ValueError: `text` (with the call's and the tensor's names in front) and what the tensor is. */
static int refuse(const char* call, const char* name, const char* text, PyObject* t) {
    PyObject *d = PyObject_GetAttr(t, s_dtype), *sh = PyObject_GetAttr(t, s_shape), *st = PyObject_CallMethodNoArgs(t, s_stride);
    if (d && sh && st) PyErr_Format(PyExc_ValueError, "%s: %s is %s, got %S %S with strides %S", call, name, text, d, sh, st);
    Py_XDECREF(d);
    Py_XDECREF(sh);
    Py_XDECREF(st);
    return -1;
}

static int pointer(PyObject* t, void** ptr) {
    PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) return -1;
    *ptr = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/* A contiguous tensor of the type (or of the other one, where given) and of nd sizes (entries < 0: any, and set). */
static int dense(const char* call, const char* name, PyObject* t, PyObject* type, PyObject* other, int nd, long long* size,
                 void** ptr) {
    int ok = has_dtype(t, type);
    if (ok == 0 && other) ok = has_dtype(t, other);
    if (ok < 0) return -1;
    long long sh[4] = {0};
    const Py_ssize_t dims = as_sizes(PyObject_GetAttr(t, s_shape), sh);
    if (dims < 0) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    ok = ok && c == Py_True && dims == nd;
    Py_DECREF(c);
    for (int i = 0; ok && i < nd; ++i) ok = size[i] < 0 || size[i] == sh[i];
    if (!ok) {
        char want[160];
        int at = 0;
        for (int i = 0; i < nd; ++i)
            at += size[i] < 0 ? snprintf(want + at, sizeof want - (size_t)at, "%sany", i ? ", " : "")
                              : snprintf(want + at, sizeof want - (size_t)at, "%s%lld", i ? ", " : "", size[i]);
        PyObject* text = PyUnicode_FromFormat("a contiguous %S tensor [%s]", type, want);
        if (text) refuse(call, name, PyUnicode_AsUTF8(text), t);
        Py_XDECREF(text);
        return -1;
    }
    for (int i = 0; i < nd; ++i) size[i] = sh[i];
    return pointer(t, ptr);
}

/* bf16 rows [tokens, heads, dim] (size; entries < 0: any, and set), each token's dense; elements between tokens. */
static int token_rows(const char* call, const char* name, PyObject* t, long long size[3], int64_t* stride, void** ptr) {
    const int bf16 = has_dtype(t, o_bf16);
    long long sh[4] = {0}, st[4] = {0};
    if (bf16 < 0) return -1;
    const Py_ssize_t dims = as_sizes(PyObject_GetAttr(t, s_shape), sh);
    if (dims < 0) return -1;
    int ok = bf16 && dims == 3;
    for (int i = 0; ok && i < 3; ++i) ok = size[i] < 0 || size[i] == sh[i];
    if (!ok) {
        char want[128];
        snprintf(want, sizeof want, "bf16 [%lld, %lld, %lld] (-1: any)", size[0], size[1], size[2]);
        return refuse(call, name, want, t);
    }
    if (as_sizes(PyObject_CallMethodNoArgs(t, s_stride), st) != 3) return PyErr_Occurred() ? -1 : refuse(call, name, "a matrix of rows", t);
    if ((sh[2] > 1 && st[2] != 1) || (sh[1] > 1 && st[1] != sh[2])) return refuse(call, name, "rows that must be dense for each token", t);
    for (int i = 0; i < 3; ++i) size[i] = sh[i];
    *stride = sh[0] > 1 ? st[0] : sh[1] * sh[2];
    return pointer(t, ptr);
}

/* The call's error word, or None. */
static int error_word(const char* call, PyObject* t, void** ptr) {
    *ptr = NULL;
    if (t == Py_None) return 0;
    const int i32 = has_dtype(t, o_i32);
    if (i32 < 0) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!c) return -1;
    const int ok = i32 && c == Py_True;
    Py_DECREF(c);
    return ok ? pointer(t, ptr) : refuse(call, "err", "a contiguous int32 tensor", t);
}

/* All the tensors are on the current device, which goes to *dev. */
static int on_device(const char* call, PyObject* const* t, int n, long long* dev) {
    *dev = as_int(PyObject_CallNoArgs(o_get_device));
    if (PyErr_Occurred()) return -1;
    for (int i = 0; i < n; ++i) {
        if (t[i] == Py_None) continue;
        const long long d = as_int(PyObject_CallMethodNoArgs(t[i], s_get_device));
        if (PyErr_Occurred()) return -1;
        if (d != *dev) {
            PyObject* v = PyObject_GetAttr(t[i], s_device);
            if (v) PyErr_Format(PyExc_ValueError, "%s: a tensor is on %S, the current device is cuda:%lld", call, v, *dev);
            Py_XDECREF(v);
            return -1;
        }
    }
    return 0;
}

static int small(const char* call, const char* name, long long x) {
    if (x <= INT32_MAX) return 0;
    PyErr_Format(PyExc_ValueError, "%s: %lld %s are too many", call, x, name);
    return -1;
}

static int takes(Py_ssize_t got, Py_ssize_t want, const char* call) {
    if (got == want && fn_store_rope) return 0;
    PyErr_Format(PyExc_TypeError, "%s: bind() first, then %zd arguments", call, want);
    return -1;
}

/* attn_prompt(q, k, v, indptr, sm_scale, out, lse, err, stream) -> status */
static PyObject* prompt(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    static const char call[] = "attn_prompt";
    if (takes(na, 9, call)) return NULL;
    void *q, *k, *v, *ind, *out, *lse = NULL, *err;
    int64_t qs, ks, vs;
    long long qn[3] = {-1, -1, -1};
    if (token_rows(call, "q", a[0], qn, &qs, &q)) return NULL;
    long long kn[3] = {qn[0], -1, qn[2]};
    if (token_rows(call, "k", a[1], kn, &ks, &k)) return NULL;
    long long vn[3] = {qn[0], kn[1], qn[2]}, ln[2] = {qn[0], qn[1]}, in[1] = {-1};
    if (token_rows(call, "v", a[2], vn, &vs, &v) || dense(call, "out", a[5], o_bf16, NULL, 3, qn, &out)) return NULL;
    if (a[6] != Py_None && dense(call, "lse", a[6], o_f32, NULL, 2, ln, &lse)) return NULL;
    if (dense(call, "indptr", a[3], o_i32, NULL, 1, in, &ind) || error_word(call, a[7], &err)) return NULL;
    if (in[0] == 0) {
        PyErr_SetString(PyExc_ValueError, "attn_prompt: indptr has batch + 1 entries");
        return NULL;
    }
    if (small(call, "prompts", in[0]) || small(call, "heads", qn[1]) || small(call, "heads", kn[1]) || small(call, "elements", qn[2]))
        return NULL;
    const double scale = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return NULL;
    PyObject* const t[7] = {a[0], a[1], a[2], a[3], a[5], a[6], a[7]};
    long long dev;
    rc_stream_t stream;
    if (on_device(call, t, 7, &dev) || stream_of(a[8], dev, &stream)) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_prompt(q, qs, k, ks, v, vs, (const int32_t*)ind, (int32_t)(in[0] - 1), qn[0], (int32_t)qn[1], (int32_t)kn[1],
                   (int32_t)qn[2], (float)scale, out, (float*)lse, (int32_t*)err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* kv_load(pool, slots, k_out, v_out, stream, pool's device) -> status.  pool: the descriptor's address. */
static PyObject* load(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    static const char call[] = "kv_load";
    if (takes(na, 6, call)) return NULL;
    const rc_pool_desc* pool = (const rc_pool_desc*)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    if (PyErr_Occurred()) return NULL;
    void *slots, *k = NULL, *v = NULL;
    int64_t ks = 0, vs = 0;
    long long n[1] = {-1};
    if (dense(call, "slots", a[1], o_i32, NULL, 1, n, &slots) || small(call, "slots", n[0])) return NULL;
    long long kn[3] = {n[0], pool->kv_heads, pool->head_dim_k}, vn[3] = {n[0], pool->kv_heads, pool->head_dim_v};
    if (a[2] != Py_None && token_rows(call, "k_out", a[2], kn, &ks, &k)) return NULL;
    if (a[3] != Py_None && token_rows(call, "v_out", a[3], vn, &vs, &v)) return NULL;
    long long dev;
    rc_stream_t stream;
    if (on_device(call, a + 1, 3, &dev)) return NULL;
    if (a[5] != Py_None) {
        const long long d = PyLong_AsLongLong(a[5]);
        if (PyErr_Occurred()) return NULL;
        if (d != dev) {
            PyErr_Format(PyExc_ValueError,
                         "%s: a descriptor's arrays are on device %lld (-1: the host, -2: several), the current device is %lld",
                         call, d, dev);
            return NULL;
        }
    }
    if (stream_of(a[4], dev, &stream)) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_load(pool, (const int32_t*)slots, (int32_t)n[0], k, ks, v, vs, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* beam_select(logits, scores, out_scores, out_tokens, out_parents, done, end_token, out_done, err, stream) -> status */
static PyObject* select_beams(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    static const char call[] = "beam_select";
    if (takes(na, 10, call)) return NULL;
    long long ls[4] = {0}, lt[4] = {0};
    const Py_ssize_t dims = as_sizes(PyObject_GetAttr(a[0], s_shape), ls);
    if (dims < 0) return NULL;
    const int f32 = has_dtype(a[0], o_f32), bf16 = f32 ? 0 : has_dtype(a[0], o_bf16);
    if (f32 < 0 || bf16 < 0) return NULL;
    if (dims != 3 || !(f32 || bf16)) {
        refuse(call, "logits", "bf16 or fp32 [batch, beams, vocab]", a[0]);
        return NULL;
    }
    if (as_sizes(PyObject_CallMethodNoArgs(a[0], s_stride), lt) != 3) return NULL;
    const long long b = ls[0], w = ls[1], vocab = ls[2], stride = w > 1 ? lt[1] : b > 1 ? lt[0] : vocab;
    if ((vocab > 1 && lt[2] != 1) || (b > 1 && w > 1 && lt[0] != w * stride)) {
        refuse(call, "logits", "rows that must be dense and evenly apart", a[0]);
        return NULL;
    }
    void *logits, *scores, *done = NULL, *o_scores, *o_tokens, *o_parents, *o_done = NULL, *err;
    long long in[2] = {b, w}, out[2] = {b, -1};
    if (pointer(a[0], &logits) || dense(call, "scores", a[1], o_f32, NULL, 2, in, &scores)) return NULL;
    if (a[5] != Py_None && dense(call, "done", a[5], o_u8, o_bool, 2, in, &done)) return NULL;
    if (dense(call, "out_scores", a[2], o_f32, NULL, 2, out, &o_scores) ||
        dense(call, "out_tokens", a[3], o_i32, NULL, 2, out, &o_tokens) ||
        dense(call, "out_parents", a[4], o_i32, NULL, 2, out, &o_parents))
        return NULL;
    if (a[7] != Py_None && dense(call, "out_done", a[7], o_u8, o_bool, 2, out, &o_done)) return NULL;
    if (error_word(call, a[8], &err)) return NULL;
    if (small(call, "requests", b) || small(call, "beams", w) || small(call, "tokens", vocab) || small(call, "results", out[1]))
        return NULL;
    const long end = PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return NULL;
    if (end < INT32_MIN || end > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%s: no such end token: %ld", call, end);
        return NULL;
    }
    PyObject* const t[8] = {a[0], a[1], a[2], a[3], a[4], a[5], a[7], a[8]};
    long long dev;
    rc_stream_t stream;
    if (on_device(call, t, 8, &dev) || stream_of(a[9], dev, &stream)) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_select(logits, f32, stride, (int32_t)b, (int32_t)w, (int32_t)vocab, (const float*)scores, (const uint8_t*)done,
                   (int32_t)end, (int32_t)out[1], (float*)o_scores, (int32_t*)o_tokens, (int32_t*)o_parents,
                   (uint8_t*)o_done, (int32_t*)err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* beam_reorder(table, start, first, last, parents, max_cols, out, err, stream) -> status */
static PyObject* reorder(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    static const char call[] = "beam_reorder";
    if (takes(na, 9, call)) return NULL;
    PyObject* const both[2] = {a[0], a[6] == Py_None ? a[0] : a[6]};
    void *table[2], *start, *first, *last, *parents, *err;
    long long numel[2];
    for (int i = 0; i < 2; ++i) {
        const int ok = has_dtype(both[i], o_i32);
        if (ok < 0) return NULL;
        PyObject* c = PyObject_CallMethodNoArgs(both[i], s_is_contiguous);
        if (!c) return NULL;
        const int same = c == Py_True;
        Py_DECREF(c);
        if (!ok || !same) {
            refuse(call, i ? "out" : "table", "a contiguous int32 tensor", both[i]);
            return NULL;
        }
        numel[i] = as_int(PyObject_CallMethodNoArgs(both[i], s_numel));
        if (PyErr_Occurred() || pointer(both[i], &table[i])) return NULL;
    }
    if (numel[0] != numel[1]) {
        PyErr_Format(PyExc_ValueError, "%s: table and out differ in size", call);
        return NULL;
    }
    long long n[2] = {-1, -1};
    if (dense(call, "parents", a[4], o_i32, NULL, 2, n, &parents) || dense(call, "start", a[1], o_i32, NULL, 2, n, &start) ||
        dense(call, "first", a[2], o_i32, NULL, 1, n, &first) || dense(call, "last", a[3], o_i32, NULL, 1, n, &last) ||
        error_word(call, a[7], &err) || small(call, "requests", n[0]) || small(call, "beams", n[1]))
        return NULL;
    const long cols = PyLong_AsLong(a[5]);
    if (PyErr_Occurred() || small(call, "columns", cols)) return NULL;
    PyObject* const t[7] = {both[0], both[1], a[1], a[2], a[3], a[4], a[7]};
    long long dev;
    rc_stream_t stream;
    if (on_device(call, t, 7, &dev) || stream_of(a[8], dev, &stream)) return NULL;
    rc_status st;
    Py_BEGIN_ALLOW_THREADS
    st = fn_reorder((const int32_t*)table[0], (int32_t*)table[1], numel[0], (const int32_t*)start, (const int32_t*)first,
                    (const int32_t*)last, (const int32_t*)parents, (int32_t)n[0], (int32_t)n[1],
                    cols < 0 ? -1 : (int32_t)cols, (int32_t*)err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* bind(addresses of kv_store_rope, attn_prompt, kv_load, beam_select and beam_reorder, torch.bfloat16, torch.int32,
 * torch.float32, torch.uint8, torch.bool, current device, current stream of a device) */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t na) {
    (void)self;
    if (na != 12) {
        PyErr_SetString(PyExc_TypeError, "bind: 12 arguments");
        return NULL;
    }
    unsigned long long f[5];
    for (int i = 0; i < 5; ++i) {
        f[i] = PyLong_AsUnsignedLongLong(a[i]);
        if (PyErr_Occurred()) return NULL;
    }
    PyObject** const to[7] = {&o_bf16, &o_i32, &o_f32, &o_u8, &o_bool, &o_get_device, &o_get_stream};
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(a[i + 5]);
        Py_XDECREF(*to[i]);
        *to[i] = a[i + 5];
    }
    fn_store_rope = (store_rope_fn)(uintptr_t)f[0];
    fn_prompt = (prompt_fn)(uintptr_t)f[1];
    fn_load = (load_fn)(uintptr_t)f[2];
    fn_select = (select_fn)(uintptr_t)f[3];
    fn_reorder = (reorder_fn)(uintptr_t)f[4];
    Py_RETURN_NONE;
}

#define CALL(name, f) {name, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {CALL("kv_store_rope", store_rope),  CALL("attn_prompt", prompt),   CALL("kv_load", load),
                                CALL("beam_select", select_beams),  CALL("beam_reorder", reorder), CALL("bind", bind),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "radixattn_host", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_radixattn_host(void) {
    static const char* const names[] = {"data_ptr",      "shape",       "stride", "dtype", "get_device",
                                        "is_contiguous", "cuda_stream", "numel",  "device"};
    PyObject** const to[] = {&s_data_ptr,      &s_shape,       &s_stride, &s_dtype, &s_get_device,
                             &s_is_contiguous, &s_cuda_stream, &s_numel,  &s_device};
    for (int i = 0; i < 9; ++i)
        if (!(*to[i] = PyUnicode_InternFromString(names[i]))) return NULL;
    return PyModule_Create(&module);
}
