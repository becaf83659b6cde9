/*
 * pkv_binding.c -- argument marshalling of the per-step calls, as a CPython
 * module.
 *
 * A decode step makes a handful of calls whose kernels take 3 to 10 us when a
 * batch is small, and the step's host time is then the launches plus the
 * marshalling.  In the interpreter, with ctypes, that marshalling costs 5 us a
 * call (17 arguments, eight tensors); here it costs about 1 us.  The functions
 * check what the calls' Python wrappers document (types, shapes, devices, pool
 * sizes), raise TypeError / ValueError like them, call the C ABI through the
 * addresses given to bind() and return its status.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "../../include/pagedkv.h"

static struct {
    pkv_status (*append)(const void*, const void*, int32_t, int32_t, const int64_t*, void*, void*, const pkv_cache_desc*,
                         void*);
    pkv_status (*read)(const int64_t*, int32_t, const void*, const void*, const pkv_cache_desc*, void*, void*, int32_t,
                       void*);
    pkv_status (*decode)(const void*, int32_t, int32_t, int32_t, const void*, const void*, const pkv_cache_desc*,
                         const int32_t*, int32_t, const int32_t*, int32_t, float, void*, void*, size_t, int32_t, void*);
    pkv_status (*bounds)(const void*, const pkv_cache_desc*, const int32_t*, int32_t, const int32_t*, const int32_t*,
                         int32_t, int32_t, void*, int32_t, void*);
    pkv_status (*select)(const void*, int32_t, int32_t, int32_t, const void*, const pkv_cache_desc*, const int32_t*,
                         int32_t, const int32_t*, int32_t, int32_t, int32_t, int32_t, int32_t*, void*, size_t, void*);
    pkv_status (*sparse)(const void*, int32_t, int32_t, int32_t, const void*, const void*, const pkv_cache_desc*,
                         const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t, float, void*, void*, size_t,
                         int32_t, void*);
    pkv_status (*scored)(const void*, int32_t, int32_t, int32_t, const void*, const void*, const pkv_cache_desc*,
                         const int32_t*, int32_t, const int32_t*, int32_t, float, const pkv_score_mod*, float*,
                         const int32_t*, void*, void*, size_t, int32_t, void*);
    pkv_status (*prefill)(const void*, int32_t, int32_t, int32_t, int32_t, const int32_t*, int32_t, const void*, const void*,
                          const pkv_cache_desc*, const int32_t*, int32_t, const int32_t*, const int32_t*, int32_t, float,
                          const pkv_score_mod*, void*, void*, size_t, void*);
    pkv_status (*rope)(const void*, int64_t, int32_t, const void*, int64_t, const void*, int64_t, int32_t, int32_t,
                       const int32_t*, const int64_t*, const float*, int32_t, int32_t, float, void*, void*,
                       const pkv_cache_desc*, void*, int64_t, void*);
    pkv_status (*select_tokens)(const float*, const pkv_cache_desc*, const int32_t*, int32_t, const int32_t*, int32_t,
                                int32_t, int32_t, int32_t, int32_t, int32_t*, void*);
    pkv_status (*compact)(const int32_t*, int32_t, void*, void*, float*, const pkv_cache_desc*, const int32_t*, int32_t,
                          const int32_t*, int32_t, const int32_t*, int32_t, void*);
    size_t (*block_bytes)(const pkv_cache_desc*);
} fn;

/* Objects of torch that bind() keeps. */
static PyObject *t_i32, *t_i64, *t_f16, *t_bf16, *t_f32, *f_device, *f_raw_stream, *f_stream;
/* Attribute and method names. */
static PyObject *s_get_device, *s_is_contiguous, *s_stride, *s_data_ptr, *s_shape, *s_dtype, *s_nbytes, *s_num_blocks,
    *s_block_size, *s_num_kv_heads, *s_head_size, *s_kv_dtype, *s_k_scale, *s_v_scale, *s_cap, *s_window, *s_slopes,
    *s_first, *s_prefix_lens;

static const char* const kDtypes[5] = {"f16", "bf16", "e4m3", "int8", "int4"};

static int as_i32(PyObject* o, int32_t* out) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "a size does not fit 32 bits");
        return -1;
    }
    *out = (int32_t)v;
    return 0;
}

static int attr_i32(PyObject* o, PyObject* name, int32_t* out) {
    PyObject* a = PyObject_GetAttr(o, name);
    if (!a) return -1;
    const int r = as_i32(a, out);
    Py_DECREF(a);
    return r;
}

static int attr_float(PyObject* o, PyObject* name, float* out) {
    PyObject* a = PyObject_GetAttr(o, name);
    if (!a) return -1;
    const double v = PyFloat_AsDouble(a);
    Py_DECREF(a);
    if (v == -1.0 && PyErr_Occurred()) return -1;
    *out = (float)v;
    return 0;
}

static int dtype_of_name(PyObject* name, int32_t* out) {
    for (int i = 0; i < 5; ++i)
        if (PyUnicode_Check(name) && PyUnicode_CompareWithASCIIString(name, kDtypes[i]) == 0) {
            *out = i;
            return 0;
        }
    PyErr_SetObject(PyExc_KeyError, name);
    return -1;
}

static int get_desc(PyObject* d, pkv_cache_desc* c) {
    if (attr_i32(d, s_num_blocks, &c->num_blocks) || attr_i32(d, s_block_size, &c->block_size) ||
        attr_i32(d, s_num_kv_heads, &c->num_kv_heads) || attr_i32(d, s_head_size, &c->head_size) ||
        attr_float(d, s_k_scale, &c->k_scale) || attr_float(d, s_v_scale, &c->v_scale))
        return -1;
    PyObject* a = PyObject_GetAttr(d, s_kv_dtype);
    if (!a) return -1;
    const int r = dtype_of_name(a, &c->kv_dtype);
    Py_DECREF(a);
    return r;
}

/* 16-bit element type of a tensor, or the declared one. */
static int element_type(PyObject* t, PyObject* declared, int32_t* out) {
    if (declared != Py_None) return dtype_of_name(declared, out);
    PyObject* a = PyObject_GetAttr(t, s_dtype);
    if (!a) return -1;
    int r = 0;
    if (a == t_f16)
        *out = PKV_F16;
    else if (a == t_bf16)
        *out = PKV_BF16;
    else {
        PyErr_Format(PyExc_TypeError, "cannot infer element type from %S; pass it explicitly", a);
        r = -1;
    }
    Py_DECREF(a);
    return r;
}

/* 1 if the tensor has the element type (an object of torch), 0 if not, -1 on error. */
static int is_type(PyObject* t, PyObject* dtype) {
    PyObject* a = PyObject_GetAttr(t, s_dtype);
    if (!a) return -1;
    Py_DECREF(a);
    return a == dtype;
}

static int want_i32(PyObject* t, const char* what) {
    const int r = is_type(t, t_i32);
    if (r == 0) PyErr_Format(PyExc_TypeError, "%s must be int32", what);
    return r == 1 ? 0 : -1;
}

/* The first n sizes of a tensor, which has n dimensions or (more) at least n. */
static int sizes(PyObject* t, const char* name, int n, int more, int32_t* out) {
    PyObject* a = PyObject_GetAttr(t, s_shape);
    if (!a) return -1;
    int r = 0;
    if (!PyTuple_Check(a) || PyTuple_GET_SIZE(a) < n || (!more && PyTuple_GET_SIZE(a) != n)) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", name, n);
        r = -1;
    }
    for (int i = 0; i < n && r == 0; ++i) r = as_i32(PyTuple_GET_ITEM(a, i), out + i);
    Py_DECREF(a);
    return r;
}

static int dims(PyObject* t, const char* name, int n, int32_t* out) { return sizes(t, name, n, 0, out); }

/* Data pointer of a contiguous CUDA tensor; dev >= 0: of that device only. */
static int ptr_of(PyObject* t, const char* name, long dev, void** out) {
    PyObject* r = PyObject_CallMethodNoArgs(t, s_get_device);
    const long d = r ? PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    if (d < 0) {
        PyErr_Clear();
        PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
        return -1;
    }
    if (dev >= 0 && d != dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the current device is cuda:%ld", name, d, dev);
        return -1;
    }
    r = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!r) return -1;
    Py_DECREF(r);
    if (r != Py_True) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
        return -1;
    }
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) return -1;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return PyErr_Occurred() ? -1 : 0;
}

static int bytes_of(PyObject* t, size_t* out) {
    PyObject* a = PyObject_GetAttr(t, s_nbytes);
    if (!a) return -1;
    *out = PyLong_AsSize_t(a);
    Py_DECREF(a);
    return *out == (size_t)-1 && PyErr_Occurred() ? -1 : 0;
}

/* A tensor whose type may be declared by name has n elements of 16 bits. */
static int bytes16(PyObject* t, size_t n, const char* name) {
    size_t got;
    if (bytes_of(t, &got)) return -1;
    if (got == 2 * n) return 0;
    PyErr_Format(PyExc_TypeError, "%s must be of a 16-bit type", name);
    return -1;
}

/* A pool tensor has the size its description gives (a description that is not
 * supported is left to the call's own checks). */
static int pool_size(PyObject* t, const pkv_cache_desc* c, const char* name) {
    const size_t block = fn.block_bytes(c);
    size_t n;
    if (bytes_of(t, &n)) return -1;
    if (block && c->num_blocks >= 0 && n != block * (size_t)c->num_blocks) {
        PyErr_Format(PyExc_ValueError, "%s must hold %d blocks of %zu bytes", name, c->num_blocks, block);
        return -1;
    }
    return 0;
}

static int is_int(const pkv_cache_desc* c) { return c->kv_dtype == PKV_INT8 || c->kv_dtype == PKV_INT4; }

static int int_pools(const pkv_cache_desc* c, PyObject* k, PyObject* v) {
    if (!is_int(c)) return 0;
    return pool_size(k, c, "k_cache") || pool_size(v, c, "v_cache") ? -1 : 0;
}

/* Two operands of a call on an integer-coded pool: one type, and rows for each token or query head. */
static int int_rows(const pkv_cache_desc* c, PyObject* x, PyObject* y, int32_t n, int32_t heads, const char* what) {
    if (!is_int(c)) return 0;
    size_t nx, ny;
    PyObject* d = PyObject_GetAttr(x, s_dtype);
    if (!d) return -1;
    const int alike = is_type(y, d);
    Py_DECREF(d);
    if (alike < 0 || bytes_of(x, &nx) || bytes_of(y, &ny)) return -1;
    const size_t want = heads < 0 || c->head_size < 0 ? 0 : (size_t)n * heads * c->head_size * 2;
    if (!alike || nx < want || ny < want) {
        PyErr_Format(PyExc_ValueError, "%s must be of one 16-bit type and hold %zu bytes each", what, want);
        return -1;
    }
    return 0;
}

static int current_device(long* dev) {
    PyObject* r = PyObject_CallNoArgs(f_device);
    if (!r) return -1;
    *dev = PyLong_AsLong(r);
    Py_DECREF(r);
    return *dev == -1 && PyErr_Occurred() ? -1 : 0;
}

/* The device that a call on an integer-coded pool expects its tensors on, that of x and current; -1 (any) otherwise. */
static int int_device(const pkv_cache_desc* c, PyObject* x, const char* name, long* dev) {
    void* p;
    *dev = -1;
    if (!is_int(c)) return 0;
    return ptr_of(x, name, -1, &p) || current_device(dev) ? -1 : 0;
}

/* The stream's handle: the current one of the current device for None. */
static int stream_of(PyObject* s, void** out) {
    PyObject* r;
    if (s == Py_None) {
        PyObject* d = PyObject_CallNoArgs(f_device);
        if (!d) return -1;
        r = PyObject_CallOneArg(f_raw_stream, d);
        Py_DECREF(d);
    } else {
        r = PyObject_CallOneArg(f_stream, s);
    }
    if (!r) return -1;
    *out = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return PyErr_Occurred() ? -1 : 0;
}

static int workspace_of(PyObject* w, long dev, void** p, size_t* n) {
    *p = NULL;
    *n = 0;
    if (w == Py_None) return 0;
    return ptr_of(w, "workspace", dev, p) || bytes_of(w, n) ? -1 : 0;
}

static int same(int32_t got, int32_t want, const char* what) {
    if (got == want) return 0;
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

static int nargs_ok(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 1;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return 0;
}

/* Makes the call without the interpreter's lock (a launch may wait for room in the queue). */
#define DONE(call)                               \
    do {                                         \
        pkv_status status_;                      \
        Py_BEGIN_ALLOW_THREADS                   \
        status_ = (call);                        \
        Py_END_ALLOW_THREADS                     \
        return PyLong_FromLong((long)status_);   \
    } while (0)

/* append(k, v, slot_mapping, k_cache, v_cache, desc, in_dtype, stream) */
static PyObject* py_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, T[1];
    void *k, *v, *slots, *kc, *vc, *st;
    long dev;
    if (!nargs_ok(n, 8)) return NULL;
    const int i64 = is_type(a[2], t_i64);
    if (i64 < 0) return NULL;
    if (!i64) {
        PyErr_SetString(PyExc_TypeError, "slot_mapping must be int64");
        return NULL;
    }
    if (get_desc(a[5], &c) || int_pools(&c, a[3], a[4]) || sizes(a[2], "slot_mapping", 1, 1, T) ||
        int_rows(&c, a[0], a[1], T[0], c.num_kv_heads, "k and v") || int_device(&c, a[0], "k", &dev) ||
        ptr_of(a[0], "k", dev, &k) || ptr_of(a[1], "v", dev, &v) || element_type(a[0], a[6], &type) ||
        ptr_of(a[2], "slot_mapping", dev, &slots) || ptr_of(a[3], "k_cache", dev, &kc) ||
        ptr_of(a[4], "v_cache", dev, &vc) || stream_of(a[7], &st))
        return NULL;
    DONE(fn.append(k, v, type, T[0], (const int64_t*)slots, kc, vc, &c, st));
}

/* read(slot_mapping, k_cache, v_cache, desc, k_out, v_out, out_dtype, stream) */
static PyObject* py_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, T[1], ks[3], vs[3];
    void *slots, *kc, *vc, *ko, *vo, *st;
    long dev;
    if (!nargs_ok(n, 8)) return NULL;
    const int i64 = is_type(a[0], t_i64);
    if (i64 < 0) return NULL;
    if (!i64) {
        PyErr_SetString(PyExc_TypeError, "slot_mapping must be int64");
        return NULL;
    }
    if (get_desc(a[3], &c) || dims(a[0], "slot_mapping", 1, T) || dims(a[4], "k_out", 3, ks) ||
        dims(a[5], "v_out", 3, vs))
        return NULL;
    for (int i = 0; i < 3; ++i) {
        const int32_t want = i == 0 ? T[0] : (i == 1 ? c.num_kv_heads : c.head_size);
        if (same(ks[i], want, "k_out must have shape [num_tokens, num_kv_heads, head_size]") ||
            same(vs[i], want, "v_out must have shape [num_tokens, num_kv_heads, head_size]"))
            return NULL;
    }
    if (element_type(a[4], a[6], &type)) return NULL;
    PyObject* d = PyObject_GetAttr(a[4], s_dtype);
    if (!d) return NULL;
    const int alike = is_type(a[5], d);
    Py_DECREF(d);
    if (alike < 0) return NULL;
    size_t nk;
    if (bytes_of(a[4], &nk)) return NULL;
    if (!alike || nk != (size_t)T[0] * c.num_kv_heads * c.head_size * 2) {
        PyErr_SetString(PyExc_TypeError, "k_out and v_out must be of one 16-bit type");
        return NULL;
    }
    if (ptr_of(a[0], "slot_mapping", -1, &slots) || current_device(&dev) || ptr_of(a[0], "slot_mapping", dev, &slots) ||
        pool_size(a[1], &c, "k_cache") || pool_size(a[2], &c, "v_cache") || ptr_of(a[1], "k_cache", dev, &kc) ||
        ptr_of(a[2], "v_cache", dev, &vc) || ptr_of(a[4], "k_out", dev, &ko) || ptr_of(a[5], "v_out", dev, &vo) ||
        stream_of(a[7], &st))
        return NULL;
    DONE(fn.read((const int64_t*)slots, T[0], kc, vc, &c, ko, vo, type, st));
}

/* decode(q, k_cache, v_cache, desc, block_tables, seq_lens, max_seq_len, scale, out, workspace, partition_tokens,
 *        q_dtype, stream) */
static PyObject* py_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, qs[2], ts[2], S[1], max_len, part;
    void *q, *kc, *vc, *tables, *lens, *out, *ws, *st;
    size_t wn;
    long dev;
    if (!nargs_ok(n, 13)) return NULL;
    if (want_i32(a[4], "block_tables and seq_lens") || want_i32(a[5], "block_tables and seq_lens") ||
        get_desc(a[3], &c) || int_pools(&c, a[1], a[2]) || sizes(a[0], "q", 2, 1, qs) || sizes(a[4], "block_tables", 2, 1, ts) ||
        as_i32(a[6], &max_len) || as_i32(a[10], &part))
        return NULL;
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    if (is_int(&c)) {
        if (int_rows(&c, a[0], a[8], qs[0], qs[1], "q and out") || sizes(a[5], "seq_lens", 1, 1, S)) return NULL;
        if (ts[0] < qs[0] || S[0] < qs[0]) {
            PyErr_SetString(PyExc_ValueError, "block_tables and seq_lens must have a row for each sequence");
            return NULL;
        }
    }
    if (int_device(&c, a[0], "q", &dev) || ptr_of(a[0], "q", dev, &q) || element_type(a[0], a[11], &type) ||
        ptr_of(a[1], "k_cache", dev, &kc) || ptr_of(a[2], "v_cache", dev, &vc) ||
        ptr_of(a[4], "block_tables", dev, &tables) || ptr_of(a[5], "seq_lens", dev, &lens) ||
        ptr_of(a[8], "out", dev, &out) || workspace_of(a[9], dev, &ws, &wn) ||
        stream_of(a[12], &st))
        return NULL;
    DONE(fn.decode(q, type, qs[0], qs[1], kc, vc, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens, max_len,
                   (float)scale, out, ws, wn, part, st));
}

/* key_bounds(k_cache, desc, block_tables, seq_lens, new_lens, max_new_len, bounds, bounds_dtype, stream) */
static PyObject* py_bounds(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, ts[2], S[1], N[1], bs[4], max_new;
    void *kc, *tables, *lens, *fresh = NULL, *bounds, *st;
    long dev;
    if (!nargs_ok(n, 9)) return NULL;
    if (want_i32(a[2], "block_tables and seq_lens") || want_i32(a[3], "block_tables and seq_lens") ||
        get_desc(a[1], &c) || dims(a[2], "block_tables", 2, ts) || dims(a[3], "seq_lens", 1, S) ||
        same(ts[0], S[0], "block_tables must have one row per sequence"))
        return NULL;
    if (a[4] != Py_None) {
        const int ok = is_type(a[4], t_i32);
        if (ok < 0 || dims(a[4], "new_lens", 1, N)) return NULL;
        if (!ok || N[0] != S[0]) {
            PyErr_SetString(PyExc_ValueError, "new_lens must be int32 with one entry per sequence");
            return NULL;
        }
    }
    if (as_i32(a[5], &max_new) || dims(a[6], "bounds", 4, bs)) return NULL;
    const int32_t want[4] = {c.num_blocks, c.num_kv_heads, 2, c.head_size};
    for (int i = 0; i < 4; ++i)
        if (same(bs[i], want[i], "bounds must have shape [num_blocks, num_kv_heads, 2, head_size]")) return NULL;
    if (element_type(a[6], a[7], &type) || bytes16(a[6], (size_t)bs[0] * bs[1] * 2 * bs[3], "bounds")) return NULL;
    if (ptr_of(a[3], "seq_lens", -1, &lens) || current_device(&dev) || ptr_of(a[3], "seq_lens", dev, &lens) ||
        pool_size(a[0], &c, "k_cache") || ptr_of(a[0], "k_cache", dev, &kc) ||
        ptr_of(a[2], "block_tables", dev, &tables) || (a[4] != Py_None && ptr_of(a[4], "new_lens", dev, &fresh)) ||
        ptr_of(a[6], "bounds", dev, &bounds) || stream_of(a[8], &st))
        return NULL;
    DONE(fn.bounds(kc, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens, (const int32_t*)fresh, max_new, S[0],
                   bounds, type, st));
}

/* Shapes that selection and sparse decode share: q [S, Hq, D], block_tables [S, MB], seq_lens [S], selected [S, Hkv, n]. */
static int lists_ok(PyObject* q, PyObject* tables, PyObject* lens, PyObject* selected, const pkv_cache_desc* c,
                    int32_t* qs, int32_t* ts, int32_t* ss) {
    int32_t S[1];
    if (want_i32(tables, "block_tables, seq_lens and selected") || want_i32(lens, "block_tables, seq_lens and selected") ||
        want_i32(selected, "block_tables, seq_lens and selected") || dims(q, "q", 3, qs) ||
        dims(tables, "block_tables", 2, ts) || dims(lens, "seq_lens", 1, S) || dims(selected, "selected", 3, ss) ||
        same(qs[2], c->head_size, "q must have the cache's head_size") ||
        same(ss[0], qs[0], "selected must have shape [num_seqs, num_kv_heads, n]") ||
        same(ss[1], c->num_kv_heads, "selected must have shape [num_seqs, num_kv_heads, n]") ||
        same(ts[0], qs[0], "block_tables and seq_lens must have one row per sequence") ||
        same(S[0], qs[0], "block_tables and seq_lens must have one row per sequence"))
        return -1;
    return bytes16(q, (size_t)qs[0] * qs[1] * qs[2], "q");
}

/* select(q, bounds, desc, block_tables, seq_lens, max_seq_len, selected, workspace, sink_blocks, recent_blocks, q_dtype,
 *        stream) */
static PyObject* py_select(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, qs[3], ts[2], ss[3], bs[4], max_len, sink, recent;
    void *q, *bounds, *tables, *lens, *selected, *ws, *st;
    size_t wn;
    long dev;
    if (!nargs_ok(n, 12)) return NULL;
    PyObject* d = PyObject_GetAttr(a[0], s_dtype);
    if (!d) return NULL;
    const int alike = is_type(a[1], d);
    Py_DECREF(d);
    if (alike < 0) return NULL;
    if (!alike) {
        PyErr_SetString(PyExc_TypeError, "bounds must have q's type");
        return NULL;
    }
    if (get_desc(a[2], &c) || lists_ok(a[0], a[3], a[4], a[6], &c, qs, ts, ss) || dims(a[1], "bounds", 4, bs)) return NULL;
    const int32_t want[4] = {c.num_blocks, c.num_kv_heads, 2, c.head_size};
    for (int i = 0; i < 4; ++i)
        if (same(bs[i], want[i], "bounds must have shape [num_blocks, num_kv_heads, 2, head_size]")) return NULL;
    if (bytes16(a[1], (size_t)bs[0] * bs[1] * 2 * bs[3], "bounds")) return NULL;
    if (as_i32(a[5], &max_len) || as_i32(a[8], &sink) || as_i32(a[9], &recent) || element_type(a[0], a[10], &type) ||
        ptr_of(a[0], "q", -1, &q) || current_device(&dev) || ptr_of(a[0], "q", dev, &q) ||
        ptr_of(a[1], "bounds", dev, &bounds) || ptr_of(a[3], "block_tables", dev, &tables) ||
        ptr_of(a[4], "seq_lens", dev, &lens) || ptr_of(a[6], "selected", dev, &selected) ||
        workspace_of(a[7], dev, &ws, &wn) || stream_of(a[11], &st))
        return NULL;
    DONE(fn.select(q, type, qs[0], qs[1], bounds, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens, max_len, ss[2],
                   sink, recent, (int32_t*)selected, ws, wn, st));
}

/* sparse(q, k_cache, v_cache, desc, block_tables, seq_lens, selected, scale, out, workspace, partition_blocks, q_dtype,
 *        stream) */
static PyObject* py_sparse(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, qs[3], ts[2], ss[3], os[3], part;
    void *q, *kc, *vc, *tables, *lens, *selected, *out, *ws, *st;
    size_t wn;
    long dev;
    if (!nargs_ok(n, 13)) return NULL;
    if (get_desc(a[3], &c) || lists_ok(a[0], a[4], a[5], a[6], &c, qs, ts, ss) || dims(a[8], "out", 3, os)) return NULL;
    PyObject* d = PyObject_GetAttr(a[0], s_dtype);
    if (!d) return NULL;
    const int alike = is_type(a[8], d);
    Py_DECREF(d);
    if (alike < 0) return NULL;
    if (!alike || os[0] != qs[0] || os[1] != qs[1] || os[2] != qs[2]) {
        PyErr_SetString(PyExc_ValueError, "out must have q's shape and type");
        return NULL;
    }
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    if (as_i32(a[10], &part) || element_type(a[0], a[11], &type) || ptr_of(a[0], "q", -1, &q) || current_device(&dev) ||
        ptr_of(a[0], "q", dev, &q) || pool_size(a[1], &c, "k_cache") || pool_size(a[2], &c, "v_cache") ||
        ptr_of(a[1], "k_cache", dev, &kc) || ptr_of(a[2], "v_cache", dev, &vc) ||
        ptr_of(a[4], "block_tables", dev, &tables) || ptr_of(a[5], "seq_lens", dev, &lens) ||
        ptr_of(a[6], "selected", dev, &selected) || ptr_of(a[8], "out", dev, &out) ||
        workspace_of(a[9], dev, &ws, &wn) || stream_of(a[12], &st))
        return NULL;
    DONE(fn.sparse(q, type, qs[0], qs[1], kc, vc, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens,
                   (const int32_t*)selected, ss[2], (float)scale, out, ws, wn, part, st));
}

/* Pointer of an optional tensor of n elements of a type; NULL for None.  p NULL: its type and size alone. */
static int optional_vector(PyObject* t, PyObject* dtype, int32_t n, const char* name, const char* kind, long dev, void** p) {
    int32_t got[1];
    if (p) *p = NULL;
    if (t == Py_None) return 0;
    const int ok = is_type(t, dtype);
    if (ok < 0 || dims(t, name, 1, got)) return -1;
    if (!ok || got[0] != n) {
        PyErr_Format(PyExc_ValueError, "%s must be %s with %d entries", name, kind, n);
        return -1;
    }
    return p ? ptr_of(t, name, dev, p) : 0;
}

/* A ScoreMod (None: plain scores): heads slopes, n first positions, S prefix lengths.  pointers 0: their types and
 * sizes alone. */
static int get_score(PyObject* o, int32_t heads, int32_t n, int32_t S, long dev, int pointers, pkv_score_mod* m) {
    memset(m, 0, sizeof *m);
    if (o == Py_None) return 0;
    if (attr_float(o, s_cap, &m->cap) || attr_i32(o, s_window, &m->window)) return -1;
    PyObject* const names[3] = {s_slopes, s_first, s_prefix_lens};
    void* p[3] = {NULL, NULL, NULL};
    for (int i = 0; i < 3; ++i) {
        PyObject* a = PyObject_GetAttr(o, names[i]);
        if (!a) return -1;
        void** at = pointers ? &p[i] : NULL;
        const int r = i == 0   ? optional_vector(a, t_f32, heads, "slopes", "float32", dev, at)
                      : i == 1 ? optional_vector(a, t_i32, n, "first", "int32", dev, at)
                               : optional_vector(a, t_i32, S, "prefix_lens", "int32", dev, at);
        Py_DECREF(a);
        if (r) return -1;
    }
    m->slopes = (const float*)p[0];
    m->first = (const int32_t*)p[1];
    m->prefix_lens = (const int32_t*)p[2];
    return 0;
}

/* Weights of cached tokens, float32 [num_blocks, num_kv_heads, block_size]. */
static int weights_of(PyObject* t, const pkv_cache_desc* c, long dev, void** p) {
    int32_t ws[3];
    *p = NULL;
    if (t == Py_None) return 0;
    const int ok = is_type(t, t_f32);
    if (ok < 0 || dims(t, "weights", 3, ws)) return -1;
    if (!ok || ws[0] != c->num_blocks || ws[1] != c->num_kv_heads || ws[2] != c->block_size) {
        PyErr_SetString(PyExc_ValueError, "weights must be float32 [num_blocks, num_kv_heads, block_size]");
        return -1;
    }
    return ptr_of(t, "weights", dev, p);
}

/* q [S, Hq, D] with a table row and a length for each sequence. */
static int batch_ok(PyObject* q, PyObject* tables, PyObject* lens, const pkv_cache_desc* c, int32_t* qs, int32_t* ts) {
    int32_t S[1];
    if (want_i32(tables, "block_tables and seq_lens") || want_i32(lens, "block_tables and seq_lens") ||
        dims(q, "q", 3, qs) || dims(tables, "block_tables", 2, ts) || dims(lens, "seq_lens", 1, S) ||
        same(qs[2], c->head_size, "q must have the cache's head_size") ||
        same(ts[0], qs[0], "block_tables and seq_lens must have one row per sequence") ||
        same(S[0], qs[0], "block_tables and seq_lens must have one row per sequence"))
        return -1;
    return bytes16(q, (size_t)qs[0] * qs[1] * qs[2], "q");
}

/* 0 if y has x's shape (three sizes) and type. */
static int alike3(PyObject* x, const int32_t* xs, PyObject* y, const char* name, const char* what) {
    int32_t ys[3];
    if (dims(y, name, 3, ys)) return -1;
    PyObject* d = PyObject_GetAttr(x, s_dtype);
    if (!d) return -1;
    const int ok = is_type(y, d);
    Py_DECREF(d);
    if (ok < 0) return -1;
    if (ok && ys[0] == xs[0] && ys[1] == xs[1] && ys[2] == xs[2]) return 0;
    PyErr_SetString(PyExc_ValueError, what);
    return -1;
}

/* scored(q, k_cache, v_cache, desc, block_tables, seq_lens, max_seq_len, scale, out, score, weights, new_lens, workspace,
 *        partition_tokens, q_dtype, stream) */
static PyObject* py_scored(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    pkv_score_mod m;
    int32_t type, qs[3], ts[2], max_len, part;
    void *q, *kc, *vc, *tables, *lens, *out, *w, *fresh, *ws, *st;
    size_t wn;
    long dev;
    if (!nargs_ok(n, 16)) return NULL;
    if (get_desc(a[3], &c) || batch_ok(a[0], a[4], a[5], &c, qs, ts) ||
        alike3(a[0], qs, a[8], "out", "out must have q's shape and type"))
        return NULL;
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    if (as_i32(a[6], &max_len) || as_i32(a[13], &part) || element_type(a[0], a[14], &type) || ptr_of(a[0], "q", -1, &q) ||
        current_device(&dev) || ptr_of(a[0], "q", dev, &q) || pool_size(a[1], &c, "k_cache") ||
        pool_size(a[2], &c, "v_cache") || ptr_of(a[1], "k_cache", dev, &kc) || ptr_of(a[2], "v_cache", dev, &vc) ||
        ptr_of(a[4], "block_tables", dev, &tables) || ptr_of(a[5], "seq_lens", dev, &lens) ||
        ptr_of(a[8], "out", dev, &out) || get_score(a[9], qs[1], qs[0], qs[0], dev, 1, &m) ||
        weights_of(a[10], &c, dev, &w) || optional_vector(a[11], t_i32, qs[0], "new_lens", "int32", dev, &fresh) ||
        workspace_of(a[12], dev, &ws, &wn) || stream_of(a[15], &st))
        return NULL;
    DONE(fn.scored(q, type, qs[0], qs[1], kc, vc, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens, max_len,
                   (float)scale, &m, (float*)w, (const int32_t*)fresh, out, ws, wn, part, st));
}

/* prefill_scored(q, k_cache, v_cache, desc, query_start, max_query_len, block_tables, seq_lens, scale, out, score,
 *                work_units, workspace, q_dtype, stream) */
static PyObject* py_prefill_scored(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    pkv_score_mod m;
    int32_t type, qs[3], ts[2], S[1], starts[1], most, units[1] = {0};
    void *q, *kc, *vc, *start, *tables, *lens, *out, *work = NULL, *ws, *st;
    size_t wn;
    long dev;
    if (!nargs_ok(n, 15)) return NULL;
    static const char ints[] = "query_start, block_tables, seq_lens and work_units";
    if (get_desc(a[3], &c) || want_i32(a[4], ints) || want_i32(a[6], ints) || want_i32(a[7], ints) ||
        (a[11] != Py_None && (want_i32(a[11], ints) || dims(a[11], "work_units", 1, units))) || dims(a[0], "q", 3, qs) ||
        same(qs[2], c.head_size, "q must have the cache's head_size") || bytes16(a[0], (size_t)qs[0] * qs[1] * qs[2], "q") ||
        alike3(a[0], qs, a[9], "out", "out must have q's shape and type") || dims(a[7], "seq_lens", 1, S) ||
        dims(a[4], "query_start", 1, starts) ||
        same(starts[0] - 1, S[0], "query_start must have num_seqs + 1 entries") || dims(a[6], "block_tables", 2, ts) ||
        same(ts[0], S[0], "block_tables and seq_lens must have one row per sequence") || as_i32(a[5], &most) ||
        pool_size(a[1], &c, "k_cache") || pool_size(a[2], &c, "v_cache") || element_type(a[0], a[13], &type) ||
        get_score(a[10], qs[1], qs[0], S[0], -1, 0, &m))
        return NULL;
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    if (ptr_of(a[0], "q", -1, &q) || current_device(&dev) || ptr_of(a[0], "q", dev, &q) ||
        ptr_of(a[1], "k_cache", dev, &kc) || ptr_of(a[2], "v_cache", dev, &vc) || ptr_of(a[4], "query_start", dev, &start) ||
        ptr_of(a[6], "block_tables", dev, &tables) || ptr_of(a[7], "seq_lens", dev, &lens) ||
        ptr_of(a[9], "out", dev, &out) || get_score(a[10], qs[1], qs[0], S[0], dev, 1, &m) ||
        (units[0] > 0 && ptr_of(a[11], "work_units", dev, &work)) || workspace_of(a[12], dev, &ws, &wn) ||
        stream_of(a[14], &st))
        return NULL;
    DONE(fn.prefill(q, type, qs[0], qs[1], S[0], (const int32_t*)start, most, kc, vc, &c, (const int32_t*)tables, ts[1],
                    (const int32_t*)lens, (const int32_t*)work, units[0], (float)scale, &m, out, ws, wn, st));
}

/* A 16-bit tensor [n, heads, D] (heads < 0: any number, returned) whose tokens may lie apart: pointer and elements from
 * one token to the next.  dev: its device, set by the first call (-1) and demanded by later ones. */
static int token_rows(PyObject* t, const char* name, PyObject* type_of, int32_t n, int32_t D, long* dev, int32_t* heads,
                      void** p, int64_t* step) {
    int32_t ts[3];
    if (dims(t, name, 3, ts)) return -1;
    PyObject* d = PyObject_GetAttr(type_of, s_dtype);
    if (!d) return -1;
    const int ok = is_type(t, d);
    Py_DECREF(d);
    if (ok < 0) return -1;
    if (!ok || ts[0] != n || ts[2] != D || (*heads >= 0 && ts[1] != *heads)) {
        PyErr_Format(PyExc_ValueError, "%s must have one type with k and a row of heads of %d elements for each of %d tokens",
                     name, D, n);
        return -1;
    }
    *heads = ts[1];
    PyObject* r = PyObject_CallMethodNoArgs(t, s_stride);
    if (!r) return -1;
    long long at[3] = {0, 0, 0};
    int good = PyTuple_Check(r) && PyTuple_GET_SIZE(r) == 3;
    for (int i = 0; i < 3 && good; ++i) {
        at[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(r, i));
        good = !(at[i] == -1 && PyErr_Occurred());
    }
    Py_DECREF(r);
    if (PyErr_Occurred()) return -1;
    /* sizes of one have any stride */
    if (!good || (at[2] != 1 && ts[2] > 1) || (at[1] != D && ts[1] > 1)) {
        PyErr_Format(PyExc_ValueError, "%s must have a token's heads side by side", name);
        return -1;
    }
    *step = ts[0] > 1 ? at[0] : (int64_t)ts[1] * D;
    r = PyObject_CallMethodNoArgs(t, s_get_device);
    const long on = r ? PyLong_AsLong(r) : -1;
    Py_XDECREF(r);
    if (on < 0) {
        PyErr_Clear();
        PyErr_Format(PyExc_TypeError, "%s must be a CUDA tensor", name);
        return -1;
    }
    if (*dev < 0) {
        if (current_device(dev)) return -1;
    }
    if (on != *dev) {
        PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the current device is cuda:%ld", name, on, *dev);
        return -1;
    }
    r = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!r) return -1;
    *p = PyLong_AsVoidPtr(r);
    Py_DECREF(r);
    return PyErr_Occurred() ? -1 : 0;
}

/* rope(q, k, v, positions, slot_mapping, freqs, k_cache, v_cache, desc, q_out, interleaved, magnitude, stream) */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t type, T[1], fs[2], Hq = 0, Hk, Hv;
    void *q = NULL, *k, *v, *pos, *slots, *freqs, *kc, *vc, *o = NULL, *st;
    int64_t qstep = 0, kstep, vstep, ostep = 0;
    long dev = -1;
    if (!nargs_ok(n, 13)) return NULL;
    if (get_desc(a[8], &c) || dims(a[4], "slot_mapping", 1, T) || dims(a[5], "freqs", 2, fs)) return NULL;
    int ok = is_type(a[4], t_i64);
    if (ok < 0) return NULL;
    if (!ok) {
        PyErr_SetString(PyExc_TypeError, "slot_mapping must be int64");
        return NULL;
    }
    ok = is_type(a[5], t_f32);
    if (ok < 0) return NULL;
    if (!ok || fs[1] != 2) {
        PyErr_SetString(PyExc_ValueError, "freqs must be float32 [rotary_dim / 2, 2]");
        return NULL;
    }
    const double magnitude = PyFloat_AsDouble(a[11]);
    if (magnitude == -1.0 && PyErr_Occurred()) return NULL;
    const int inter = PyObject_IsTrue(a[10]);
    if (inter < 0 || element_type(a[1], Py_None, &type)) return NULL;
    if ((a[0] == Py_None) != (a[9] == Py_None)) {
        PyErr_SetString(PyExc_ValueError, "q and q_out go together");
        return NULL;
    }
    if (a[3] == Py_None) {
        PyErr_SetString(PyExc_TypeError, "positions must be int32");
        return NULL;
    }
    Hk = Hv = c.num_kv_heads;
    if (Hk < 0 || fs[0] > INT32_MAX / 2) {
        PyErr_SetString(PyExc_ValueError, "sizes out of range");
        return NULL;
    }
    if (token_rows(a[1], "k", a[1], T[0], c.head_size, &dev, &Hk, &k, &kstep) ||
        token_rows(a[2], "v", a[1], T[0], c.head_size, &dev, &Hv, &v, &vstep))
        return NULL;
    if (a[0] != Py_None) {
        Hq = -1;
        if (token_rows(a[0], "q", a[1], T[0], c.head_size, &dev, &Hq, &q, &qstep) ||
            token_rows(a[9], "q_out", a[1], T[0], c.head_size, &dev, &Hq, &o, &ostep))
            return NULL;
    }
    if (optional_vector(a[3], t_i32, T[0], "positions", "int32", dev, &pos) ||
        ptr_of(a[4], "slot_mapping", dev, &slots) || ptr_of(a[5], "freqs", dev, &freqs) ||
        pool_size(a[6], &c, "k_cache") || pool_size(a[7], &c, "v_cache") || ptr_of(a[6], "k_cache", dev, &kc) ||
        ptr_of(a[7], "v_cache", dev, &vc) || stream_of(a[12], &st))
        return NULL;
    DONE(fn.rope(q, qstep, Hq, k, kstep, v, vstep, type, T[0], (const int32_t*)pos, (const int64_t*)slots,
                 (const float*)freqs, 2 * fs[0], inter, (float)magnitude, kc, vc, &c, o, ostep, st));
}

/* kept [S, Hkv, n], block_tables [S, MB] and seq_lens [S] of an eviction. */
static int kept_ok(PyObject* kept, PyObject* tables, PyObject* lens, const pkv_cache_desc* c, int32_t* ks, int32_t* ts) {
    int32_t S[1];
    if (want_i32(kept, "kept, block_tables and seq_lens") || want_i32(tables, "kept, block_tables and seq_lens") ||
        want_i32(lens, "kept, block_tables and seq_lens") || dims(kept, "kept", 3, ks) ||
        dims(tables, "block_tables", 2, ts) || dims(lens, "seq_lens", 1, S) ||
        same(ks[1], c->num_kv_heads, "kept must have shape [num_seqs, num_kv_heads, n]") ||
        same(ks[0], S[0], "kept must have shape [num_seqs, num_kv_heads, n]") ||
        same(ts[0], S[0], "block_tables must have one row per sequence"))
        return -1;
    return 0;
}

/* select_tokens(weights, desc, block_tables, seq_lens, max_seq_len, kept, sink_tokens, recent_tokens, stream) */
static PyObject* py_select_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t ks[3], ts[2], max_len, sink, recent;
    void *w, *tables, *lens, *kept, *st;
    long dev;
    if (!nargs_ok(n, 9)) return NULL;
    if (get_desc(a[1], &c) || kept_ok(a[5], a[2], a[3], &c, ks, ts) || as_i32(a[4], &max_len) || as_i32(a[6], &sink) ||
        as_i32(a[7], &recent))
        return NULL;
    if (a[0] == Py_None) {
        PyErr_SetString(PyExc_TypeError, "weights must be a CUDA tensor");
        return NULL;
    }
    if (ptr_of(a[5], "kept", -1, &kept) || current_device(&dev) || ptr_of(a[5], "kept", dev, &kept) ||
        weights_of(a[0], &c, dev, &w) || ptr_of(a[2], "block_tables", dev, &tables) ||
        ptr_of(a[3], "seq_lens", dev, &lens) || stream_of(a[8], &st))
        return NULL;
    DONE(fn.select_tokens((const float*)w, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens, max_len, ks[0], ks[2],
                          sink, recent, (int32_t*)kept, st));
}

/* compact(kept, k_cache, v_cache, desc, block_tables, seq_lens, dst_tables, weights, stream) */
static PyObject* py_compact(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    pkv_cache_desc c;
    int32_t ks[3], ts[2], ds[2];
    void *w, *tables, *lens, *kept, *dst, *kc, *vc, *st;
    long dev;
    if (!nargs_ok(n, 9)) return NULL;
    if (get_desc(a[3], &c) || kept_ok(a[0], a[4], a[5], &c, ks, ts) || want_i32(a[6], "dst_tables") ||
        dims(a[6], "dst_tables", 2, ds) || same(ds[0], ks[0], "dst_tables must have one row per sequence"))
        return NULL;
    if (ptr_of(a[0], "kept", -1, &kept) || current_device(&dev) || ptr_of(a[0], "kept", dev, &kept) ||
        pool_size(a[1], &c, "k_cache") || pool_size(a[2], &c, "v_cache") || ptr_of(a[1], "k_cache", dev, &kc) ||
        ptr_of(a[2], "v_cache", dev, &vc) || ptr_of(a[4], "block_tables", dev, &tables) ||
        ptr_of(a[5], "seq_lens", dev, &lens) || ptr_of(a[6], "dst_tables", dev, &dst) ||
        weights_of(a[7], &c, dev, &w) || stream_of(a[8], &st))
        return NULL;
    DONE(fn.compact((const int32_t*)kept, ks[2], kc, vc, (float*)w, &c, (const int32_t*)tables, ts[1], (const int32_t*)lens,
                    ks[0], (const int32_t*)dst, ds[1], st));
}

static int address(PyObject* map, const char* name, void* slot) {
    PyObject* a = PyDict_GetItemString(map, name);
    void* p = a ? PyLong_AsVoidPtr(a) : NULL;
    if (!p) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_KeyError, "%s", name);
        return -1;
    }
    memcpy(slot, &p, sizeof p);
    return 0;
}

/* bind(torch, addresses, stream): addresses of the C ABI by name; stream(s) gives a stream's handle. */
static PyObject* py_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (!nargs_ok(n, 3)) return NULL;
    PyObject* c = PyObject_GetAttrString(a[0], "_C");
    if (!c) return NULL;
    struct {
        PyObject** to;
        PyObject* from;
        const char* name;
    } keep[] = {{&t_i32, a[0], "int32"},    {&t_i64, a[0], "int64"},          {&t_f16, a[0], "float16"},
                {&t_bf16, a[0], "bfloat16"}, {&t_f32, a[0], "float32"}, {&f_device, c, "_cuda_getDevice"}, {&f_raw_stream, c, "_cuda_getCurrentRawStream"}};
    for (size_t i = 0; i < sizeof keep / sizeof keep[0]; ++i) {
        PyObject* v = PyObject_GetAttrString(keep[i].from, keep[i].name);
        if (!v && keep[i].from == c) {  /* a torch without CUDA: no call gets as far as needing it */
            PyErr_Clear();
            v = Py_NewRef(Py_None);
        }
        if (!v) {
            Py_DECREF(c);
            return NULL;
        }
        Py_XSETREF(*keep[i].to, v);
    }
    Py_DECREF(c);
    Py_XSETREF(f_stream, Py_NewRef(a[2]));
    if (address(a[1], "pkv_paged_kv_append", &fn.append) || address(a[1], "pkv_paged_kv_read", &fn.read) ||
        address(a[1], "pkv_paged_attention_decode", &fn.decode) || address(a[1], "pkv_paged_key_bounds", &fn.bounds) ||
        address(a[1], "pkv_select_blocks", &fn.select) ||
        address(a[1], "pkv_paged_attention_decode_sparse", &fn.sparse) ||
        address(a[1], "pkv_paged_attention_decode_scored", &fn.scored) ||
        address(a[1], "pkv_paged_attention_prefill_scored", &fn.prefill) ||
        address(a[1], "pkv_paged_rope_append", &fn.rope) || address(a[1], "pkv_select_tokens", &fn.select_tokens) ||
        address(a[1], "pkv_paged_kv_compact", &fn.compact) ||
        address(a[1], "pkv_cache_block_bytes", &fn.block_bytes))
        return NULL;
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind),   METHOD(append), METHOD(read),   METHOD(decode),
                                METHOD(bounds), METHOD(select), METHOD(sparse), METHOD(scored), METHOD(rope),
                                METHOD(select_tokens), METHOD(compact), METHOD(prefill_scored),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pkv_binding(void) {
    static const struct {
        PyObject** to;
        const char* name;
    } names[] = {{&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"},
                 {&s_shape, "shape"},           {&s_dtype, "dtype"},                 {&s_nbytes, "nbytes"},
                 {&s_num_blocks, "num_blocks"}, {&s_block_size, "block_size"},       {&s_num_kv_heads, "num_kv_heads"},
                 {&s_head_size, "head_size"},   {&s_kv_dtype, "kv_dtype"},           {&s_k_scale, "k_scale"},
                 {&s_v_scale, "v_scale"},       {&s_cap, "cap"},                     {&s_window, "window"},
                 {&s_slopes, "slopes"},         {&s_first, "first"},                 {&s_prefix_lens, "prefix_lens"},
                 {&s_stride, "stride"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
