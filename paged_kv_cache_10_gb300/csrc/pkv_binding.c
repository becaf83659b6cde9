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
    size_t (*block_bytes)(const pkv_cache_desc*);
} fn;

/* Objects of torch that bind() keeps. */
static PyObject *t_i32, *t_i64, *t_f16, *t_bf16, *f_device, *f_raw_stream, *f_stream;
/* Attribute and method names. */
static PyObject *s_get_device, *s_is_contiguous, *s_data_ptr, *s_shape, *s_dtype, *s_nbytes, *s_num_blocks,
    *s_block_size, *s_num_kv_heads, *s_head_size, *s_kv_dtype, *s_k_scale, *s_v_scale;

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
                {&t_bf16, a[0], "bfloat16"}, {&f_device, c, "_cuda_getDevice"}, {&f_raw_stream, c, "_cuda_getCurrentRawStream"}};
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
        address(a[1], "pkv_cache_block_bytes", &fn.block_bytes))
        return NULL;
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(bind),   METHOD(append), METHOD(read),   METHOD(decode),
                                METHOD(bounds), METHOD(select), METHOD(sparse), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pkv_binding(void) {
    static const struct {
        PyObject** to;
        const char* name;
    } names[] = {{&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"},
                 {&s_shape, "shape"},           {&s_dtype, "dtype"},                 {&s_nbytes, "nbytes"},
                 {&s_num_blocks, "num_blocks"}, {&s_block_size, "block_size"},       {&s_num_kv_heads, "num_kv_heads"},
                 {&s_head_size, "head_size"},   {&s_kv_dtype, "kv_dtype"},           {&s_k_scale, "k_scale"},
                 {&s_v_scale, "v_scale"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
