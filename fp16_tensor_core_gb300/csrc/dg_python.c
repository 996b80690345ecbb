/* dg_python.c -- argument marshalling of the serving entry points (rotary
 * positions, cache writes and reads, attention) for Python.
 *
 * A decode step makes these calls for every layer and token, with kernels of
 * 2 to 10 us: read attribute by attribute in Python and handed over through
 * ctypes, the arguments take longer than the launch (a cache write 8.4 us,
 * 5.3 of them the arguments; 4.4 us here).  The functions here take the
 * tensors as they are, by position; the package's Python functions give them
 * their names, defaults and documentation.  Nothing here knows PyTorch's headers: tensors
 * are read through their Python attributes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <math.h>
#include <stdint.h>

#include "dg.h"

/* From bind(): the library's functions, and what the package knows of torch. */
static dg_status (*lib_rope)(const dg_heads*, const dg_heads*, int64_t, int, int, const int32_t*,
                             const dg_rotary*, int, dg_dtype, dg_stream_t);
static dg_status (*lib_kv_append)(const dg_heads*, const dg_heads*, int, const dg_heads*, const dg_heads*,
                                  int64_t, const int32_t*, const dg_rotary*, const int32_t*,
                                  const dg_kv_cache*, dg_dtype, dg_stream_t);
static dg_status (*lib_kv_read)(const dg_kv_cache*, const int32_t*, int64_t, const dg_heads*, const dg_heads*,
                                dg_dtype, dg_stream_t);
static dg_status (*lib_attn_decode)(const dg_heads*, const dg_heads*, float*, int, int, int, const dg_kv_cache*,
                                    const int32_t*, int64_t, int64_t, const int32_t*, const int32_t*, int64_t,
                                    double, dg_dtype, void*, int64_t, dg_stream_t);
static PyObject *type_bf16, *type_fp16, *type_int32, *type_float32;   /* torch.dtype objects */
static PyObject *current_stream;   /* (device) -> handle of its current stream */
static PyObject *current_device;   /* () -> index */
static PyObject *check;            /* (status, name): raises unless DG_OK */

static PyObject *n_stride, *n_shape, *n_dtype, *n_is_cuda, *n_data_ptr, *n_numel, *n_is_contiguous, *n_nbytes,
    *n_rotary, *n_cache, *n_cuda_stream;

static int fail(const char* message) {
    PyErr_SetString(PyExc_ValueError, message);
    return -1;
}

static int fail_about(const char* what, const char* message) {
    PyErr_Format(PyExc_ValueError, "%s %s", what, message);
    return -1;
}

static int as_int64(PyObject* v, int64_t* out) {   /* takes the reference */
    if (v == NULL) return -1;
    *out = PyLong_AsLongLong(v);
    Py_DECREF(v);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int as_address(PyObject* v, void** out) {   /* takes the reference */
    if (v == NULL) return -1;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* Whether an attribute or method result is the object `want`; -1: an error. */
static int is_object(PyObject* v, PyObject* want) {   /* takes the reference */
    if (v == NULL) return -1;
    const int same = v == want;
    Py_DECREF(v);
    return same;
}

static int on_device(PyObject* t) {
    const int yes = is_object(PyObject_GetAttr(t, n_is_cuda), Py_True);
    return yes == 0 ? fail("tensor must be in CUDA device memory") : yes < 0 ? -1 : 0;
}

/* A tuple's first n numbers (exactly n entries wanted). */
static int numbers(PyObject* tuple, Py_ssize_t n, int64_t* out, const char* what,
                   const char* message) {   /* takes the reference */
    if (tuple == NULL) return -1;
    int rc = PyTuple_Check(tuple) && PyTuple_GET_SIZE(tuple) == n ? 0 : fail_about(what, message);
    for (Py_ssize_t i = 0; rc == 0 && i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
        if (out[i] == -1 && PyErr_Occurred()) rc = -1;
    }
    Py_DECREF(tuple);
    return rc;
}

typedef struct {
    dg_heads c;
    int64_t shape[3];
    dg_dtype type;
} heads_arg;

/* [tokens, heads, head_dim] BF16 or FP16, any token and head stride. */
static int get_heads(PyObject* t, const char* what, const heads_arg* like, heads_arg* h) {
    static const char kWanted[] = "must be BF16 or FP16 [tokens, heads, head_dim] with contiguous heads";
    int64_t stride[3];
    if (numbers(PyObject_CallMethodNoArgs(t, n_stride), 3, stride, what, kWanted) < 0 ||
        numbers(PyObject_GetAttr(t, n_shape), 3, h->shape, what, kWanted) < 0)
        return -1;
    PyObject* type = PyObject_GetAttr(t, n_dtype);
    if (type == NULL) return -1;
    const int bf16 = type == type_bf16, fp16 = type == type_fp16;
    Py_DECREF(type);
    if (!(bf16 || fp16) || (stride[2] != 1 && h->shape[2] > 1)) return fail_about(what, kWanted);
    h->type = bf16 ? DG_BF16 : DG_FP16;
    if (like != NULL && (h->type != like->type || h->shape[0] != like->shape[0] || h->shape[1] != like->shape[1] ||
                         h->shape[2] != like->shape[2]))
        return fail_about(what, "must have the shape and type of its counterpart");
    void* data;
    if (on_device(t) < 0 || as_address(PyObject_CallMethodNoArgs(t, n_data_ptr), &data) < 0) return -1;
    h->c.data = data;
    h->c.token_stride = h->shape[0] > 1 ? stride[0] : 0;   /* a single one's stride may be anything */
    h->c.head_stride = h->shape[1] > 1 ? stride[1] : 0;
    return 0;
}

/* Address of a contiguous device tensor. */
static int get_data(PyObject* t, void** out) {
    if (on_device(t) < 0) return -1;
    const int yes = is_object(PyObject_CallMethodNoArgs(t, n_is_contiguous), Py_True);
    if (yes <= 0) return yes < 0 ? -1 : fail("tensor must be contiguous");
    return as_address(PyObject_CallMethodNoArgs(t, n_data_ptr), out);
}

/* Address of a tensor of n elements of a type (n < 0: any number). */
static int get_array(PyObject* t, PyObject* type, const char* type_name, int64_t n, const char* what, void** out) {
    int64_t have = 0;
    const int yes = is_object(PyObject_GetAttr(t, n_dtype), type);
    if (yes < 0 || as_int64(PyObject_CallMethodNoArgs(t, n_numel), &have) < 0) return -1;
    if (!yes || (n >= 0 && have != n)) {
        PyErr_Format(PyExc_ValueError, "%s must be %s with %lld elements", what, type_name,
                     (long long)(n < 0 ? have : n));
        return -1;
    }
    return get_data(t, out);
}

/* The struct that a DgRotary or DgKvCache holds. */
static int get_rotary(PyObject* handle, void** out) { return as_address(PyObject_GetAttr(handle, n_rotary), out); }
static int get_cache(PyObject* handle, void** out) { return as_address(PyObject_GetAttr(handle, n_cache), out); }

/* None: the current device's current stream; else a handle or a Stream. */
static int get_stream(PyObject* s, dg_stream_t* out) {
    void* p = NULL;
    int rc;
    if (s == Py_None) {
        PyObject* device = PyObject_CallNoArgs(current_device);
        if (device == NULL) return -1;
        rc = as_address(PyObject_CallOneArg(current_stream, device), &p);
        Py_DECREF(device);
    } else {
        rc = as_address(PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttr(s, n_cuda_stream), &p);
    }
    *out = (dg_stream_t)p;
    return rc;
}

static int want_args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments wanted, %zd given", want, n);
    return -1;
}

static PyObject* done(dg_status status, const char* name) {
    if (status == DG_OK) Py_RETURN_NONE;
    return PyObject_CallFunction(check, "is", (int)status, name);
}

static int to_int(int64_t v) { return v > INT32_MAX ? INT32_MAX : v < INT32_MIN ? INT32_MIN : (int)v; }

/* (x, out, positions, rotary, inverse, stream) */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    heads_arg x, out;
    void *positions, *rotary;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 6) < 0 || get_heads(a[0], "x", NULL, &x) < 0 || get_heads(a[1], "out", &x, &out) < 0 ||
        get_array(a[2], type_int32, "int32", x.shape[0], "positions", &positions) < 0 ||
        get_rotary(a[3], &rotary) < 0)
        return NULL;
    const int inverse = PyObject_IsTrue(a[4]);
    if (inverse < 0 || get_stream(a[5], &stream) < 0) return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_rope(&x.c, &out.c, x.shape[0], to_int(x.shape[1]), to_int(x.shape[2]), positions, rotary, inverse,
                      x.type, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_rope");
}

static int cache_heads(const heads_arg* h, const dg_kv_cache* cache) {
    return h->shape[1] == cache->kv_heads && h->shape[2] == cache->head_dim
               ? 0
               : fail("k and v must have the cache's heads and head_dim");
}

/* (k, v, slots, cache, positions, rotary, q, q_out, stream) */
static PyObject* py_kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    heads_arg k, v, q, q_out;
    void *slots, *cache, *positions = NULL, *rotary = NULL;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 9) < 0 || get_heads(a[0], "k", NULL, &k) < 0 || get_heads(a[1], "v", &k, &v) < 0 ||
        get_cache(a[3], &cache) < 0 || cache_heads(&k, cache) < 0)
        return NULL;
    const int queries = a[6] != Py_None;
    if (queries != (a[7] != Py_None)) {
        fail("q and q_out must be given together");
        return NULL;
    }
    if (queries) {
        if (get_heads(a[6], "q", NULL, &q) < 0 || get_heads(a[7], "q_out", &q, &q_out) < 0) return NULL;
        if (q.shape[0] != k.shape[0] || q.shape[2] != k.shape[2] || q.type != k.type) {
            fail("q must have the tokens, head_dim and type of k");
            return NULL;
        }
    }
    if ((a[4] != Py_None && get_array(a[4], type_int32, "int32", k.shape[0], "positions", &positions) < 0) ||
        (a[5] != Py_None && get_rotary(a[5], &rotary) < 0) ||
        get_array(a[2], type_int32, "int32", k.shape[0], "slots", &slots) < 0 || get_stream(a[8], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_kv_append(queries ? &q.c : NULL, queries ? &q_out.c : NULL, queries ? to_int(q.shape[1]) : 0, &k.c,
                           &v.c, k.shape[0], positions, rotary, slots, cache, k.type, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_kv_append");
}

/* (cache, slots, k, v, stream), k and v not both None */
static PyObject* py_kv_read(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    heads_arg k, v;
    void *cache, *slots;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 5) < 0) return NULL;
    const int keys = a[2] != Py_None, values = a[3] != Py_None;
    const heads_arg* some = keys ? &k : &v;
    if ((keys && get_heads(a[2], "k", NULL, &k) < 0) ||
        ((values || !keys) && get_heads(a[3], "v", keys ? &k : NULL, &v) < 0) || get_cache(a[0], &cache) < 0 ||
        cache_heads(some, cache) < 0 ||
        get_array(a[1], type_int32, "int32", some->shape[0], "slots", &slots) < 0 || get_stream(a[4], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_kv_read(cache, slots, some->shape[0], keys ? &k.c : NULL, values ? &v.c : NULL, some->type, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_kv_read");
}

/* (q, out, cache, page_table, kv_lens, scratch, scale, lse, prefix_pages, prefix_len, stream) */
static PyObject* py_attn_decode(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    static const char kTable[] = "must have the cache's head_dim, page_table must be int32 with contiguous rows";
    heads_arg q, out;
    void *handle, *table, *lens, *scratch, *lse = NULL, *prefix = NULL;
    int64_t shape[2], stride[2], scratch_bytes, prefix_len = 0;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 11) < 0 || (a[9] != Py_None && as_int64(Py_NewRef(a[9]), &prefix_len) < 0)) return NULL;
    if (a[8] == Py_None ? prefix_len != 0 : a[9] == Py_None) {   /* a length of 0 is no prefix, pages or not */
        fail("prefix_pages and prefix_len must be given together");
        return NULL;
    }
    if (get_heads(a[0], "q", NULL, &q) < 0 || get_heads(a[1], "out", &q, &out) < 0 ||
        get_cache(a[2], &handle) < 0 || numbers(PyObject_GetAttr(a[3], n_shape), 2, shape, "q", kTable) < 0 ||
        numbers(PyObject_CallMethodNoArgs(a[3], n_stride), 2, stride, "q", kTable) < 0)
        return NULL;
    const dg_kv_cache* cache = handle;
    const int64_t tokens = q.shape[0], batch = shape[0], pages = shape[1];
    const int typed = is_object(PyObject_GetAttr(a[3], n_dtype), type_int32);
    const int there = typed < 0 ? -1 : is_object(PyObject_GetAttr(a[3], n_is_cuda), Py_True);
    if (there < 0) return NULL;
    if (q.shape[2] != cache->head_dim || !typed || !there || (pages > 1 && stride[1] != 1)) {
        fail_about("q", kTable);
        return NULL;
    }
    if (batch > 1 && stride[0] < pages) {   /* rows that share entries: an expanded table, overlapping windows */
        fail("page_table must have a row of its own for each request");
        return NULL;
    }
    if (batch != 0 ? tokens % batch != 0 : tokens != 0) {
        fail("q must have the same number of tokens for each request");
        return NULL;
    }
    if (as_address(PyObject_CallMethodNoArgs(a[3], n_data_ptr), &table) < 0 ||
        get_array(a[4], type_int32, "int32", batch, "kv_lens", &lens) < 0 || get_data(a[5], &scratch) < 0 ||
        as_int64(PyObject_GetAttr(a[5], n_nbytes), &scratch_bytes) < 0)
        return NULL;
    double scale;
    if (a[6] == Py_None) {
        scale = pow((double)q.shape[2], -0.5);
    } else {
        scale = PyFloat_AsDouble(a[6]);
        if (scale == -1.0 && PyErr_Occurred()) return NULL;
    }
    if (a[7] != Py_None && get_array(a[7], type_float32, "FP32", tokens * q.shape[1], "lse", &lse) < 0) return NULL;
    if (prefix_len != 0) {
        int64_t named;
        if (get_array(a[8], type_int32, "int32", -1, "prefix_pages", &prefix) < 0 ||
            as_int64(PyObject_CallMethodNoArgs(a[8], n_numel), &named) < 0)
            return NULL;
        if (prefix_len > 0 && cache->page_size > 0 && named < (prefix_len - 1) / cache->page_size + 1) {
            fail("prefix_pages must name every page of the prefix");
            return NULL;
        }
    }
    if (get_stream(a[10], &stream) < 0) return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_attn_decode(&q.c, &out.c, lse, to_int(batch), to_int(batch != 0 ? tokens / batch : 1),
                             to_int(q.shape[1]), cache, table, batch > 1 ? stride[0] : pages, pages, lens,
                             prefix, prefix_len, scale, q.type, scratch, scratch_bytes, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_attn_decode");
}

/* (addresses of dg_rope, dg_kv_append, dg_kv_read, dg_attn_decode; torch's
 * bfloat16, float16, int32, float32; current_stream; current_device; check) */
static PyObject* py_bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* f[4];
    (void)self;
    if (want_args(n, 11) < 0) return NULL;
    for (int i = 0; i < 4; ++i)
        if (as_address(Py_NewRef(a[i]), &f[i]) < 0) return NULL;
    *(void**)&lib_rope = f[0];
    *(void**)&lib_kv_append = f[1];
    *(void**)&lib_kv_read = f[2];
    *(void**)&lib_attn_decode = f[3];
    PyObject** keep[] = {&type_bf16, &type_fp16, &type_int32, &type_float32, &current_stream, &current_device, &check};
    for (int i = 0; i < 7; ++i) Py_XSETREF(*keep[i], Py_NewRef(a[4 + i]));
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL, NULL},
    {"rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, NULL},
    {"kv_append", (PyCFunction)(void (*)(void))py_kv_append, METH_FASTCALL, NULL},
    {"kv_read", (PyCFunction)(void (*)(void))py_kv_read, METH_FASTCALL, NULL},
    {"attn_decode", (PyCFunction)(void (*)(void))py_attn_decode, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "dg_python", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_dg_python(void) {
    static const struct {
        PyObject** at;
        const char* name;
    } names[] = {
        {&n_stride, "stride"}, {&n_shape, "shape"}, {&n_dtype, "dtype"}, {&n_is_cuda, "is_cuda"},
        {&n_data_ptr, "data_ptr"}, {&n_numel, "numel"}, {&n_is_contiguous, "is_contiguous"}, {&n_nbytes, "nbytes"},
        {&n_rotary, "rotary_address"}, {&n_cache, "cache_address"}, {&n_cuda_stream, "cuda_stream"},
    };
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if (*names[i].at == NULL && (*names[i].at = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
    return PyModule_Create(&module);
}
