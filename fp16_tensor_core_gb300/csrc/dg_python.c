/* dg_python.c -- argument marshalling of the serving entry points (rotary
 * positions, cache writes and reads, attention) and of those around a layer's
 * products (norm, activation, fused products) for Python.
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
static dg_status (*lib_rmsnorm)(const dg_rows*, const dg_rows*, const dg_rows*, const void*, int64_t, int64_t,
                                double, dg_dtype, const dg_rows*, dg_stream_t);
static dg_status (*lib_rmsnorm_e4m3)(const dg_rows*, const dg_rows*, const dg_rows*, const void*, int64_t, int64_t,
                                     double, dg_dtype, uint8_t*, float*, dg_stream_t);
static dg_status (*lib_rmsnorm_e4m3_amax)(const dg_rows*, const dg_rows*, const dg_rows*, const void*, int64_t,
                                          int64_t, double, dg_dtype, const float*, uint8_t*, float*, float*,
                                          dg_stream_t);
static dg_status (*lib_rmsnorm_grad)(const dg_rows*, const void*, const dg_rows*, const dg_rows*, int64_t, int64_t,
                                     double, dg_dtype, const dg_rows*, float*, void*, int64_t, dg_stream_t);
static dg_status (*lib_activate)(const dg_rows*, int, dg_activation, int64_t, int64_t, dg_dtype, const dg_rows*,
                                 uint8_t*, float*, uint8_t*, float*, dg_stream_t);
static dg_status (*lib_activate_grad)(const dg_rows*, const dg_rows*, const uint8_t*, const float*, int,
                                      dg_activation, int64_t, int64_t, dg_dtype, const dg_rows*, float*, void*,
                                      int64_t, dg_stream_t);
static dg_status (*lib_fp8_gemm_fused)(const uint8_t*, const uint8_t*, void*, int64_t, int64_t, int64_t,
                                       const dg_epilogue*, dg_dtype, dg_stream_t);
static dg_status (*lib_hgemm_fused)(const uint16_t*, const uint16_t*, void*, int64_t, int64_t, int64_t,
                                    const dg_epilogue*, dg_dtype, dg_stream_t);
static PyObject *type_bf16, *type_fp16, *type_int32, *type_float32, *type_uint8;   /* torch.dtype objects */
static PyObject *current_stream;   /* (device) -> handle of its current stream */
static PyObject *current_device;   /* () -> index */
static PyObject *check;            /* (status, name): raises unless DG_OK */

static PyObject *n_stride, *n_shape, *n_dtype, *n_is_cuda, *n_data_ptr, *n_numel, *n_is_contiguous, *n_nbytes,
    *n_rotary, *n_cache, *n_cuda_stream, *n_get_device;

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

/* Whether a tensor is on the current device, where the library launches: for
 * the calls around a layer's products (one attribute serves as well as
 * is_cuda).  *current is the device's index once it has been asked for, -1
 * before. */
static int on_current_device(PyObject* t, int64_t* current) {
    int64_t device;
    if (as_int64(PyObject_CallMethodNoArgs(t, n_get_device), &device) < 0) return -1;
    if (device < 0) return fail("tensor must be in CUDA device memory");
    if (*current < 0 && as_int64(PyObject_CallNoArgs(current_device), current) < 0) return -1;
    return device == *current ? 0 : fail("tensor must be on the current device");
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

/* Address of a contiguous tensor on the current device. */
static int get_data_here(PyObject* t, int64_t* device, void** out) {
    if (on_current_device(t, device) < 0) return -1;
    const int yes = is_object(PyObject_CallMethodNoArgs(t, n_is_contiguous), Py_True);
    if (yes <= 0) return yes < 0 ? -1 : fail("tensor must be contiguous");
    return as_address(PyObject_CallMethodNoArgs(t, n_data_ptr), out);
}

/* Of n elements of a type. */
static int get_array_here(PyObject* t, PyObject* type, const char* type_name, int64_t n, const char* what,
                          int64_t* device, void** out) {
    int64_t have = 0;
    const int yes = is_object(PyObject_GetAttr(t, n_dtype), type);
    if (yes < 0 || as_int64(PyObject_CallMethodNoArgs(t, n_numel), &have) < 0) return -1;
    if (!yes || have != n) {
        PyErr_Format(PyExc_ValueError, "%s must be %s with %lld elements", what, type_name, (long long)n);
        return -1;
    }
    return get_data_here(t, device, out);
}

/* The same, or NULL for None. */
static int get_optional(PyObject* t, PyObject* type, const char* type_name, int64_t n, const char* what,
                        int64_t* device, void** out) {
    *out = NULL;
    return t == Py_None ? 0 : get_array_here(t, type, type_name, n, what, device, out);
}

typedef struct {
    dg_rows c;
    int64_t shape[2];
    dg_dtype type;
} rows_arg;

/* [rows, columns] BF16 or FP16, any row stride; with `like`, of its type and
 * rows and (cols >= 0) this many columns. */
static int get_rows(PyObject* t, const char* what, const rows_arg* like, int64_t cols, int64_t* device, rows_arg* r) {
    static const char kWanted[] = "must be BF16 or FP16 [rows, columns] with contiguous rows";
    int64_t stride[2];
    if (numbers(PyObject_CallMethodNoArgs(t, n_stride), 2, stride, what, kWanted) < 0 ||
        numbers(PyObject_GetAttr(t, n_shape), 2, r->shape, what, kWanted) < 0)
        return -1;
    PyObject* type = PyObject_GetAttr(t, n_dtype);
    if (type == NULL) return -1;
    const int bf16 = type == type_bf16, fp16 = type == type_fp16;
    Py_DECREF(type);
    if (!(bf16 || fp16) || (stride[1] != 1 && r->shape[1] > 1)) return fail_about(what, kWanted);
    r->type = bf16 ? DG_BF16 : DG_FP16;
    if (like != NULL && (r->type != like->type || r->shape[0] != like->shape[0] || (cols >= 0 && r->shape[1] != cols)))
        return fail_about(what, "must have the shape and type of its counterpart");
    void* data;
    if (on_current_device(t, device) < 0 || as_address(PyObject_CallMethodNoArgs(t, n_data_ptr), &data) < 0) return -1;
    r->c.data = data;
    r->c.stride = r->shape[0] > 1 ? stride[0] : r->shape[1];   /* a single one's stride may be anything */
    return 0;
}
/* The same, or no view (*c NULL) for None. */
static int get_rows_or_none(PyObject* t, const char* what, const rows_arg* like, int64_t cols, int64_t* device,
                            rows_arg* r, const dg_rows** c) {
    *c = NULL;
    if (t == Py_None) return 0;
    *c = &r->c;
    return get_rows(t, what, like, cols, device, r);
}

/* A contiguous tensor's address and bytes, or NULL and 0 for None. */
static int get_scratch(PyObject* t, int64_t* device, void** data, int64_t* bytes) {
    *data = NULL;
    *bytes = 0;
    if (t == Py_None) return 0;
    return get_data_here(t, device, data) < 0 || as_int64(PyObject_GetAttr(t, n_nbytes), bytes) < 0 ? -1 : 0;
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

/* What every norm takes: x, weight, residual, sum, eps. */
typedef struct {
    rows_arg x, residual, sum;
    const dg_rows *r, *s;
    void* weight;
    double eps;
    int64_t device;
} norm_arg;

static int get_norm(PyObject* x, PyObject* weight, PyObject* residual, PyObject* sum, PyObject* eps, norm_arg* n) {
    n->device = -1;
    if (get_rows(x, "x", NULL, -1, &n->device, &n->x) < 0 ||
        get_rows_or_none(residual, "residual", &n->x, n->x.shape[1], &n->device, &n->residual, &n->r) < 0 ||
        get_rows_or_none(sum, "sum", &n->x, n->x.shape[1], &n->device, &n->sum, &n->s) < 0 ||
        get_optional(weight, n->x.type == DG_BF16 ? type_bf16 : type_fp16, "of x's type", n->x.shape[1], "weight",
                     &n->device, &n->weight) < 0)
        return -1;
    n->eps = PyFloat_AsDouble(eps);
    return n->eps == -1.0 && PyErr_Occurred() ? -1 : 0;
}

/* (x, y, weight, residual, sum, eps, stream) */
static PyObject* py_rmsnorm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    norm_arg m;
    rows_arg y;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 7) < 0 || get_norm(a[0], a[2], a[3], a[4], a[5], &m) < 0 ||
        get_rows(a[1], "y", &m.x, m.x.shape[1], &m.device, &y) < 0 || get_stream(a[6], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_rmsnorm(&m.x.c, m.r, m.s, m.weight, m.x.shape[0], m.x.shape[1], m.eps, m.x.type, &y.c, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_rmsnorm");
}

/* (x, q, row_scale, weight, residual, sum, eps, stream) */
static PyObject* py_rmsnorm_e4m3(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    norm_arg m;
    void *q, *scale;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 8) < 0 || get_norm(a[0], a[3], a[4], a[5], a[6], &m) < 0 ||
        get_array_here(a[1], type_uint8, "uint8", m.x.shape[0] * m.x.shape[1], "q", &m.device, &q) < 0 ||
        get_array_here(a[2], type_float32, "FP32", m.x.shape[0], "row_scale", &m.device, &scale) < 0 || get_stream(a[7], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_rmsnorm_e4m3(&m.x.c, m.r, m.s, m.weight, m.x.shape[0], m.x.shape[1], m.eps, m.x.type, q, scale,
                              stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_rmsnorm_e4m3");
}

/* (x, scale, q, amax_out, next_scale_out, weight, residual, sum, eps, stream) */
static PyObject* py_rmsnorm_e4m3_amax(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    norm_arg m;
    void *scale, *q, *amax, *next;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 10) < 0 || get_norm(a[0], a[5], a[6], a[7], a[8], &m) < 0 ||
        get_array_here(a[1], type_float32, "FP32", 1, "scale", &m.device, &scale) < 0 ||
        get_array_here(a[2], type_uint8, "uint8", m.x.shape[0] * m.x.shape[1], "q", &m.device, &q) < 0 ||
        get_array_here(a[3], type_float32, "FP32", 1, "amax_out", &m.device, &amax) < 0 ||
        get_optional(a[4], type_float32, "FP32", 1, "next_scale_out", &m.device, &next) < 0 || get_stream(a[9], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_rmsnorm_e4m3_amax(&m.x.c, m.r, m.s, m.weight, m.x.shape[0], m.x.shape[1], m.eps, m.x.type, scale, q,
                                   amax, next, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_rmsnorm_e4m3_amax");
}

/* (s, dy, dx, weight, dsum, dweight, scratch, eps, stream) */
static PyObject* py_rmsnorm_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    norm_arg m;
    rows_arg dy, dx, dsum;
    const dg_rows* extra;
    void *dweight, *scratch;
    int64_t bytes;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 9) < 0 || get_norm(a[0], a[3], Py_None, Py_None, a[7], &m) < 0) return NULL;
    const int64_t cols = m.x.shape[1];
    if (get_rows(a[1], "dy", &m.x, cols, &m.device, &dy) < 0 || get_rows(a[2], "dx", &m.x, cols, &m.device, &dx) < 0 ||
        get_rows_or_none(a[4], "dsum", &m.x, cols, &m.device, &dsum, &extra) < 0 ||
        get_optional(a[5], type_float32, "FP32", cols, "dweight", &m.device, &dweight) < 0 ||
        get_scratch(a[6], &m.device, &scratch, &bytes) < 0 || get_stream(a[8], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_rmsnorm_grad(&m.x.c, m.weight, &dy.c, extra, m.x.shape[0], cols, m.eps, m.x.type, &dx.c, dweight,
                              scratch, bytes, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_rmsnorm_grad");
}

/* gated as 0 or 1, and the activation. */
static int get_activation(PyObject* gated_arg, PyObject* act_arg, int* gated, dg_activation* act) {
    int64_t kind;
    *gated = PyObject_IsTrue(gated_arg);
    if (*gated < 0 || as_int64(PyNumber_Index(act_arg), &kind) < 0) return -1;
    *act = (dg_activation)to_int(kind);
    return 0;
}

/* (x, act, y, q, q_scale, x_q, x_scale, gated, stream) */
static PyObject* py_activate(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    rows_arg x, y;
    const dg_rows* out;
    void *q, *q_scale, *x_q, *x_scale;
    int gated;
    int64_t device = -1;
    dg_activation act;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 9) < 0 || get_activation(a[7], a[1], &gated, &act) < 0 || get_rows(a[0], "x", NULL, -1, &device, &x) < 0)
        return NULL;
    if (gated && x.shape[1] % 2 != 0) {
        fail("x must have two halves when gated");
        return NULL;
    }
    const int64_t rows = x.shape[0], width = x.shape[1], cols = gated ? width / 2 : width;
    if (get_rows_or_none(a[2], "y", &x, cols, &device, &y, &out) < 0 ||
        get_optional(a[3], type_uint8, "uint8", rows * cols, "q", &device, &q) < 0 ||
        get_optional(a[4], type_float32, "FP32", rows, "q_scale", &device, &q_scale) < 0 ||
        get_optional(a[5], type_uint8, "uint8", rows * width, "x_q", &device, &x_q) < 0 ||
        get_optional(a[6], type_float32, "FP32", gated ? 2 * rows : rows, "x_scale", &device, &x_scale) < 0 ||
        get_stream(a[8], &stream) < 0)
        return NULL;
    if ((a[3] == Py_None) != (a[4] == Py_None) || (a[5] == Py_None) != (a[6] == Py_None)) {
        fail("codes and their scales must be given together");
        return NULL;
    }
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_activate(&x.c, gated, act, rows, cols, x.type, out, q, q_scale, x_q, x_scale, stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_activate");
}

/* (dy, act, dx, x, x_q, x_scale, gated, dbias, scratch, stream) */
static PyObject* py_activate_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    rows_arg dy, dx, x;
    const dg_rows* in;
    void *x_q, *x_scale, *dbias, *scratch;
    int64_t bytes;
    int gated;
    int64_t device = -1;
    dg_activation act;
    dg_stream_t stream;
    (void)self;
    if (want_args(n, 10) < 0 || get_activation(a[6], a[1], &gated, &act) < 0 ||
        get_rows(a[0], "dy", NULL, -1, &device, &dy) < 0)
        return NULL;
    const int64_t rows = dy.shape[0], cols = dy.shape[1], width = gated ? 2 * cols : cols;
    if ((a[3] == Py_None) == (a[4] == Py_None) || (a[4] == Py_None) != (a[5] == Py_None)) {
        fail("x, or x_q and x_scale, must be given");
        return NULL;
    }
    if (get_rows(a[2], "dx", &dy, width, &device, &dx) < 0 || get_rows_or_none(a[3], "x", &dy, width, &device, &x, &in) < 0 ||
        get_optional(a[4], type_uint8, "uint8", rows * width, "x_q", &device, &x_q) < 0 ||
        get_optional(a[5], type_float32, "FP32", gated ? 2 * rows : rows, "x_scale", &device, &x_scale) < 0 ||
        get_optional(a[7], type_float32, "FP32", width, "dbias", &device, &dbias) < 0 ||
        get_scratch(a[8], &device, &scratch, &bytes) < 0 || get_stream(a[9], &stream) < 0)
        return NULL;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = lib_activate_grad(&dy.c, in, x_q, x_scale, gated, act, rows, cols, dy.type, &dx.c, dbias, scratch, bytes,
                               stream);
    Py_END_ALLOW_THREADS
    return done(status, "dg_activate_grad");
}

/* A contiguous matrix: address, rows, columns, bytes an element, and whether
 * its type is one of the two. */
typedef struct {
    void* data;
    int64_t rows, cols, bytes;
    int bf16, fp16;
} matrix_arg;

static int get_matrix(PyObject* t, const char* what, int64_t* device, matrix_arg* m) {
    int64_t shape[2], bytes;
    if (numbers(PyObject_GetAttr(t, n_shape), 2, shape, what, "must have two dimensions") < 0 ||
        get_data_here(t, device, &m->data) < 0 || as_int64(PyObject_GetAttr(t, n_nbytes), &bytes) < 0)
        return -1;
    PyObject* type = PyObject_GetAttr(t, n_dtype);
    if (type == NULL) return -1;
    m->bf16 = type == type_bf16;
    m->fp16 = type == type_fp16;
    Py_DECREF(type);
    m->rows = shape[0];
    m->cols = shape[1];
    m->bytes = shape[0] > 0 && shape[1] > 0 ? bytes / (shape[0] * shape[1]) : 0;
    return 0;
}

/* A scale for the whole operand, or one a row. */
static int get_scales(PyObject* t, const char* what, int64_t rows, int64_t* device, void** out, int* per_row) {
    int64_t n;
    *out = NULL;
    *per_row = 0;
    if (t == Py_None) return 0;
    if (as_int64(PyObject_CallMethodNoArgs(t, n_numel), &n) < 0) return -1;
    *per_row = n != 1;
    return get_array_here(t, type_float32, "FP32", n == 1 ? 1 : rows, what, device, out);
}

/* (A, B, D, scale_a, scale_b, bias, act, residual, scale_d, amax_d, out, stream) */
static PyObject* fused(PyObject* const* a, Py_ssize_t n, int fp16) {
    const char* name = fp16 ? "dg_hgemm_fused" : "dg_fp8_gemm_fused";
    const int64_t in_bytes = fp16 ? 2 : 1;
    matrix_arg A, B, D, R;
    dg_epilogue e;
    void *sa, *sb, *bias, *sd, *amax;
    int64_t act, out, device = -1;
    dg_stream_t stream;
    if (want_args(n, 12) < 0 || get_matrix(a[0], "A", &device, &A) < 0 || get_matrix(a[1], "B", &device, &B) < 0 ||
        get_matrix(a[2], "D", &device, &D) < 0 || as_int64(PyNumber_Index(a[6]), &act) < 0 ||
        as_int64(PyNumber_Index(a[10]), &out) < 0)
        return NULL;
    const int64_t out_bytes = out == DG_E4M3 ? 1 : 2;
    if (A.cols != B.cols || D.rows != A.rows || D.cols != B.rows || (A.bytes != 0 && A.bytes != in_bytes) ||
        (B.bytes != 0 && B.bytes != in_bytes) || (D.bytes != 0 && D.bytes != out_bytes) || A.bf16 || B.bf16 ||
        (D.bf16 && out != DG_BF16) || (D.fp16 && out != DG_FP16)) {
        fail("A [M, K], B [N, K] and D [M, N] must agree, with elements of the operands' and the output's type");
        return NULL;
    }
    e.residual = NULL;
    e.residual_type = DG_BF16;
    if (a[7] != Py_None) {
        if (get_matrix(a[7], "residual", &device, &R) < 0) return NULL;
        if (!(R.bf16 || R.fp16) || R.rows != D.rows || R.cols != D.cols) {
            fail_about("residual", "must be BF16 or FP16 with the shape of D");
            return NULL;
        }
        e.residual = R.data;
        e.residual_type = R.bf16 ? DG_BF16 : DG_FP16;
    }
    if (get_scales(a[3], "scale_a", A.rows, &device, &sa, &e.scale_a_rows) < 0 ||
        get_scales(a[4], "scale_b", B.rows, &device, &sb, &e.scale_b_rows) < 0 ||
        get_optional(a[5], type_float32, "FP32", B.rows, "bias", &device, &bias) < 0 ||
        get_optional(a[8], type_float32, "FP32", 1, "scale_d", &device, &sd) < 0 ||
        get_optional(a[9], type_float32, "FP32", 1, "amax_d", &device, &amax) < 0 || get_stream(a[11], &stream) < 0)
        return NULL;
    e.scale_a = sa;
    e.scale_b = sb;
    e.bias = bias;
    e.act = (dg_activation)to_int(act);
    e.scale_d = sd;
    e.amax_d = amax;
    dg_status status;
    Py_BEGIN_ALLOW_THREADS
    status = fp16 ? lib_hgemm_fused(A.data, B.data, D.data, A.rows, B.rows, A.cols, &e, (dg_dtype)to_int(out), stream)
                  : lib_fp8_gemm_fused(A.data, B.data, D.data, A.rows, B.rows, A.cols, &e, (dg_dtype)to_int(out),
                                       stream);
    Py_END_ALLOW_THREADS
    return done(status, name);
}

static PyObject* py_fp8_gemm_fused(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return fused(a, n, 0);
}
static PyObject* py_hgemm_fused(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    return fused(a, n, 1);
}

/* (addresses of the library's functions around a layer's products, in the
 * order of the pointers above; torch's uint8) */
static PyObject* py_bind_layer(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    void* f[8];
    (void)self;
    if (want_args(n, 9) < 0) return NULL;
    for (int i = 0; i < 8; ++i)
        if (as_address(Py_NewRef(a[i]), &f[i]) < 0) return NULL;
    *(void**)&lib_rmsnorm = f[0];
    *(void**)&lib_rmsnorm_e4m3 = f[1];
    *(void**)&lib_rmsnorm_e4m3_amax = f[2];
    *(void**)&lib_rmsnorm_grad = f[3];
    *(void**)&lib_activate = f[4];
    *(void**)&lib_activate_grad = f[5];
    *(void**)&lib_fp8_gemm_fused = f[6];
    *(void**)&lib_hgemm_fused = f[7];
    Py_XSETREF(type_uint8, Py_NewRef(a[8]));
    Py_RETURN_NONE;
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
    {"bind_layer", (PyCFunction)(void (*)(void))py_bind_layer, METH_FASTCALL, NULL},
    {"rmsnorm", (PyCFunction)(void (*)(void))py_rmsnorm, METH_FASTCALL, NULL},
    {"rmsnorm_e4m3", (PyCFunction)(void (*)(void))py_rmsnorm_e4m3, METH_FASTCALL, NULL},
    {"rmsnorm_e4m3_amax", (PyCFunction)(void (*)(void))py_rmsnorm_e4m3_amax, METH_FASTCALL, NULL},
    {"rmsnorm_grad", (PyCFunction)(void (*)(void))py_rmsnorm_grad, METH_FASTCALL, NULL},
    {"fp8_gemm_fused", (PyCFunction)(void (*)(void))py_fp8_gemm_fused, METH_FASTCALL, NULL},
    {"hgemm_fused", (PyCFunction)(void (*)(void))py_hgemm_fused, METH_FASTCALL, NULL},
    {"activate", (PyCFunction)(void (*)(void))py_activate, METH_FASTCALL, NULL},
    {"activate_grad", (PyCFunction)(void (*)(void))py_activate_grad, METH_FASTCALL, NULL},
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
        {&n_get_device, "get_device"},
    };
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if (*names[i].at == NULL && (*names[i].at = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
    return PyModule_Create(&module);
}
