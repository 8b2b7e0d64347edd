/* pycalls.c -- the Python side of the calls between a decode step's
 * projections: lora_rms_norm, lora_kv4_append, lora_kv4_read, lora_kv4_attend,
 * and of drafted decoding: lora_kv4_plan, lora_kv4_attend_tree, lora_kv4_keep,
 * lora_logits_adjust.
 *
 * A kernel of 3 us is launched from Python by a call of up to nineteen
 * arguments.  Read and converted by the interpreter one at a time they took
 * longer than the kernel (7.6 us a norm, of which the launch was 1.7); here
 * the tensors' attributes are read through the C API, and the library is
 * called directly.  The checks are those that the C ABI cannot make: a
 * tensor on a CUDA device, of the element type the kernel reads, with the
 * rows and columns it will touch and unit column stride.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>

#include "lora.h"

static PyObject *s_is_cuda, *s_dtype, *s_device, *s_shape, *s_stride, *s_data_ptr, *s_nbytes, *s_is_contiguous, *s_cuda_stream, *s_numel;
static PyObject *bf16, *f32, *i32, *e4m3;      /* torch's dtype objects */
static PyObject *current_device, *raw_stream;  /* () -> device index; (device index) -> stream handle */
static __typeof__(&lora_rms_norm) norm_fn;
static __typeof__(&lora_kv4_append) append_fn;
static __typeof__(&lora_kv4_read) read_fn;
static __typeof__(&lora_kv4_attend) attend_fn;
static __typeof__(&lora_kv4_plan) plan_fn;
static __typeof__(&lora_kv4_attend_tree) tree_fn;
static __typeof__(&lora_kv4_keep) keep_fn;
static __typeof__(&lora_logits_adjust) logits_fn;

static PyObject* call0(PyObject* o, PyObject* method)
{
    return PyObject_VectorcallMethod(method, &o, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

static int as_int(PyObject* o, const char* name, int* out)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) return -1;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s is out of range: %ld", name, v);
        return -1;
    }
    *out = (int)v;
    return 0;
}

/* Pointer of a CUDA tensor of one of two element types (want NULL: any); which of them in `second` where there are two. */
static int pointer_of(PyObject* t, const char* name, PyObject* want, PyObject* other, int* second, void** out)
{
    PyObject *cuda = PyObject_GetAttr(t, s_is_cuda), *dtype = NULL, *p;
    if (!cuda) return -1;
    const int is_cuda = cuda == Py_True;
    Py_DECREF(cuda);
    if (!(dtype = PyObject_GetAttr(t, s_dtype))) return -1;
    if (second) *second = dtype == other;
    if (!is_cuda || (want && dtype != want && dtype != other)) {
        PyObject* device = PyObject_GetAttr(t, s_device);
        if (device && want) PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor of %S, got %S on %S", name, want, dtype, device);
        else if (device) PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor, got one on %S", name, device);
        Py_XDECREF(device);
        Py_DECREF(dtype);
        return -1;
    }
    Py_DECREF(dtype);
    if (!(p = call0(t, s_data_ptr))) return -1;
    *out = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return PyErr_Occurred() ? -1 : 0;
}

/* ... of this one. */
static int pointer(PyObject* t, const char* name, PyObject* want, void** out) { return pointer_of(t, name, want, want, NULL, out); }

/* A tensor's sizes: how many dimensions, the first three of them in `out`; -1 with an error. */
static int sizes(PyObject* t, long out[3])
{
    PyObject* shape = PyObject_GetAttr(t, s_shape);
    if (!shape) return -1;
    if (!PyTuple_Check(shape)) {
        Py_DECREF(shape);
        PyErr_SetString(PyExc_TypeError, "a tensor's shape must be a tuple");
        return -1;
    }
    const int n = (int)PyTuple_GET_SIZE(shape);
    for (int i = 0; i < n && i < 3; ++i) out[i] = PyLong_AsLong(PyTuple_GET_ITEM(shape, i));
    Py_DECREF(shape);
    return PyErr_Occurred() ? -1 : n;
}

/* Strides of a tensor of `n` dimensions. */
static int strides(PyObject* t, int n, long* out)
{
    PyObject* st = call0(t, s_stride);
    if (!st) return -1;
    if (!PyTuple_Check(st) || PyTuple_GET_SIZE(st) != n) {
        Py_DECREF(st);
        PyErr_SetString(PyExc_TypeError, "a tensor's strides must be a tuple, one to a dimension");
        return -1;
    }
    for (int i = 0; i < n; ++i) out[i] = PyLong_AsLong(PyTuple_GET_ITEM(st, i));
    Py_DECREF(st);
    return PyErr_Occurred() ? -1 : 0;
}

/* Pointer and leading dimension of a row-major operand: a CUDA tensor of
 * one of two element types (which of them in `second`) with so many rows and
 * columns at least and unit column stride; its sizes in `n`. */
static int matrix_of(PyObject* t, const char* name, PyObject* dtype, PyObject* other, int* second, long rows, long cols, void** out, int* ld, long n[3])
{
    long st[2];
    *out = NULL;
    *ld = 0;
    n[0] = n[1] = 0;
    if (t == Py_None) return 0;
    if (pointer_of(t, name, dtype, other, second, out)) return -1;
    const int dims = sizes(t, n);
    if (dims < 0) return -1;
    if (dims != 2 || n[0] < rows || n[1] < cols) {
        PyErr_Format(PyExc_ValueError, "%s must be 2-D with %ld rows and %ld columns at least", name, rows, cols);
        return -1;
    }
    if (strides(t, 2, st)) return -1;
    if ((st[1] != 1 && n[1] > 1) || st[0] < 0 || st[0] > INT_MAX) {
        PyErr_Format(PyExc_ValueError, "%s must have unit column stride, and rows less than 2^31 elements apart", name);
        return -1;
    }
    *ld = (int)st[0];
    return 0;
}

/* ... of this one.  None: (NULL, 0). */
static int matrix(PyObject* t, const char* name, PyObject* dtype, long rows, long cols, void** out, int* ld)
{
    long n[3];
    return matrix_of(t, name, dtype, dtype, NULL, rows, cols, out, ld, n);
}

/* A tensor, a raw pointer as an integer, or None. */
static int device(PyObject* t, const char* name, PyObject* dtype, void** out)
{
    *out = NULL;
    if (t == Py_None) return 0;
    if (!PyLong_Check(t)) return pointer(t, name, dtype, out);
    *out = PyLong_AsVoidPtr(t);
    return PyErr_Occurred() ? -1 : 0;
}

/* A stream object, a raw handle, or None: the current stream (a CUDA tensor
 * has been seen, so that CUDA is up). */
static int stream_of(PyObject* s, void** out)
{
    PyObject *h, *dev = NULL;
    if (PyLong_Check(s)) {
        *out = PyLong_AsVoidPtr(s);
        return PyErr_Occurred() ? -1 : 0;
    }
    if (s != Py_None) h = PyObject_GetAttr(s, s_cuda_stream);
    else h = (dev = PyObject_CallNoArgs(current_device)) ? PyObject_CallOneArg(raw_stream, dev) : NULL;
    Py_XDECREF(dev);
    if (!h) return -1;
    *out = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    return PyErr_Occurred() ? -1 : 0;
}

static int count(Py_ssize_t n, Py_ssize_t want)
{
    if (n == want) return 0;
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    return -1;
}

#define CALL(status, ...)              \
    lora_status_t status;              \
    Py_BEGIN_ALLOW_THREADS             \
    status = __VA_ARGS__;              \
    Py_END_ALLOW_THREADS               \
    return PyLong_FromLong((long)status)

/* (x, weight, eps, residual, residual_out, y, y8, scales, group, stream) */
static PyObject* rms_norm(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void *x, *w, *res, *res_out, *y, *y8, *scales, *stream;
    int ld_x, ld_res, ld_ro, ld_y, ld_y8, ld_s, group;
    long sx[3], sw[3], st;
    if (count(n, 10) || as_int(a[8], "group", &group)) return NULL;
    const float eps = (float)PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) return NULL;
    const int dims = sizes(a[0], sx), wdims = sizes(a[1], sw);
    if (dims < 0 || wdims < 0) return NULL;
    if (dims != 2 || sx[0] > INT_MAX || sx[1] > INT_MAX) return PyErr_Format(PyExc_ValueError, "x must be 2-D, its sizes below 2^31");
    if (wdims == 1 && strides(a[1], 1, &st)) return NULL;
    if (wdims != 1 || sw[0] != sx[1] || st != 1) return PyErr_Format(PyExc_ValueError, "weight must hold %ld adjacent values", sx[1]);
    const long groups = group > 0 ? (sx[1] + group - 1) / group : 1;
    if (matrix(a[5], "y", bf16, sx[0], sx[1], &y, &ld_y) || matrix(a[6], "y8", e4m3, sx[0], sx[1], &y8, &ld_y8) ||
        matrix(a[7], "scales", f32, sx[0], groups, &scales, &ld_s) || matrix(a[4], "residual_out", bf16, sx[0], sx[1], &res_out, &ld_ro) ||
        matrix(a[0], "x", bf16, sx[0], sx[1], &x, &ld_x) || matrix(a[3], "residual", bf16, sx[0], sx[1], &res, &ld_res) ||
        pointer(a[1], "weight", bf16, &w) || stream_of(a[9], &stream))
        return NULL;
    CALL(status, norm_fn(y, ld_y, y8, ld_y8, scales, ld_s, group, res_out, ld_ro, x, ld_x, res, ld_res, w, (int)sx[0], (int)sx[1], eps, stream));
}

/* The C structs of a store.KV4Cache and a store.KV4Batch, by their addresses. */
static int structs(PyObject* c, PyObject* b, const lora_kv4_cache_t** cache, const lora_kv4_batch_t** batch)
{
    *cache = PyLong_AsVoidPtr(c);
    *batch = PyLong_AsVoidPtr(b);
    if (PyErr_Occurred()) return -1;
    if (*cache && *batch) return 0;
    PyErr_SetString(PyExc_ValueError, "no cache or no batch");
    return -1;
}

/* (q_out, x, cache, batch, n_heads, q_off, k_off, v_off, rope, positions, axis_pairs, dev_status, stream) */
static PyObject* kv4_append(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    const lora_kv4_cache_t* cache;
    const lora_kv4_batch_t* batch;
    void *q, *x, *rope = NULL, *pos = NULL, *status_word, *stream;
    int ld_q, ld_x, ld_pos = 0, heads, q_off, k_off, v_off, rot = 0, max_pos = 0, axes = 0, pairs[LORA_MAX_ROPE_AXES];
    if (count(n, 13) || structs(a[2], a[3], &cache, &batch) || as_int(a[4], "n_heads", &heads) || as_int(a[5], "q_off", &q_off) ||
        as_int(a[6], "k_off", &k_off) || as_int(a[7], "v_off", &v_off))
        return NULL;
    /* the columns that the slices end at, of x itself: the library knows the row stride of the buffer that x may be a part of */
    const long nq = (long)heads * cache->head_dim, nk = (long)cache->n_kv * cache->head_dim;
    const long kv_end = (k_off > v_off ? k_off : v_off) + nk, end = q_off + nq > kv_end ? q_off + nq : kv_end;
    if (matrix(a[0], "q_out", bf16, batch->n_rows, nq, &q, &ld_q) || matrix(a[1], "x", bf16, batch->n_rows, end, &x, &ld_x)) return NULL;
    if (a[8] != Py_None) {
        long s[3];
        const int dims = sizes(a[8], s);
        if (dims < 0) return NULL;
        PyObject* c = call0(a[8], s_is_contiguous);
        if (!c) return NULL;
        const int ok = dims == 3 && s[2] == 2 && c == Py_True && s[0] <= INT_MAX && s[1] <= INT_MAX / 2;
        Py_DECREF(c);
        if (!ok) return PyErr_Format(PyExc_ValueError, "rope must be contiguous [max_pos][pairs][2]");
        if (pointer(a[8], "rope", f32, &rope)) return NULL;
        max_pos = (int)s[0];
        rot = 2 * (int)s[1];
        if (a[10] == Py_None) {
            axes = 1;
            pairs[0] = (int)s[1];
        } else {
            PyObject* seq = PySequence_Fast(a[10], "axis_pairs must be a sequence");
            if (!seq) return NULL;
            const Py_ssize_t k = PySequence_Fast_GET_SIZE(seq);
            int bad = k < 1 || k > LORA_MAX_ROPE_AXES;
            if (bad) PyErr_Format(PyExc_ValueError, "axis_pairs must have 1 to %d entries", LORA_MAX_ROPE_AXES);
            for (Py_ssize_t i = 0; i < k && !bad; ++i) bad = as_int(PySequence_Fast_GET_ITEM(seq, i), "axis_pairs", &pairs[i]) != 0;
            Py_DECREF(seq);
            if (bad) return NULL;
            axes = (int)k;
        }
        if (matrix(a[9], "positions", i32, batch->n_rows, axes, &pos, &ld_pos)) return NULL;
    }
    if (device(a[11], "dev_status", i32, &status_word) || stream_of(a[12], &stream)) return NULL;
    CALL(status, append_fn(q, ld_q, x, ld_x, heads, q_off, k_off, v_off, rope, rot, max_pos, pos, ld_pos, axes ? pairs : NULL, axes, cache,
                           batch, status_word, stream));
}

/* (k, v, cache, batch, dev_status, stream) */
static PyObject* kv4_read(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    const lora_kv4_cache_t* cache;
    const lora_kv4_batch_t* batch;
    void *k, *v, *status_word, *stream;
    int ld_k, ld_v;
    if (count(n, 6) || structs(a[2], a[3], &cache, &batch)) return NULL;
    const long width = (long)cache->n_kv * cache->head_dim;
    if (matrix(a[0], "k", bf16, batch->n_rows, width, &k, &ld_k) || matrix(a[1], "v", bf16, batch->n_rows, width, &v, &ld_v) ||
        device(a[4], "dev_status", i32, &status_word) || stream_of(a[5], &stream))
        return NULL;
    CALL(status, read_fn(k, ld_k, v, ld_v, cache, batch, status_word, stream));
}

/* (out, q, cache, batch, workspace, n_heads, scale, window, dev_status, stream) */
static PyObject* kv4_attend(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    const lora_kv4_cache_t* cache;
    const lora_kv4_batch_t* batch;
    void *out, *q, *ws, *status_word, *stream;
    int ld_out, ld_q, heads, window;
    if (count(n, 10) || structs(a[2], a[3], &cache, &batch) || as_int(a[5], "n_heads", &heads) || as_int(a[7], "window", &window)) return NULL;
    const float scale = (float)PyFloat_AsDouble(a[6]);
    if (PyErr_Occurred()) return NULL;
    const long width = (long)heads * cache->head_dim;
    if (matrix(a[0], "out", bf16, batch->n_rows, width, &out, &ld_out) || matrix(a[1], "q", bf16, batch->n_rows, width, &q, &ld_q) ||
        pointer(a[4], "workspace", NULL, &ws))
        return NULL;
    PyObject* nb = PyObject_GetAttr(a[4], s_nbytes);
    if (!nb) return NULL;
    const size_t bytes = PyLong_AsSize_t(nb);
    Py_DECREF(nb);
    if (PyErr_Occurred() || device(a[8], "dev_status", i32, &status_word) || stream_of(a[9], &stream)) return NULL;
    CALL(status, attend_fn(out, ld_out, q, ld_q, heads, scale, window, cache, batch, ws, bytes, status_word, stream));
}

/* So many adjacent entries at least, of a contiguous tensor of this element type; None: NULL.  (Two attributes that are
 * cheaper than sizes and strides: a call may have six such tensors.) */
static int vector(PyObject* t, const char* name, PyObject* dtype, long count, void** out)
{
    *out = NULL;
    if (t == Py_None) return 0;
    if (pointer(t, name, dtype, out)) return -1;
    PyObject *n = call0(t, s_numel), *c = n ? call0(t, s_is_contiguous) : NULL;
    const long has = c ? PyLong_AsLong(n) : 0;
    const int ok = c && !PyErr_Occurred() && c == Py_True && has >= count;
    Py_XDECREF(n);
    Py_XDECREF(c);
    if (!ok && !PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s must hold %ld adjacent entries at least", name, count);
    return ok ? 0 : -1;
}

/* What store.KV4Plan hands over: the call's arguments but for the lengths. */
typedef struct {
    int32_t *q_starts, *ctx_lens, *row_seq, *positions;
    int64_t* slots;
    int32_t n_seqs, max_rows, max_q_len, max_ctx_len;
    lora_kv4_pool_t pool;
} plan_t;

/* (plan, q_lens, lens, depths, dev_status, stream) */
static PyObject* kv4_plan(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void *q, *lens, *depths, *status_word, *stream;
    if (count(n, 6)) return NULL;
    const plan_t* p = PyLong_AsVoidPtr(a[0]);
    if (PyErr_Occurred()) return NULL;
    if (!p) return PyErr_Format(PyExc_ValueError, "no plan");
    if (vector(a[1], "q_lens", i32, p->n_seqs, &q) || vector(a[2], "lens", i32, p->n_seqs, &lens) || vector(a[3], "depths", i32, p->max_rows, &depths) ||
        device(a[4], "dev_status", i32, &status_word) || stream_of(a[5], &stream))
        return NULL;
    CALL(status, plan_fn(p->q_starts, p->ctx_lens, p->row_seq, p->positions, p->slots, q, lens, depths, p->n_seqs, p->max_rows, p->max_q_len,
                         p->max_ctx_len, &p->pool, status_word, stream));
}

/* (out, q, cache, batch, tree, workspace, n_heads, scale, window, dev_status, stream) */
static PyObject* kv4_attend_tree(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    const lora_kv4_cache_t* cache;
    const lora_kv4_batch_t* batch;
    void *out, *q, *tree, *ws, *status_word, *stream;
    int ld_out, ld_q, ld_tree, heads, window;
    if (count(n, 11) || structs(a[2], a[3], &cache, &batch) || as_int(a[6], "n_heads", &heads) || as_int(a[8], "window", &window)) return NULL;
    const float scale = (float)PyFloat_AsDouble(a[7]);
    if (PyErr_Occurred()) return NULL;
    const long width = (long)heads * cache->head_dim;
    if (matrix(a[0], "out", bf16, batch->n_rows, width, &out, &ld_out) || matrix(a[1], "q", bf16, batch->n_rows, width, &q, &ld_q) ||
        matrix(a[4], "tree", i32, batch->n_rows, (batch->max_q_len + 31L) / 32, &tree, &ld_tree) || pointer(a[5], "workspace", NULL, &ws))
        return NULL;
    if (batch->n_rows == 1 && ld_tree < (batch->max_q_len + 31L) / 32) ld_tree = (int)((batch->max_q_len + 31L) / 32);   /* one row: any stride */
    PyObject* nb = PyObject_GetAttr(a[5], s_nbytes);
    if (!nb) return NULL;
    const size_t bytes = PyLong_AsSize_t(nb);
    Py_DECREF(nb);
    if (PyErr_Occurred() || device(a[9], "dev_status", i32, &status_word) || stream_of(a[10], &stream)) return NULL;
    CALL(status, tree_fn(out, ld_out, q, ld_q, heads, scale, window, tree, ld_tree, cache, batch, ws, bytes, status_word, stream));
}

/* (caches, n_caches, batch, n_keep, path, lens, dev_status, stream) */
static PyObject* kv4_keep(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    const lora_kv4_cache_t* caches;
    const lora_kv4_batch_t* batch;
    void *keep, *path, *lens, *status_word, *stream;
    int n_caches, ld_path;
    long s[3];
    if (count(n, 8) || structs(a[0], a[2], &caches, &batch) || as_int(a[1], "n_caches", &n_caches)) return NULL;
    if (vector(a[3], "n_keep", i32, batch->n_seqs, &keep) || matrix_of(a[4], "path", i32, i32, NULL, batch->n_seqs, 0, &path, &ld_path, s) ||
        vector(a[5], "lens", i32, batch->n_seqs, &lens) || device(a[6], "dev_status", i32, &status_word) || stream_of(a[7], &stream))
        return NULL;
    if (batch->n_seqs > 1 && s[1] != ld_path) return PyErr_Format(PyExc_ValueError, "path must be contiguous");   /* a row's entries are its columns */
    CALL(status, keep_fn(caches, n_caches, batch, keep, path, (int)s[1], lens, status_word, stream));
}

/* (out, logits, rules, row_seq, drafts, tree, q_starts, allowed, allowed_rows, dev_status, stream) */
static PyObject* logits_adjust(PyObject* self, PyObject* const* a, Py_ssize_t n)
{
    void *out, *in, *row_seq, *drafts, *tree, *starts, *allowed, *allowed_rows, *status_word, *stream;
    int ld_out, ld, ld_tree, ld_allowed, n_allowed = 0;
    long so[3], si[3], sa[3], st[3];
    int out_f32 = 0, in_f32 = 0;
    if (count(n, 11)) return NULL;
    const lora_logits_rules_t* rules = PyLong_AsVoidPtr(a[2]);
    if (PyErr_Occurred()) return NULL;
    if (matrix_of(a[0], "out", bf16, f32, &out_f32, 0, 0, &out, &ld_out, so) || matrix_of(a[1], "logits", bf16, f32, &in_f32, 0, 0, &in, &ld, si)) return NULL;
    if (so[0] != si[0] || so[1] != si[1] || si[0] > INT_MAX || si[1] > INT_MAX)
        return PyErr_Format(PyExc_ValueError, "out must have the shape of logits, its sizes below 2^31");
    const long rows = si[0], words = (si[1] + 31) / 32;
    if (vector(a[3], "row_seq", i32, rows, &row_seq) || vector(a[4], "drafts", i32, rows, &drafts) ||
        matrix_of(a[5], "tree", i32, i32, NULL, rows, 1, &tree, &ld_tree, st) ||
        vector(a[6], "q_starts", i32, rules ? rules->n_seqs + 1L : 0, &starts) ||
        matrix_of(a[7], "allowed", i32, i32, NULL, 1, words, &allowed, &ld_allowed, sa) ||
        vector(a[8], "allowed_rows", i32, rows, &allowed_rows) || device(a[9], "dev_status", i32, &status_word) || stream_of(a[10], &stream))
        return NULL;
    if (allowed) {
        if (sa[0] > INT_MAX) return PyErr_Format(PyExc_ValueError, "allowed must have less than 2^31 rows");
        n_allowed = (int)sa[0];
        if (n_allowed == 1 && ld_allowed < words) ld_allowed = (int)words;   /* one row: any stride */
    }
    if (tree) {   /* a row's words are its columns: what lies between rows of a wider buffer is not looked at */
        if (rows > 1 && st[1] != ld_tree) return PyErr_Format(PyExc_ValueError, "tree must be contiguous");
        ld_tree = (int)st[1];
    }
    CALL(status, logits_fn(out, out_f32 ? LORA_F32 : LORA_BF16, ld_out, in, in_f32 ? LORA_F32 : LORA_BF16, ld, (int)rows, (int)si[1], rules, row_seq, drafts, tree, ld_tree, starts, allowed,
                           ld_allowed, n_allowed, allowed_rows, status_word, stream));
}

/* ((addresses of lora_rms_norm, lora_kv4_append, lora_kv4_read, lora_kv4_attend, lora_kv4_plan, lora_kv4_attend_tree, lora_kv4_keep,
 * lora_logits_adjust), (bf16, fp32, int32, e4m3), current_device, raw_stream) */
static PyObject* bind(PyObject* self, PyObject* args)
{
    unsigned long long fn[8];
    PyObject* o[6];
    if (!PyArg_ParseTuple(args, "(KKKKKKKK)(OOOO)OO", &fn[0], &fn[1], &fn[2], &fn[3], &fn[4], &fn[5], &fn[6], &fn[7], &o[0], &o[1], &o[2], &o[3], &o[4], &o[5])) return NULL;
    PyObject** to[6] = {&bf16, &f32, &i32, &e4m3, &current_device, &raw_stream};
    for (int i = 0; i < 6; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*to[i], o[i]);
    }
    norm_fn = (__typeof__(norm_fn))(uintptr_t)fn[0];
    append_fn = (__typeof__(append_fn))(uintptr_t)fn[1];
    read_fn = (__typeof__(read_fn))(uintptr_t)fn[2];
    attend_fn = (__typeof__(attend_fn))(uintptr_t)fn[3];
    plan_fn = (__typeof__(plan_fn))(uintptr_t)fn[4];
    tree_fn = (__typeof__(tree_fn))(uintptr_t)fn[5];
    keep_fn = (__typeof__(keep_fn))(uintptr_t)fn[6];
    logits_fn = (__typeof__(logits_fn))(uintptr_t)fn[7];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, NULL},
    {"kv4_append", (PyCFunction)(void (*)(void))kv4_append, METH_FASTCALL, NULL},
    {"kv4_read", (PyCFunction)(void (*)(void))kv4_read, METH_FASTCALL, NULL},
    {"kv4_attend", (PyCFunction)(void (*)(void))kv4_attend, METH_FASTCALL, NULL},
    {"kv4_plan", (PyCFunction)(void (*)(void))kv4_plan, METH_FASTCALL, NULL},
    {"kv4_attend_tree", (PyCFunction)(void (*)(void))kv4_attend_tree, METH_FASTCALL, NULL},
    {"kv4_keep", (PyCFunction)(void (*)(void))kv4_keep, METH_FASTCALL, NULL},
    {"logits_adjust", (PyCFunction)(void (*)(void))logits_adjust, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycalls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycalls(void)
{
    PyObject** names[] = {&s_is_cuda, &s_dtype, &s_device, &s_shape, &s_stride, &s_data_ptr, &s_nbytes, &s_is_contiguous, &s_cuda_stream, &s_numel};
    const char* text[] = {"is_cuda", "dtype", "device", "shape", "stride", "data_ptr", "nbytes", "is_contiguous", "cuda_stream", "numel"};
    for (int i = 0; i < 10; ++i)
        if (!*names[i] && !(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
    return PyModule_Create(&module);
}
