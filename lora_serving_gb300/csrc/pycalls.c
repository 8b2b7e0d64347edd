/* pycalls.c -- the Python side of the calls between a decode step's
 * projections: lora_rms_norm, lora_kv4_append, lora_kv4_read, lora_kv4_attend.
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

static PyObject *s_is_cuda, *s_dtype, *s_device, *s_shape, *s_stride, *s_data_ptr, *s_nbytes, *s_is_contiguous, *s_cuda_stream;
static PyObject *bf16, *f32, *i32, *e4m3;      /* torch's dtype objects */
static PyObject *current_device, *raw_stream;  /* () -> device index; (device index) -> stream handle */
static __typeof__(&lora_rms_norm) norm_fn;
static __typeof__(&lora_kv4_append) append_fn;
static __typeof__(&lora_kv4_read) read_fn;
static __typeof__(&lora_kv4_attend) attend_fn;

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

/* Pointer of a CUDA tensor of this element type (NULL: any). */
static int pointer(PyObject* t, const char* name, PyObject* want, void** out)
{
    PyObject *cuda = PyObject_GetAttr(t, s_is_cuda), *dtype = NULL, *p;
    if (!cuda) return -1;
    const int is_cuda = cuda == Py_True;
    Py_DECREF(cuda);
    if (!(dtype = PyObject_GetAttr(t, s_dtype))) return -1;
    if (!is_cuda || (want && dtype != want)) {
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

/* Pointer and leading dimension of a row-major operand: a CUDA tensor of this
 * element type with so many rows and columns at least and unit column
 * stride; its sizes in `shape` where asked for.  None: (NULL, 0). */
static int matrix(PyObject* t, const char* name, PyObject* dtype, long rows, long cols, void** out, int* ld)
{
    long n[3], st[2];
    *out = NULL;
    *ld = 0;
    if (t == Py_None) return 0;
    if (pointer(t, name, dtype, out)) return -1;
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

/* ((addresses of lora_rms_norm, lora_kv4_append, lora_kv4_read, lora_kv4_attend), (bf16, fp32, int32, e4m3),
 * current_device, raw_stream) */
static PyObject* bind(PyObject* self, PyObject* args)
{
    unsigned long long fn[4];
    PyObject* o[6];
    if (!PyArg_ParseTuple(args, "(KKKK)(OOOO)OO", &fn[0], &fn[1], &fn[2], &fn[3], &o[0], &o[1], &o[2], &o[3], &o[4], &o[5])) return NULL;
    PyObject** to[6] = {&bf16, &f32, &i32, &e4m3, &current_device, &raw_stream};
    for (int i = 0; i < 6; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*to[i], o[i]);
    }
    norm_fn = (__typeof__(norm_fn))(uintptr_t)fn[0];
    append_fn = (__typeof__(append_fn))(uintptr_t)fn[1];
    read_fn = (__typeof__(read_fn))(uintptr_t)fn[2];
    attend_fn = (__typeof__(attend_fn))(uintptr_t)fn[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, NULL},
    {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, NULL},
    {"kv4_append", (PyCFunction)(void (*)(void))kv4_append, METH_FASTCALL, NULL},
    {"kv4_read", (PyCFunction)(void (*)(void))kv4_read, METH_FASTCALL, NULL},
    {"kv4_attend", (PyCFunction)(void (*)(void))kv4_attend, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL},
};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycalls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycalls(void)
{
    PyObject** names[] = {&s_is_cuda, &s_dtype, &s_device, &s_shape, &s_stride, &s_data_ptr, &s_nbytes, &s_is_contiguous, &s_cuda_stream};
    const char* text[] = {"is_cuda", "dtype", "device", "shape", "stride", "data_ptr", "nbytes", "is_contiguous", "cuda_stream"};
    for (int i = 0; i < 9; ++i)
        if (!*names[i] && !(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
    return PyModule_Create(&module);
}
