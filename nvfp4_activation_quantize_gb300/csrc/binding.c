/*
 * binding.c -- the Python binding's short way into the calls that are made once a layer and token.
 *
 * A decoding step's calls run for a few microseconds on the GPU; checking a dozen
 * tensors in Python took two to three times that.  Each function here looks at its
 * tensors through their public attributes (type, dtype, device, shape, strides,
 * data_ptr) and, where all of them are what the call needs, calls the library and
 * returns its status.  Where anything is not, it returns None without a word: the Python
 * code then goes the long way, whose checks say what is wrong.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "../../include/h3q.h"

#define MAX_DIMS 4

static PyObject *g_tensor, *g_bf16, *g_u8, *g_i32, *g_i64, *g_f32; /* torch's class and dtypes */
static PyObject *g_get_device, *g_get_stream;                     /* current device, its current stream's handle */
static PyObject *s_dtype, *s_device, *s_shape, *s_index, *s_type, *s_cuda, *s_contiguous, *s_data_ptr, *s_stride,
    *s_numel;

typedef int (*write_fn)(const void *, int64_t, const void *, int64_t, int64_t, const int32_t *, const int32_t *,
                        const int32_t *, int64_t, int64_t, const float *, const float *, uint8_t *, uint8_t *,
                        uint8_t *, uint8_t *, int64_t, int64_t, int64_t, int64_t, void *);
typedef int (*read_fn)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, int64_t, int64_t, int64_t,
                       int64_t, const float *, const float *, int64_t, const int32_t *, const int32_t *,
                       const int32_t *, int64_t, int64_t, void *, void *, void *);
typedef int (*cached_fn)(const void *, int64_t, int64_t, int64_t, int64_t, const int32_t *, const int32_t *,
                         const int32_t *, int64_t, int64_t, const int64_t *, const uint8_t *, const uint8_t *,
                         const uint8_t *, const uint8_t *, int64_t, int64_t, int64_t, int64_t, const float *,
                         const float *, float, void *, float *, void *, int64_t, void *);
typedef int (*varlen_fn)(const void *, int64_t, const void *, int64_t, const void *, int64_t, const int32_t *,
                         const int32_t *, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, float, void *,
                         float *, void *);
typedef int (*axes_fn)(const void *, int64_t, const void *, int64_t, const void *, int64_t, const void *,
                       const void *, const void *, const void *, const void *, const int32_t *, int64_t,
                       const int64_t *, const double *, const double *, int, int, int, int64_t, int64_t, int64_t,
                       int64_t, float, void *, void *, void *, void *);
typedef int (*postnorm_fn)(float *, int64_t, const void *, int64_t, const void *, const void *, const void *, float,
                           const void *, const void *, int64_t, const int32_t *, int64_t, float, int64_t, int64_t,
                           const float *, uint8_t *, uint8_t *, float *, void *);
typedef int (*select_fn)(const void *, int64_t, const void *, int64_t, const int32_t *, const int32_t *, int64_t,
                         int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int, int64_t,
                         int32_t *, float *, void *, int64_t, void *);
typedef int (*blocks_fn)(const void *, int64_t, const void *, int64_t, const void *, int64_t, const int32_t *,
                         const int32_t *, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                         const int32_t *, int64_t, int, float, void *, float *, void *);
static write_fn g_write;
static read_fn g_read;
static cached_fn g_cached;
static varlen_fn g_varlen;
static axes_fn g_axes;
static postnorm_fn g_postnorm;
static select_fn g_select;
static blocks_fn g_blocks;

/* One tensor as the calls see it. */
typedef struct {
    void *ptr;
    int nd;
    int64_t dim[MAX_DIMS];
    int64_t stride[MAX_DIMS]; /* where asked for */
} View;

static int attr_is(PyObject *o, PyObject *name, PyObject *want)
{
    PyObject *v = PyObject_GetAttr(o, name);
    int same = v == want;
    Py_XDECREF(v);
    return same;
}

/* Whether the tensor is on this device. */
static int on_device(PyObject *t, PyObject *device)
{
    PyObject *d = PyObject_GetAttr(t, s_device);
    if (d == NULL) return 0;
    int same = d == device || PyObject_RichCompareBool(d, device, Py_EQ) == 1;
    Py_DECREF(d);
    return same;
}

/* The tensor's dimensions, if it is one of this dtype with nd of them on this device. */
static int look(PyObject *t, PyObject *dtype, PyObject *device, int nd, View *v)
{
    if (Py_TYPE(t) != (PyTypeObject *)g_tensor && !PyType_IsSubtype(Py_TYPE(t), (PyTypeObject *)g_tensor)) return 0;
    if (!attr_is(t, s_dtype, dtype) || !on_device(t, device)) return 0;
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    if (shape == NULL || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) != nd) {
        Py_XDECREF(shape);
        return 0;
    }
    v->nd = nd;
    for (int i = 0; i < nd; ++i) v->dim[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    Py_DECREF(shape);
    PyObject *p = PyObject_VectorcallMethod(s_data_ptr, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    if (p == NULL) return 0;
    v->ptr = PyLong_AsVoidPtr(p);
    Py_DECREF(p);
    return !PyErr_Occurred();
}

/* A contiguous tensor of this shape (-1: any extent). */
static int dense(PyObject *t, PyObject *dtype, PyObject *device, int nd, const int64_t *dim, View *v)
{
    if (!look(t, dtype, device, nd, v)) return 0;
    for (int i = 0; i < nd; ++i)
        if (dim[i] >= 0 && v->dim[i] != dim[i]) return 0;
    PyObject *c = PyObject_VectorcallMethod(s_contiguous, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    int yes = c == Py_True;
    Py_XDECREF(c);
    return yes;
}

/* bf16 [rows, heads, dim] with contiguous rows; the row stride in *ld. */
static int head_rows(PyObject *t, PyObject *device, View *v, int64_t *ld)
{
    if (!look(t, g_bf16, device, 3, v)) return 0;
    PyObject *st = PyObject_VectorcallMethod(s_stride, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    if (st == NULL || !PyTuple_Check(st) || PyTuple_GET_SIZE(st) != 3) {
        Py_XDECREF(st);
        return 0;
    }
    for (int i = 0; i < 3; ++i) v->stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    Py_DECREF(st);
    if ((v->dim[2] > 1 && v->stride[2] != 1) || (v->dim[1] > 1 && v->stride[1] != v->dim[2])) return 0;
    *ld = v->dim[0] > 1 ? v->stride[0] : v->dim[1] * v->dim[2];
    return !PyErr_Occurred();
}

/* One fp32 value of any shape. */
static int one_float(PyObject *t, PyObject *device, void **p)
{
    if (Py_TYPE(t) != (PyTypeObject *)g_tensor && !PyType_IsSubtype(Py_TYPE(t), (PyTypeObject *)g_tensor)) return 0;
    if (!attr_is(t, s_dtype, g_f32)) return 0;
    PyObject *d = PyObject_GetAttr(t, s_device);
    if (d == NULL) return 0;
    int same = PyObject_RichCompareBool(d, device, Py_EQ);
    Py_DECREF(d);
    if (same != 1) return 0;
    PyObject *n = PyObject_VectorcallMethod(s_numel, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    if (n == NULL) return 0;
    int is_one = PyLong_AsLongLong(n) == 1;
    Py_DECREF(n);
    if (!is_one) return 0;
    PyObject *a = PyObject_VectorcallMethod(s_data_ptr, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    if (a == NULL) return 0;
    *p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return !PyErr_Occurred();
}

/* The four cache tensors: dims pages, heads, page, head_dim. */
static int cache_of(PyObject *cache, PyObject *device, void *p[4], int64_t dims[4])
{
    if (!PyTuple_CheckExact(cache) || PyTuple_GET_SIZE(cache) != 4) return 0;
    int64_t codes[4] = {-1, -1, -1, -1}, scales[4];
    for (int i = 0; i < 4; ++i) {
        View v;
        if (!dense(PyTuple_GET_ITEM(cache, i), g_u8, device, 4, i % 2 ? scales : codes, &v)) return 0;
        p[i] = v.ptr;
        if (i == 0) {
            for (int k = 0; k < 4; ++k) codes[k] = scales[k] = v.dim[k];
            if (v.dim[3] % 8) return 0;
            scales[3] = v.dim[3] / 8;
        }
    }
    dims[0] = codes[0], dims[1] = codes[1], dims[2] = codes[2], dims[3] = 2 * codes[3];
    return 1;
}

static int lists_of(PyObject *cu, PyObject *len, PyObject *table, PyObject *device, void *p[3], int64_t *batch,
                    int64_t *max_pages)
{
    View v;
    int64_t d[2] = {-1, -1};
    if (!dense(len, g_i32, device, 1, d, &v)) return 0;
    p[1] = v.ptr;
    *batch = d[0] = v.dim[0];
    if (!dense(table, g_i32, device, 2, d, &v)) return 0;
    p[2] = v.ptr;
    *max_pages = v.dim[1];
    d[0] = *batch + 1;
    if (!dense(cu, g_i32, device, 1, d, &v)) return 0;
    p[0] = v.ptr;
    return 1;
}

/* The device is CUDA's current one; the handle of its current stream, or of the one given as a number. */
static int stream_of(PyObject *device, PyObject *stream, void **handle)
{
    PyObject *type = PyObject_GetAttr(device, s_type);
    int cuda = type != NULL && PyUnicode_Check(type) && PyUnicode_Compare(type, s_cuda) == 0;
    Py_XDECREF(type);
    if (!cuda) return 0;
    PyObject *index = PyObject_GetAttr(device, s_index), *current = NULL, *raw = NULL;
    int ok = 0;
    if (index != NULL && PyLong_Check(index) && (current = PyObject_CallNoArgs(g_get_device)) != NULL &&
        PyLong_AsLong(current) == PyLong_AsLong(index)) {
        if (stream != Py_None) {
            Py_INCREF(stream);
            raw = stream;
        } else {
            raw = PyObject_CallOneArg(g_get_stream, index);
        }
        if (raw != NULL && PyLong_Check(raw)) {
            *handle = PyLong_AsVoidPtr(raw);
            ok = !PyErr_Occurred();
        }
    }
    Py_XDECREF(index);
    Py_XDECREF(current);
    Py_XDECREF(raw);
    return ok;
}

static PyObject *give_up(void)
{
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* write(k, v, cache, cu_rows, kv_len, block_table, k_scale, v_scale, device, stream) */
static PyObject *py_write(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *c[4], *l[3], *kg, *vg, *stream;
    int64_t dims[4], batch, max_pages, ld_k, ld_v;
    View k, v;
    if (n != 10 || !cache_of(a[2], a[8], c, dims) || !head_rows(a[0], a[8], &k, &ld_k) ||
        !head_rows(a[1], a[8], &v, &ld_v) || k.dim[1] != dims[1] || k.dim[2] != dims[3] || v.dim[0] != k.dim[0] ||
        v.dim[1] != dims[1] || v.dim[2] != dims[3] || !lists_of(a[3], a[4], a[5], a[8], l, &batch, &max_pages) ||
        !one_float(a[6], a[8], &kg) || !one_float(a[7], a[8], &vg) || !stream_of(a[8], a[9], &stream))
        return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_write(k.ptr, ld_k, v.ptr, ld_v, k.dim[0], l[0], l[1], l[2], batch, max_pages, kg, vg, c[0], c[1], c[2],
                 c[3], dims[0], dims[2], dims[1], dims[3], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* read(cache, cu_rows, kv_len, block_table, k_scale, v_scale, k_out, v_out, device, stream) */
static PyObject *py_read(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *c[4], *l[3], *kg, *vg, *stream;
    int64_t dims[4], batch, max_pages;
    View k, v;
    if (n != 10 || !cache_of(a[0], a[8], c, dims) || !lists_of(a[1], a[2], a[3], a[8], l, &batch, &max_pages) ||
        !one_float(a[4], a[8], &kg) || !one_float(a[5], a[8], &vg))
        return give_up();
    int64_t d[3] = {-1, dims[1], dims[3]};
    if (!dense(a[6], g_bf16, a[8], 3, d, &k)) return give_up();
    d[0] = k.dim[0];
    if (!dense(a[7], g_bf16, a[8], 3, d, &v) || !stream_of(a[8], a[9], &stream)) return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_read(c[0], c[1], c[2], c[3], dims[0], dims[2], dims[1], dims[3], kg, vg, k.dim[0], l[0], l[1], l[2], batch,
                max_pages, k.ptr, v.ptr, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* Optional fp32 [heads, rows]. */
static int lse_of(PyObject *t, PyObject *device, int64_t heads, int64_t rows, void **p)
{
    *p = NULL;
    if (t == Py_None) return 1;
    View v;
    const int64_t d[2] = {heads, rows};
    if (!dense(t, g_f32, device, 2, d, &v)) return 0;
    *p = v.ptr;
    return 1;
}

/* cached(q, cache, cu_rows, kv_len, block_table, k_scale, v_scale, max_rows, tree_mask, scale, out, lse,
 *        workspace, device, stream) */
static PyObject *py_cached(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *c[4], *l[3], *kg, *vg, *stream, *lse, *mask = NULL;
    int64_t dims[4], batch, max_pages, ld;
    View q, v, o, w;
    if (n != 15 || !cache_of(a[1], a[13], c, dims) || !head_rows(a[0], a[13], &q, &ld) || q.dim[2] != dims[3] ||
        !lists_of(a[2], a[3], a[4], a[13], l, &batch, &max_pages) || !one_float(a[5], a[13], &kg) ||
        !one_float(a[6], a[13], &vg) || !PyLong_CheckExact(a[7]) || !PyFloat_CheckExact(a[9]))
        return give_up();
    if (a[8] != Py_None) {
        if (!dense(a[8], g_i64, a[13], 1, q.dim, &v)) return give_up();
        mask = v.ptr;
    }
    const int64_t any = -1;
    if (!dense(a[10], g_bf16, a[13], 3, q.dim, &o) || !lse_of(a[11], a[13], q.dim[1], q.dim[0], &lse) ||
        !dense(a[12], g_u8, a[13], 1, &any, &w) || !stream_of(a[13], a[14], &stream))
        return give_up();
    const int64_t max_rows = PyLong_AsLongLong(a[7]);
    const float scale = (float)PyFloat_AS_DOUBLE(a[9]);
    if (PyErr_Occurred()) return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_cached(q.ptr, ld, q.dim[0], q.dim[1], max_rows, l[0], l[1], l[2], batch, max_pages, mask, c[0], c[1], c[2],
                  c[3], dims[0], dims[2], dims[1], dims[3], kg, vg, scale, o.ptr, lse, w.ptr, w.dim[0], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* varlen(q, k, v, cu_q, cu_k, causal, scale, out, lse, device, stream) */
static PyObject *py_varlen(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    void *lse, *stream;
    int64_t ld_q, ld_k, ld_v, d = -1;
    View q, k, v, cq, ck, o;
    if (n != 11 || !head_rows(a[0], a[9], &q, &ld_q) || !head_rows(a[1], a[9], &k, &ld_k) ||
        !head_rows(a[2], a[9], &v, &ld_v) || k.dim[2] != q.dim[2] || v.dim[0] != k.dim[0] || v.dim[1] != k.dim[1] ||
        v.dim[2] != k.dim[2] || !dense(a[3], g_i32, a[9], 1, &d, &cq) || cq.dim[0] < 1 ||
        !dense(a[4], g_i32, a[9], 1, cq.dim, &ck) || !PyFloat_CheckExact(a[6]) ||
        !dense(a[7], g_bf16, a[9], 3, q.dim, &o) || !lse_of(a[8], a[9], q.dim[1], q.dim[0], &lse) ||
        !stream_of(a[9], a[10], &stream))
        return give_up();
    const int causal = a[5] == Py_True;
    const float scale = (float)PyFloat_AS_DOUBLE(a[6]);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_varlen(q.ptr, ld_q, k.ptr, ld_k, v.ptr, ld_v, cq.ptr, ck.ptr, cq.dim[0] - 1, q.dim[0], k.dim[0], q.dim[1],
                  k.dim[1], q.dim[2], causal, scale, o.ptr, lse, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* [rows, cols] with contiguous rows; the row stride in *ld. */
static int flat_rows(PyObject *t, PyObject *dtype, PyObject *device, View *v, int64_t *ld)
{
    if (!look(t, dtype, device, 2, v)) return 0;
    PyObject *st = PyObject_VectorcallMethod(s_stride, &t, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
    if (st == NULL || !PyTuple_Check(st) || PyTuple_GET_SIZE(st) != 2) {
        Py_XDECREF(st);
        return 0;
    }
    for (int i = 0; i < 2; ++i) v->stride[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    Py_DECREF(st);
    if (v->dim[1] > 1 && v->stride[1] != 1) return 0;
    *ld = v->dim[0] > 1 ? v->stride[0] : v->dim[1];
    return !PyErr_Occurred();
}

/* An optional contiguous tensor of this shape. */
static int dense_or_none(PyObject *t, PyObject *dtype, PyObject *device, int nd, const int64_t *dim, void **p)
{
    *p = NULL;
    if (t == Py_None) return 1;
    View v;
    if (!dense(t, dtype, device, nd, dim, &v)) return 0;
    *p = v.ptr;
    return 1;
}

/* A whole number (Python's own); a number. */
static int whole(PyObject *o, int64_t *v)
{
    if (!PyLong_CheckExact(o)) return 0;
    *v = PyLong_AsLongLong(o);
    return !PyErr_Occurred();
}
static int number(PyObject *o, double *v)
{
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) return 0;
    *v = PyFloat_AsDouble(o);
    return !PyErr_Occurred();
}

#define MAX_AXES 4

/* A number for all axes, or a tuple or list of one for each. */
static int per_axis(PyObject *o, int64_t axes, double *v)
{
    if (number(o, v)) {
        for (int64_t i = 1; i < axes; ++i) v[i] = v[0];
        return 1;
    }
    if ((!PyTuple_CheckExact(o) && !PyList_CheckExact(o)) || PySequence_Fast_GET_SIZE(o) != axes) return 0;
    for (int64_t i = 0; i < axes; ++i)
        if (!number(PySequence_Fast_GET_ITEM(o, i), v + i)) return 0;
    return 1;
}

/* A tuple or list of n, or None for n times None. */
static int items_of(PyObject *o, Py_ssize_t n, PyObject **items)
{
    if (o != Py_None && ((!PyTuple_CheckExact(o) && !PyList_CheckExact(o)) || PySequence_Fast_GET_SIZE(o) != n)) return 0;
    for (Py_ssize_t i = 0; i < n; ++i) items[i] = o == Py_None ? Py_None : PySequence_Fast_GET_ITEM(o, i);
    return 1;
}

/* axes(q, k, v, positions, axis_dims, heads, kv_heads, theta, scale, sections, biases, weights, norm, eps,
 *      interleaved, outs, device, stream) */
static PyObject *py_axes(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View x[3], p, o;
    int64_t ld[3], heads[3], dims[MAX_AXES];
    double theta[MAX_AXES], scale[MAX_AXES], eps;
    void *bias[3], *weight[2], *out[3], *stream;
    PyObject *items[3];
    if (n != 18 || !whole(a[5], &heads[0]) || !whole(a[6], &heads[1]) || heads[0] < 1 || heads[1] < 1 || !number(a[13], &eps))
        return give_up();
    heads[2] = heads[1];
    for (int i = 0; i < 3; ++i)
        if (!flat_rows(a[i], g_bf16, a[16], &x[i], &ld[i])) return give_up();
    const int64_t rows = x[0].dim[0], hd = x[0].dim[1] / heads[0];
    for (int i = 0; i < 3; ++i)
        if (x[i].dim[0] != rows || x[i].dim[1] != heads[i] * hd) return give_up();
    if (!PyTuple_CheckExact(a[4]) && !PyList_CheckExact(a[4])) return give_up();
    const int64_t axes = PySequence_Fast_GET_SIZE(a[4]);
    if (axes < 1 || axes > MAX_AXES) return give_up();
    for (int64_t i = 0; i < axes; ++i)
        if (!whole(PySequence_Fast_GET_ITEM(a[4], i), dims + i)) return give_up();
    const int64_t at[2] = {rows, axes};
    if (!dense(a[3], g_i32, a[16], 2, at, &p) || !per_axis(a[7], axes, theta) || !per_axis(a[8], axes, scale) ||
        !items_of(a[10], 3, items))
        return give_up();
    for (int i = 0; i < 3; ++i)
        if (!dense_or_none(items[i], g_bf16, a[16], 1, &x[i].dim[1], &bias[i])) return give_up();
    if (!items_of(a[11], 2, items)) return give_up();
    for (int i = 0; i < 2; ++i)
        if (!dense_or_none(items[i], g_bf16, a[16], 1, &hd, &weight[i])) return give_up();
    if (a[15] == Py_None || !items_of(a[15], 3, items)) return give_up();
    for (int i = 0; i < 3; ++i) {
        const int64_t d[3] = {rows, heads[i], hd};
        if (!dense(items[i], g_bf16, a[16], 3, d, &o)) return give_up();
        out[i] = o.ptr;
    }
    const int sections = PyObject_IsTrue(a[9]), norm = PyObject_IsTrue(a[12]), pairs = PyObject_IsTrue(a[14]);
    if (sections < 0 || norm < 0 || pairs < 0 || !stream_of(a[16], a[17], &stream)) return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_axes(x[0].ptr, ld[0], x[1].ptr, ld[1], x[2].ptr, ld[2], bias[0], bias[1], bias[2], weight[0], weight[1],
                p.ptr, axes, dims, theta, scale, sections, pairs, norm, rows, heads[0], heads[1], hd, (float)eps, out[0],
                out[1], out[2], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* postnorm(h, o, gamma_post, gamma, global_scale, bias, gate_table, mod_table, residual_scale, row_frame,
 *          rows_per_frame, eps, codes, scales, row_rstd, device, stream) */
static PyObject *py_postnorm(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View h, o, post, gamma, codes, scales, gate, table;
    int64_t ld_h, ld_o, frames = 0, per = 0;
    double keep, eps;
    void *gsf, *bias, *frame = NULL, *rstd, *stream;
    if (n != 17 || !flat_rows(a[0], g_f32, a[15], &h, &ld_h) || !flat_rows(a[1], g_bf16, a[15], &o, &ld_o) ||
        o.dim[0] != h.dim[0] || o.dim[1] != h.dim[1] || !number(a[8], &keep) || !number(a[11], &eps))
        return give_up();
    const int64_t rows = h.dim[0], cols = h.dim[1];
    if (!dense(a[2], g_bf16, a[15], 1, &cols, &post) || !dense(a[3], g_bf16, a[15], 1, &cols, &gamma) ||
        !one_float(a[4], a[15], &gsf) || !dense_or_none(a[5], g_bf16, a[15], 1, &cols, &bias))
        return give_up();
    gate.ptr = table.ptr = NULL;
    if (a[6] != Py_None) {
        const int64_t d[2] = {-1, cols};
        if (!dense(a[6], g_bf16, a[15], 2, d, &gate)) return give_up();
        frames = gate.dim[0];
    }
    if (a[7] != Py_None) {
        const int64_t d[3] = {a[6] != Py_None ? frames : -1, 2, cols};
        if (!dense(a[7], g_bf16, a[15], 3, d, &table)) return give_up();
        frames = table.dim[0];
    }
    if (gate.ptr != NULL || table.ptr != NULL) {
        if (a[9] != Py_None) {
            if (!dense_or_none(a[9], g_i32, a[15], 1, &rows, &frame)) return give_up();
        } else if (!whole(a[10], &per)) {
            return give_up();
        }
    }
    const int64_t c[2] = {rows, cols / 2}, s[2] = {(rows + 127) / 128 * 128, cols / 16};
    if (!dense(a[12], g_u8, a[15], 2, c, &codes) || !dense(a[13], g_u8, a[15], 2, s, &scales) ||
        !dense_or_none(a[14], g_f32, a[15], 1, &rows, &rstd) || !stream_of(a[15], a[16], &stream))
        return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_postnorm(h.ptr, ld_h, o.ptr, ld_o, bias, post.ptr, gate.ptr, (float)keep, gamma.ptr, table.ptr, frames, frame,
                    per, (float)eps, rows, cols, gsf, codes.ptr, scales.ptr, rstd, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* Packed sequences with blocks: q and k, their offsets. */
static int block_sequences(PyObject *q, PyObject *k, PyObject *cu_q, PyObject *cu_k, PyObject *device, View *vq, View *vk,
                           int64_t *ld_q, int64_t *ld_k, View *cq, View *ck)
{
    const int64_t any = -1;
    return head_rows(q, device, vq, ld_q) && head_rows(k, device, vk, ld_k) && vk->dim[2] == vq->dim[2] &&
           dense(cu_q, g_i32, device, 1, &any, cq) && cq->dim[0] >= 1 && dense(cu_k, g_i32, device, 1, cq->dim, ck);
}

/* select(q, k, cu_q, cu_k, top, block_q, block_k, causal, first, blocks, scores, workspace, device, stream) */
static PyObject *py_select(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View q, k, cq, ck, b, w;
    int64_t ld_q, ld_k, top, block_q, block_k, first;
    void *scores, *stream;
    const int64_t any = -1;
    if (n != 14 || !whole(a[4], &top) || !whole(a[5], &block_q) || !whole(a[6], &block_k) || !whole(a[8], &first) ||
        block_q < 1 || block_k < 1 || !block_sequences(a[0], a[1], a[2], a[3], a[12], &q, &k, &ld_q, &ld_k, &cq, &ck))
        return give_up();
    const int64_t d[3] = {k.dim[1], h3q_block_rows(q.dim[0], cq.dim[0] - 1, block_q), top};
    if (!dense(a[9], g_i32, a[12], 3, d, &b) || !dense_or_none(a[10], g_f32, a[12], 3, d, &scores) ||
        !dense(a[11], g_u8, a[12], 1, &any, &w) || !stream_of(a[12], a[13], &stream))
        return give_up();
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) return give_up();
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_select(q.ptr, ld_q, k.ptr, ld_k, cq.ptr, ck.ptr, cq.dim[0] - 1, q.dim[0], k.dim[0], q.dim[1], k.dim[1], q.dim[2],
                  block_q, block_k, top, causal, first, b.ptr, scores, w.ptr, w.dim[0], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* blocks(q, k, v, cu_q, cu_k, lists, block_q, block_k, causal, scale, out, lse, device, stream) */
static PyObject *py_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    View q, k, v, cq, ck, b, o;
    int64_t ld_q, ld_k, ld_v, block_q, block_k;
    void *lse, *stream;
    if (n != 14 || !whole(a[6], &block_q) || !whole(a[7], &block_k) || block_q < 1 || block_k < 1 ||
        !PyFloat_CheckExact(a[9]) || !block_sequences(a[0], a[1], a[3], a[4], a[12], &q, &k, &ld_q, &ld_k, &cq, &ck) ||
        !head_rows(a[2], a[12], &v, &ld_v) || v.dim[0] != k.dim[0] || v.dim[1] != k.dim[1] || v.dim[2] != k.dim[2])
        return give_up();
    const int64_t d[3] = {k.dim[1], h3q_block_rows(q.dim[0], cq.dim[0] - 1, block_q), -1};
    if (!dense(a[5], g_i32, a[12], 3, d, &b) || !dense(a[10], g_bf16, a[12], 3, q.dim, &o) ||
        !lse_of(a[11], a[12], q.dim[1], q.dim[0], &lse) || !stream_of(a[12], a[13], &stream))
        return give_up();
    const int causal = PyObject_IsTrue(a[8]);
    if (causal < 0) return give_up();
    const float scale = (float)PyFloat_AS_DOUBLE(a[9]);
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = g_blocks(q.ptr, ld_q, k.ptr, ld_k, v.ptr, ld_v, cq.ptr, ck.ptr, cq.dim[0] - 1, q.dim[0], k.dim[0], q.dim[1],
                  k.dim[1], q.dim[2], block_q, block_k, b.ptr, b.dim[2], causal, scale, o.ptr, lse, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

/* setup_blocks(axes, postnorm, select, blocks): the addresses of more of the library's functions. */
static PyObject *py_setup_blocks(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n != 4) {
        PyErr_SetString(PyExc_TypeError, "setup_blocks takes four addresses");
        return NULL;
    }
    g_axes = (axes_fn)PyLong_AsVoidPtr(a[0]);
    g_postnorm = (postnorm_fn)PyLong_AsVoidPtr(a[1]);
    g_select = (select_fn)PyLong_AsVoidPtr(a[2]);
    g_blocks = (blocks_fn)PyLong_AsVoidPtr(a[3]);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

/* setup(Tensor, bfloat16, uint8, int32, int64, float32, get_device, get_stream, write, read, cached, varlen): torch's
 * objects, and the addresses of the library's functions. */
static PyObject *py_setup(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n != 12 || !PyType_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "setup takes torch.Tensor, five dtypes, two functions and four addresses");
        return NULL;
    }
    PyObject **keep[8] = {&g_tensor, &g_bf16, &g_u8, &g_i32, &g_i64, &g_f32, &g_get_device, &g_get_stream};
    for (int i = 0; i < 8; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*keep[i], a[i]);
    }
    g_write = (write_fn)PyLong_AsVoidPtr(a[8]);
    g_read = (read_fn)PyLong_AsVoidPtr(a[9]);
    g_cached = (cached_fn)PyLong_AsVoidPtr(a[10]);
    g_varlen = (varlen_fn)PyLong_AsVoidPtr(a[11]);
    if (PyErr_Occurred()) return NULL;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))py_setup, METH_FASTCALL, "torch's objects and the library's functions"},
    {"write", (PyCFunction)(void (*)(void))py_write, METH_FASTCALL, "h3q_kv_cache_write_nvfp4, or None"},
    {"read", (PyCFunction)(void (*)(void))py_read, METH_FASTCALL, "h3q_kv_cache_read_nvfp4, or None"},
    {"cached", (PyCFunction)(void (*)(void))py_cached, METH_FASTCALL, "h3q_attention_cache_nvfp4, or None"},
    {"varlen", (PyCFunction)(void (*)(void))py_varlen, METH_FASTCALL, "h3q_attention_varlen, or None"},
    {"setup_blocks", (PyCFunction)(void (*)(void))py_setup_blocks, METH_FASTCALL, "more of the library's functions"},
    {"axes", (PyCFunction)(void (*)(void))py_axes, METH_FASTCALL, "h3q_qkv_epilogue_axes, or None"},
    {"postnorm", (PyCFunction)(void (*)(void))py_postnorm, METH_FASTCALL, "h3q_postnorm_residual_adaln_nvfp4, or None"},
    {"select", (PyCFunction)(void (*)(void))py_select, METH_FASTCALL, "h3q_select_blocks, or None"},
    {"blocks", (PyCFunction)(void (*)(void))py_blocks, METH_FASTCALL, "h3q_attention_blocks, or None"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "h3q_binding", "The short way into the library's calls.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_h3q_binding(void)
{
    struct {
        PyObject **at;
        const char *name;
    } names[] = {{&s_dtype, "dtype"}, {&s_device, "device"}, {&s_shape, "shape"}, {&s_index, "index"},
                 {&s_type, "type"}, {&s_cuda, "cuda"}, {&s_contiguous, "is_contiguous"}, {&s_data_ptr, "data_ptr"},
                 {&s_stride, "stride"}, {&s_numel, "numel"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if ((*names[i].at = PyUnicode_InternFromString(names[i].name)) == NULL) return NULL;
    return PyModule_Create(&module);
}
