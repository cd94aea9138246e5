/* call.c — the common form of the serving calls of the binding (module _call), without the interpreter
 * between the argument checks and the C ABI.
 *
 * Each function takes what the public function of the same name takes, in the form without `out`,
 * `ws` and `stream`: it checks the arguments, allocates the results with torch.empty and calls the
 * library on the current stream. Anything it does not recognise (a layout, type or device that has to
 * be refused, an Fp4 or Route that is a subclass) makes it return NotImplemented; the public function then
 * goes through the checks in Python, which has the messages. Tensors are known by what they answer (device,
 * type, shape, strides, address), so a subclass that answers as a tensor does is read as one.
 * A one-token linear layer is two such calls; in Python they took 27 us of host time, more than the kernels.
 * A combination takes 6.8 us here: 2.2 in the library, mostly the launch, 1.5 for the result's allocation,
 * the rest for what five tensors are asked.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "gptq.h"

static PyObject *s_dtype, *s_get_device, *s_shape, *s_stride, *s_data_ptr, *s_device, *s_is_contiguous, *s_mx, *s_nv;
static PyObject *o_f32, *o_bf16, *o_u8, *o_i32, *f_empty, *f_raw_stream, *f_current_device, *t_fp4, *t_route, *f_check;
static PyObject* k_empty; /* ("dtype", "device") */

static int (*p_quantize)(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int64_t, int64_t, int, const float*, uint8_t*,
                         uint8_t*, void*);
static int (*p_dequantize)(const uint8_t*, const uint8_t*, const float*, int64_t, int64_t, int, void*, int, int64_t, void*);
static int (*p_matmul)(const uint8_t*, const uint8_t*, const float*, int64_t, const uint8_t*, const uint8_t*, const float*, int64_t,
                       int64_t, int, const int32_t*, int64_t, int, void*, int64_t, void*);
static size_t (*p_sort_ws)(int64_t, int64_t, int64_t);
static int (*p_sort)(const int32_t*, int64_t, int64_t, int64_t, int32_t*, int32_t*, int32_t*, void*, size_t, void*);
static int (*p_gather)(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int64_t, const int32_t*, int64_t, void*, int64_t,
                       void*);
static int (*p_combine)(const void*, int, int64_t, int64_t, int64_t, const int32_t*, int64_t, const float*, void*, int64_t, void*);
static int (*p_combine_grad)(const void*, int64_t, const void*, int64_t, int, int64_t, int64_t, const int32_t*, int64_t,
                             const int32_t*, int64_t, const float*, void*, int64_t, float*, void*);

/* The device that a call of this thread launches on; its tensors have to be there. */
static _Thread_local long here;

static void find_device(void) {
    PyObject* d = PyObject_CallNoArgs(f_current_device);
    here = d ? PyLong_AsLong(d) : -2;   /* -1 is the host */
    Py_XDECREF(d);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        here = -2;
    }
}

/* ------------------------------------------------------------------------------ what a tensor is */

typedef struct {
    void* ptr;
    PyObject* dtype; /* borrowed: torch's dtypes live as long as the process */
    int dims;
    int64_t shape[4];
    int64_t ld; /* of two dimensions: the row stride */
} Tensor;

/* Reads t; `rows`: two dimensions whose rows are contiguous (any row stride), otherwise contiguous as a
 * whole. 0: not that, or not on the device of the call. */
static int read_tensor(PyObject* t, int rows, Tensor* out) {
    int ok = 0;
    PyObject *device = PyObject_CallMethodNoArgs(t, s_get_device), *dtype = NULL, *shape = NULL, *stride = NULL, *ptr = NULL;
    if (!device || PyLong_AsLong(device) != here) goto done;
    dtype = PyObject_GetAttr(t, s_dtype);
    shape = PyObject_GetAttr(t, s_shape);
    if (!dtype || !shape || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) > 4) goto done;
    out->dtype = dtype;
    out->dims = (int)PyTuple_GET_SIZE(shape);
    for (int i = 0; i < out->dims; ++i) out->shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    if (rows) {
        if (out->dims != 2) goto done;
        stride = PyObject_CallMethodNoArgs(t, s_stride);
        if (!stride || !PyTuple_Check(stride) || PyTuple_GET_SIZE(stride) != 2) goto done;
        const int64_t ld = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0)), one = PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1));
        if ((one != 1 && out->shape[1] > 1) || (out->shape[0] > 1 && ld < out->shape[1])) goto done;
        out->ld = out->shape[0] > 1 ? ld : out->shape[1] > 1 ? out->shape[1] : 1;
    } else {
        stride = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (stride != Py_True) goto done;
    }
    ptr = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!ptr) goto done;
    out->ptr = PyLong_AsVoidPtr(ptr);
    ok = 1;
done:
    Py_XDECREF(device);
    Py_XDECREF(dtype);
    Py_XDECREF(shape);
    Py_XDECREF(stride);
    Py_XDECREF(ptr);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        ok = 0;
    }
    return ok;
}

static int dtype_code(PyObject* d) { return d == o_bf16 ? GPTQ_BF16 : d == o_f32 ? GPTQ_F32 : -1; }

/* a matrix of bf16 or fp32 rows */
static int read_matrix(PyObject* t, Tensor* out) { return read_tensor(t, 1, out) && dtype_code(out->dtype) >= 0; }

static int read_typed(PyObject* t, PyObject* dtype, int dims, Tensor* out) {
    return read_tensor(t, 0, out) && out->dtype == dtype && out->dims == dims;
}

static int format_code(PyObject* f) {
    if (f == s_mx) return GPTQ_MXFP4;
    if (f == s_nv) return GPTQ_NVFP4;
    if (!PyUnicode_Check(f)) return -1;
    return PyUnicode_Compare(f, s_mx) == 0 ? GPTQ_MXFP4 : PyUnicode_Compare(f, s_nv) == 0 ? GPTQ_NVFP4 : -1;
}

typedef struct {
    Tensor codes, scales, g;
    int64_t experts, rows, cols, gs; /* gs: how many tensor scales */
    int format;
} Fp4;

/* experts: -1 for a single matrix */
static int read_fp4(PyObject* q, int experts, Fp4* f) {
    if (Py_TYPE(q) != (PyTypeObject*)t_fp4 || PyTuple_GET_SIZE(q) != 5) return 0;
    const int lead = experts ? 1 : 0;
    PyObject* cols = PyTuple_GET_ITEM(q, 2);
    f->format = format_code(PyTuple_GET_ITEM(q, 3));
    if (f->format < 0 || !PyLong_Check(cols) || !read_typed(PyTuple_GET_ITEM(q, 0), o_u8, 2 + lead, &f->codes) ||
        !read_typed(PyTuple_GET_ITEM(q, 1), o_u8, 3 + lead, &f->scales))
        return 0;
    f->cols = PyLong_AsLongLong(cols);
    if (PyErr_Occurred()) {   /* past 64 bits */
        PyErr_Clear();
        return 0;
    }
    const int64_t *c = f->codes.shape + lead, *s = f->scales.shape + lead, span = f->format == GPTQ_MXFP4 ? 128 : 64;
    f->rows = c[0];
    f->experts = lead ? f->codes.shape[0] : 1;
    if (f->cols < 0 || c[1] != (f->cols + 31) / 32 * 16 || s[0] != (f->rows + 127) / 128 || s[1] != (f->cols + span - 1) / span ||
        s[2] != 512 || (lead && f->scales.shape[0] != f->experts))
        return 0;
    f->g.ptr = NULL;
    f->gs = 0;
    if (f->format == GPTQ_NVFP4) {
        if (!read_typed(PyTuple_GET_ITEM(q, 4), o_f32, 1, &f->g)) return 0;
        f->gs = f->g.shape[0];
        if (f->gs != 1 && f->gs != f->experts) return 0;
    }
    return 1;
}

typedef struct {
    Tensor offsets, src, pos;
    int64_t tokens, top, experts;
} Route;

static int read_route(PyObject* r, Route* o) {
    if (Py_TYPE(r) != (PyTypeObject*)t_route || PyTuple_GET_SIZE(r) != 3 ||
        !read_typed(PyTuple_GET_ITEM(r, 0), o_i32, 1, &o->offsets) || !read_typed(PyTuple_GET_ITEM(r, 1), o_i32, 1, &o->src) ||
        !read_typed(PyTuple_GET_ITEM(r, 2), o_i32, 2, &o->pos))
        return 0;
    o->tokens = o->pos.shape[0];
    o->top = o->pos.shape[1];
    o->experts = o->offsets.shape[0] - 1;
    return o->src.shape[0] == o->tokens * o->top && o->experts >= 1;
}

/* ---------------------------------------------------------------------------- results and calls */

/* torch.empty(shape, dtype=dtype, device=like.device); *ptr its address */
static PyObject* empty(int dims, const int64_t* shape, PyObject* dtype, PyObject* like, void** ptr) {
    PyObject *t = NULL, *p = NULL, *size = PyTuple_New(dims), *device = PyObject_GetAttr(like, s_device);
    if (size && device) {
        for (int i = 0; i < dims; ++i) PyTuple_SET_ITEM(size, i, PyLong_FromLongLong(shape[i]));
        PyObject* args[3] = {size, dtype, device};
        t = PyErr_Occurred() ? NULL : PyObject_Vectorcall(f_empty, args, 1, k_empty);
    }
    if (t) {
        p = PyObject_CallMethodNoArgs(t, s_data_ptr);
        if (p) *ptr = PyLong_AsVoidPtr(p);
        if (PyErr_Occurred()) Py_CLEAR(t);
    }
    Py_XDECREF(size);
    Py_XDECREF(device);
    Py_XDECREF(p);
    return t;
}

static int current_stream(void** s) {
    PyObject *d = PyLong_FromLong(here), *v = d ? PyObject_CallOneArg(f_raw_stream, d) : NULL;
    if (v) *s = PyLong_AsVoidPtr(v);
    Py_XDECREF(d);
    Py_XDECREF(v);
    return PyErr_Occurred() ? 0 : 1;
}

/* raises for a status other than 0 */
static int check(const char* fn, int status) {
    if (status == 0) return 1;
    PyObject* r = PyObject_CallFunction(f_check, "si", fn, status);
    Py_XDECREF(r);
    return 0;
}

/* an instance of a named tuple; steals the references */
static PyObject* named(PyObject* type, int n, PyObject** items) {
    PyObject *values = PyTuple_New(n), *args = NULL, *r = NULL;
    for (int i = 0; i < n; ++i) {
        if (values) PyTuple_SET_ITEM(values, i, items[i]);
        else Py_XDECREF(items[i]);
    }
    if (values) args = PyTuple_Pack(1, values);
    if (args) r = PyTuple_Type.tp_new((PyTypeObject*)type, args, NULL);
    Py_XDECREF(args);
    Py_XDECREF(values);
    return r;
}

#define CALL(status, expr)       \
    Py_BEGIN_ALLOW_THREADS       \
    status = (expr);             \
    Py_END_ALLOW_THREADS

/* quantize(X, format, tensor_scale, index, per) */
static PyObject* quantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Tensor x, g = {0}, index = {0};
    if (n != 5) Py_RETURN_NOTIMPLEMENTED;
    const int f = format_code(a[1]);
    const int has_index = a[3] != Py_None;
    int64_t per = 1;
    if (f < 0 || !read_matrix(a[0], &x)) Py_RETURN_NOTIMPLEMENTED;
    if (f == GPTQ_NVFP4 && (!read_typed(a[2], o_f32, 1, &g) || g.shape[0] != 1)) Py_RETURN_NOTIMPLEMENTED;
    if (has_index) {
        if (!read_typed(a[3], o_i32, 1, &index) || !PyLong_Check(a[4])) Py_RETURN_NOTIMPLEMENTED;
        per = PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) return NULL;
    }
    const int64_t rows = has_index ? index.shape[0] : x.shape[0], cols = x.shape[1], span = f == GPTQ_MXFP4 ? 128 : 64;
    const int64_t cs[2] = {rows, (cols + 31) / 32 * 16}, ss[3] = {(rows + 127) / 128, (cols + span - 1) / span, 512};
    void *cp, *sp, *stream;
    PyObject *codes = empty(2, cs, o_u8, a[0], &cp), *scales = codes ? empty(3, ss, o_u8, a[0], &sp) : NULL;
    int status = 0;
    if (!scales || !current_stream(&stream)) goto fail;
    CALL(status, p_quantize(x.ptr, dtype_code(x.dtype), x.shape[0], cols, x.ld, index.ptr, per, rows, f, g.ptr, cp, sp, stream))
    if (!check("gptq_fp4_quantize", status)) goto fail;
    PyObject* scale = f == GPTQ_NVFP4 ? a[2] : Py_None;
    PyObject* items[5] = {codes, scales, PyLong_FromLongLong(cols), Py_NewRef(f == GPTQ_NVFP4 ? s_nv : s_mx), Py_NewRef(scale)};
    return named(t_fp4, 5, items);
fail:
    Py_XDECREF(codes);
    Py_XDECREF(scales);
    return NULL;
}

/* dequantize(q, dtype) */
static PyObject* dequantize(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Fp4 q;
    if (n != 2 || dtype_code(a[1]) < 0 || !read_fp4(a[0], 0, &q)) Py_RETURN_NOTIMPLEMENTED;
    const int64_t shape[2] = {q.rows, q.cols};
    void *yp, *stream;
    PyObject* y = empty(2, shape, a[1], PyTuple_GET_ITEM(a[0], 0), &yp);
    int status = 0;
    if (!y || !current_stream(&stream)) goto fail;
    CALL(status, p_dequantize(q.codes.ptr, q.scales.ptr, q.g.ptr, q.rows, q.cols, q.format, yp, dtype_code(a[1]), q.cols, stream))
    if (check("gptq_fp4_dequantize", status)) return y;
fail:
    Py_XDECREF(y);
    return NULL;
}

/* matmul(X, W, offsets, relu, out_dtype) */
static PyObject* matmul(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Fp4 x, w;
    Tensor offsets = {0};
    const int grouped = n == 5 && a[2] != Py_None;
    if (n != 5 || dtype_code(a[4]) < 0 || !read_fp4(a[0], 0, &x) || !read_fp4(a[1], grouped, &w) || x.format != w.format ||
        x.cols != w.cols || x.cols == 0 || (grouped && (!read_typed(a[2], o_i32, 1, &offsets) || offsets.shape[0] != w.experts + 1)))
        Py_RETURN_NOTIMPLEMENTED;
    const int relu = PyObject_IsTrue(a[3]);
    if (relu < 0) return NULL;
    const int flags = (relu ? GPTQ_DQ_RELU : 0) | (a[4] == o_bf16 ? GPTQ_DQ_BF16_OUT : 0) | (w.gs > 1 ? GPTQ_FP4_EXPERT_G : 0);
    const int64_t shape[2] = {x.rows, w.rows};
    void *yp, *stream;
    PyObject* y = empty(2, shape, a[4], PyTuple_GET_ITEM(a[0], 0), &yp);
    int status = 0;
    if (!y || !current_stream(&stream)) goto fail;
    CALL(status, p_matmul(x.codes.ptr, x.scales.ptr, x.g.ptr, x.rows, w.codes.ptr, w.scales.ptr, w.g.ptr, w.rows, x.cols, x.format,
                          offsets.ptr, w.experts, flags, yp, w.rows, stream))
    if (check("gptq_fp4_matmul", status)) return y;
fail:
    Py_XDECREF(y);
    return NULL;
}

/* sort(ids, experts) */
static PyObject* sort(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Tensor ids;
    if (n != 2 || !PyLong_Check(a[1]) || !read_typed(a[0], o_i32, 2, &ids)) Py_RETURN_NOTIMPLEMENTED;
    const int64_t tokens = ids.shape[0], top = ids.shape[1], experts = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred()) return NULL;
    if (experts < 1 || top < 1) Py_RETURN_NOTIMPLEMENTED;
    const int64_t os[1] = {experts + 1}, ss[1] = {tokens * top}, ps[2] = {tokens, top};
    const int64_t need[1] = {(int64_t)p_sort_ws(tokens, top, experts)};
    void *op, *sp, *pp, *ws = NULL, *stream;
    PyObject *offsets = empty(1, os, o_i32, a[0], &op), *src = NULL, *pos = NULL, *work = NULL;
    int status = 0;
    if (!offsets || !(src = empty(1, ss, o_i32, a[0], &sp)) || !(pos = empty(2, ps, o_i32, a[0], &pp)) ||
        (need[0] > 0 && !(work = empty(1, need, o_u8, a[0], &ws))) || !current_stream(&stream))
        goto fail;
    CALL(status, p_sort(ids.ptr, tokens, top, experts, op, sp, pp, ws, (size_t)need[0], stream))
    if (!check("gptq_expert_sort", status)) goto fail;
    Py_XDECREF(work);
    PyObject* items[3] = {offsets, src, pos};
    return named(t_route, 3, items);
fail:
    Py_XDECREF(offsets);
    Py_XDECREF(src);
    Py_XDECREF(pos);
    Py_XDECREF(work);
    return NULL;
}

/* gather(X, route) */
static PyObject* gather(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Tensor x;
    Route r;
    if (n != 2 || !read_matrix(a[0], &x) || !read_route(a[1], &r) || x.shape[0] != r.tokens) Py_RETURN_NOTIMPLEMENTED;
    const int64_t d = x.shape[1], shape[2] = {r.tokens * r.top, d};
    void *yp, *stream;
    PyObject* y = empty(2, shape, x.dtype, a[0], &yp);
    int status = 0;
    if (!y || !current_stream(&stream)) goto fail;
    CALL(status, p_gather(x.ptr, dtype_code(x.dtype), r.tokens, d, x.ld, r.pos.ptr, r.top, r.offsets.ptr, r.experts, yp, d, stream))
    if (check("gptq_expert_gather", status)) return y;
fail:
    Py_XDECREF(y);
    return NULL;
}

/* combine(Ys, route, weights) */
static PyObject* combine(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Tensor ys, w = {0};
    Route r;
    if (n != 3 || !read_matrix(a[0], &ys) || !read_route(a[1], &r) || ys.shape[0] != r.tokens * r.top ||
        (a[2] != Py_None && (!read_typed(a[2], o_f32, 2, &w) || w.shape[0] != r.tokens || w.shape[1] != r.top)))
        Py_RETURN_NOTIMPLEMENTED;
    const int64_t d = ys.shape[1], shape[2] = {r.tokens, d};
    void *yp, *stream;
    PyObject* y = empty(2, shape, ys.dtype, a[0], &yp);
    int status = 0;
    if (!y || !current_stream(&stream)) goto fail;
    CALL(status, p_combine(ys.ptr, dtype_code(ys.dtype), r.tokens, d, ys.ld, r.pos.ptr, r.top, w.ptr, yp, d, stream))
    if (check("gptq_expert_combine", status)) return y;
fail:
    Py_XDECREF(y);
    return NULL;
}

/* combine_grad(dY, Ys, route, weights) */
static PyObject* combine_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    find_device();
    Tensor dy, ys, w;
    Route r;
    if (n != 4 || !read_matrix(a[0], &dy) || !read_matrix(a[1], &ys) || !read_route(a[2], &r) || !read_typed(a[3], o_f32, 2, &w) ||
        dy.dtype != ys.dtype || dy.shape[0] != r.tokens || dy.shape[1] != ys.shape[1] || ys.shape[0] != r.tokens * r.top ||
        w.shape[0] != r.tokens || w.shape[1] != r.top)
        Py_RETURN_NOTIMPLEMENTED;
    const int64_t d = ys.shape[1], s1[2] = {r.tokens * r.top, d}, s2[2] = {r.tokens, r.top};
    void *xp, *wp, *stream;
    PyObject *dys = empty(2, s1, ys.dtype, a[1], &xp), *dw = dys ? empty(2, s2, o_f32, a[1], &wp) : NULL;
    int status = 0;
    if (!dw || !current_stream(&stream)) goto fail;
    CALL(status, p_combine_grad(dy.ptr, dy.ld, ys.ptr, ys.ld, dtype_code(ys.dtype), r.tokens, d, r.pos.ptr, r.top, r.offsets.ptr,
                                r.experts, w.ptr, xp, d, wp, stream))
    if (!check("gptq_expert_combine_grad", status)) goto fail;
    PyObject* both = PyTuple_New(2);
    if (!both) goto fail;
    PyTuple_SET_ITEM(both, 0, dys);
    PyTuple_SET_ITEM(both, 1, dw);
    return both;
fail:
    Py_XDECREF(dys);
    Py_XDECREF(dw);
    return NULL;
}

/* setup(objects, addresses): the Python objects and the library's entry points, by name */
static PyObject* setup(PyObject* self, PyObject* args) {
    PyObject *objects, *addresses;
    if (!PyArg_ParseTuple(args, "O!O!", &PyDict_Type, &objects, &PyDict_Type, &addresses)) return NULL;
    struct { const char* name; PyObject** to; } o[] = {
        {"float32", &o_f32}, {"bfloat16", &o_bf16}, {"uint8", &o_u8}, {"int32", &o_i32}, {"empty", &f_empty},
        {"raw_stream", &f_raw_stream}, {"current_device", &f_current_device}, {"Fp4", &t_fp4}, {"Route", &t_route},
        {"check", &f_check}};
    for (size_t i = 0; i < sizeof o / sizeof *o; ++i) {
        PyObject* v = PyDict_GetItemString(objects, o[i].name);
        if (!v) return PyErr_Format(PyExc_KeyError, "%s", o[i].name);
        Py_XSETREF(*o[i].to, Py_NewRef(v));
    }
    struct { const char* name; void* to; } f[] = {
        {"gptq_fp4_quantize", &p_quantize}, {"gptq_fp4_dequantize", &p_dequantize}, {"gptq_fp4_matmul", &p_matmul},
        {"gptq_expert_sort_workspace_bytes", &p_sort_ws}, {"gptq_expert_sort", &p_sort}, {"gptq_expert_gather", &p_gather},
        {"gptq_expert_combine", &p_combine}, {"gptq_expert_combine_grad", &p_combine_grad}};
    for (size_t i = 0; i < sizeof f / sizeof *f; ++i) {
        PyObject* v = PyDict_GetItemString(addresses, f[i].name);
        if (!v) return PyErr_Format(PyExc_KeyError, "%s", f[i].name);
        *(void**)f[i].to = PyLong_AsVoidPtr(v);
        if (PyErr_Occurred()) return NULL;
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, NULL},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
    {"dequantize", (PyCFunction)(void (*)(void))dequantize, METH_FASTCALL, NULL},
    {"matmul", (PyCFunction)(void (*)(void))matmul, METH_FASTCALL, NULL},
    {"sort", (PyCFunction)(void (*)(void))sort, METH_FASTCALL, NULL},
    {"gather", (PyCFunction)(void (*)(void))gather, METH_FASTCALL, NULL},
    {"combine", (PyCFunction)(void (*)(void))combine, METH_FASTCALL, NULL},
    {"combine_grad", (PyCFunction)(void (*)(void))combine_grad, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "The serving calls of the binding in C.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__call(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_device = PyUnicode_InternFromString("device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_mx = PyUnicode_InternFromString("mx");
    s_nv = PyUnicode_InternFromString("nv");
    k_empty = Py_BuildValue("(ss)", "dtype", "device");
    if (!k_empty || !s_nv) return NULL;
    return PyModule_Create(&module);
}
