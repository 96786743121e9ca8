/* bind.c -- the Python side of the calls over rows (the 8-bit path, dropout, the
 * layer norm, the cross entropy), as a CPython module.
 *
 * A decoding step's kernels run for a few microseconds, as long as an
 * interpreter takes to look at the tensors of one call.  Each function here
 * takes the tensors of one entry point (outputs allocated), checks them --
 * shape, type, device, strides -- and makes the C call on the given or the
 * current stream.  It knows tensors only by their Python attributes, so it
 * is compiled without torch.  The C call runs without the interpreter's lock,
 * as ctypes' calls do: it may wait for memory, for its kernels to load or for
 * room in the launch queue.  (The same checks in Python and ctypes took 5.5
 * to 7.4 us a call, launch included; these take 3.2 to 4.7.)
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/tcr.h"

static PyObject *s_shape, *s_dtype, *s_stride, *s_data_ptr, *s_get_device, *s_cuda_stream;
/* set by setup() */
static PyObject *t_f16, *t_bf16, *t_f32, *t_i8, *t_i32, *t_i64, *raw_stream, *get_device, *set_device, *error_class;
static tcr_status (*f_rmsnorm)(const tcr_norm_args *, void *);
static tcr_status (*f_backward)(const tcr_norm_back_args *, void *);
static tcr_status (*f_quantize)(const void *, size_t, const void *, size_t, void *, size_t, float *, size_t, size_t,
                                int, void *);
static tcr_status (*f_dequantize)(const void *, size_t, const float *, void *, size_t, size_t, size_t, int, void *);
static tcr_status (*f_gemm)(const void *, size_t, const void *, size_t, const float *, const float *, void *, size_t,
                            size_t, size_t, size_t, int, void *);
static tcr_status (*f_dropout)(const void *, size_t, const void *, size_t, void *, size_t, size_t, size_t,
                               const tcr_drop *, int, void *);
static tcr_status (*f_layernorm)(const tcr_layernorm_args *, void *);
static tcr_status (*f_layernorm_backward)(const tcr_layernorm_back_args *, void *);
static tcr_status (*f_xent)(const tcr_xent_args *, void *);
static tcr_status (*f_xent_backward)(const tcr_xent_back_args *, void *);

/* One call's device, and the shape that its first tensor gives. */
typedef struct {
    long dev;
    Py_ssize_t rows, cols;
} Call;

/* A new reference to the tuple attribute `name` of t (called if it is a
 * method) and its length; -1 with an error set. */
static Py_ssize_t tuple_of(PyObject *t, PyObject *name, int method, PyObject **v)
{
    *v = method ? PyObject_CallMethodNoArgs(t, name) : PyObject_GetAttr(t, name);
    if (!*v) return -1;
    if (!PyTuple_Check(*v)) {
        Py_DECREF(*v);
        PyErr_SetString(PyExc_TypeError, "expected a tensor");
        return -1;
    }
    return PyTuple_GET_SIZE(*v);
}

static long device_of(PyObject *t)
{
    PyObject *v = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!v) return -2;
    const long d = PyLong_AsLong(v);
    Py_DECREF(v);
    return d;
}

/* The tensor that gives a call its device and shape. */
static int first(const char *name, PyObject *t, Call *c)
{
    PyObject *shape;
    const Py_ssize_t n = tuple_of(t, s_shape, 0, &shape);
    if (n < 0) return -1;
    if (n == 2) {
        c->rows = PyLong_AsSsize_t(PyTuple_GET_ITEM(shape, 0));
        c->cols = PyLong_AsSsize_t(PyTuple_GET_ITEM(shape, 1));
    }
    Py_DECREF(shape);
    c->dev = device_of(t);
    if (PyErr_Occurred()) return -1;
    if (n != 2 || c->dev < 0) {
        PyErr_Format(PyExc_ValueError, "%s must be a 2-D CUDA tensor", name);
        return -1;
    }
    return 0;
}

static int float_code(PyObject *dtype)
{
    return dtype == t_bf16 ? TCR_BF16 : dtype == t_f16 ? TCR_F16 : dtype == t_f32 ? TCR_F32 : -1;
}

/* The tcr_dtype of a float tensor, and its type object (borrowed: torch keeps
 * its types); -1 with TypeError set. */
static int float_type(PyObject *t, PyObject **dtype)
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    const int code = float_code(d);
    if (code < 0) PyErr_Format(PyExc_TypeError, "expected float16, bfloat16 or float32, got %S", d);
    Py_DECREF(d);
    *dtype = d;
    return code;
}

static int on_device(const char *name, PyObject *t, const Call *c)
{
    const long dev = device_of(t);
    if (PyErr_Occurred()) return -1;
    if (dev != c->dev) {
        PyErr_Format(PyExc_ValueError, "%s must be on cuda:%ld", name, c->dev);
        return -1;
    }
    return 0;
}

/* Type and address. */
static int typed(const char *name, PyObject *t, PyObject *dtype, const void **p)
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    if (d != dtype) {
        PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, d);
        Py_DECREF(d);
        return -1;
    }
    Py_DECREF(d);
    PyObject *a = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!a) return -1;
    *p = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return PyErr_Occurred() ? -1 : 0;
}

/* A rows x cols matrix with contiguous rows, its shape and device known;
 * input: its rows may be one row for all (leading dimension 0). */
static int rows_of(const char *name, PyObject *t, Py_ssize_t rows, Py_ssize_t cols, PyObject *dtype, int input,
                   const void **p, size_t *ld)
{
    if (typed(name, t, dtype, p)) return -1;
    PyObject *stride;
    if (tuple_of(t, s_stride, 1, &stride) < 0) return -1;
    const Py_ssize_t l = PyLong_AsSsize_t(PyTuple_GET_ITEM(stride, 0)),
                     step = PyLong_AsSsize_t(PyTuple_GET_ITEM(stride, 1));
    Py_DECREF(stride);
    if (step != 1 && cols > 1) {
        PyErr_Format(PyExc_ValueError, "%s must have contiguous rows (stride 1 along its columns)", name);
        return -1;
    }
    *ld = (size_t)(rows > 1 ? l : cols);
    if (rows > 1 && l < cols && !(input && l == 0)) {
        PyErr_Format(PyExc_ValueError, "%s has overlapping rows", name);
        return -1;
    }
    return 0;
}

/* The same with its shape and device to be checked. */
static int matrix(const char *name, PyObject *t, Py_ssize_t rows, Py_ssize_t cols, PyObject *dtype, int input,
                  const Call *c, const void **p, size_t *ld)
{
    PyObject *shape;
    Py_ssize_t n = tuple_of(t, s_shape, 0, &shape);
    if (n < 0) return -1;
    const int same = n == 2 && PyLong_AsSsize_t(PyTuple_GET_ITEM(shape, 0)) == rows &&
                     PyLong_AsSsize_t(PyTuple_GET_ITEM(shape, 1)) == cols;
    if (!same) PyErr_Format(PyExc_ValueError, "%s must have shape (%zd, %zd), got %S", name, rows, cols, shape);
    Py_DECREF(shape);
    if (!same || on_device(name, t, c)) return -1;
    return rows_of(name, t, rows, cols, dtype, input, p, ld);
}

static int vector(const char *name, PyObject *t, Py_ssize_t n, PyObject *dtype, const Call *c, const void **p)
{
    PyObject *v;
    Py_ssize_t dims = tuple_of(t, s_shape, 0, &v);
    if (dims < 0) return -1;
    const int same = dims == 1 && PyLong_AsSsize_t(PyTuple_GET_ITEM(v, 0)) == n;
    if (!same) PyErr_Format(PyExc_ValueError, "%s must have shape (%zd,), got %S", name, n, v);
    Py_DECREF(v);
    if (!same) return -1;
    if (n > 1) {
        if (tuple_of(t, s_stride, 1, &v) < 0) return -1;
        const int dense = PyLong_AsSsize_t(PyTuple_GET_ITEM(v, 0)) == 1;
        Py_DECREF(v);
        if (!dense) {
            PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
            return -1;
        }
    }
    return on_device(name, t, c) ? -1 : typed(name, t, dtype, p);
}

/* The handle of the call's stream: a stream object's, a number, or (None) the
 * device's current one's. */
static int stream_of(PyObject *stream, const Call *c, void **s)
{
    PyObject *v;
    if (stream == Py_None) {
        PyObject *dev = PyLong_FromLong(c->dev);
        if (!dev) return -1;
        v = PyObject_CallOneArg(raw_stream, dev);
        Py_DECREF(dev);
    } else if (PyLong_Check(stream)) {
        v = Py_NewRef(stream);
    } else {
        v = PyObject_GetAttr(stream, s_cuda_stream);
    }
    if (!v) return -1;
    *s = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

/* Make the call's device current; *before: the one to go back to, or -1. */
static int enter_device(const Call *c, long *before)
{
    *before = -1;
    PyObject *v = PyObject_CallNoArgs(get_device);
    if (!v) return -1;
    const long now = PyLong_AsLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) return -1;
    if (now == c->dev) return 0;
    v = PyObject_CallFunction(set_device, "l", c->dev);
    if (!v) return -1;
    Py_DECREF(v);
    *before = now;
    return 0;
}

/* Back to the device before, and the call's status as None or TcrError. */
static PyObject *leave(long before, tcr_status st, const char *name)
{
    if (before >= 0) {
        PyObject *v = PyObject_CallFunction(set_device, "l", before);
        if (!v) return NULL;
        Py_DECREF(v);
    }
    if (st == TCR_OK) Py_RETURN_NONE;
    PyObject *e = PyObject_CallFunction(error_class, "is", (int)st, name);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    return NULL;
}

/* st = the C call, without the interpreter's lock; the arguments are C values
 * of tensors that the caller holds. */
#define UNLOCKED(st, call)      \
    do {                        \
        Py_BEGIN_ALLOW_THREADS; \
        (st) = (call);          \
        Py_END_ALLOW_THREADS;   \
    } while (0)

#define WANT_TRAINING(n)                                                             \
    WANT_ARGS(n);                                                                    \
    if (!t_i64) {                                                                    \
        PyErr_SetString(PyExc_RuntimeError, "setup_training() has not been called"); \
        return NULL;                                                                 \
    }

#define WANT_ARGS(n)                                                           \
    if (nargs != (n)) {                                                        \
        PyErr_Format(PyExc_TypeError, "%s takes %d arguments", __func__, (n)); \
        return NULL;                                                           \
    }                                                                          \
    if (!error_class) {                                                        \
        PyErr_SetString(PyExc_RuntimeError, "setup() has not been called");    \
        return NULL;                                                           \
    }

/* rmsnorm(x, weight, residual, eps, h, out, scale, rstd, stream) */
static PyObject *rmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(9);
    Call c;
    tcr_norm_args n = {0};
    PyObject *dt;
    if (first("x", a[0], &c) || (n.dtype = float_type(a[0], &dt)) < 0) return NULL;
    PyObject *ot = PyObject_GetAttr(a[5], s_dtype);
    if (!ot) return NULL;
    const int i8 = ot == t_i8;
    Py_DECREF(ot);
    n.y_dtype = i8 ? TCR_I8 : n.dtype;
    n.rows = (size_t)c.rows;
    n.cols = (size_t)c.cols;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    n.eps = (float)eps;
    if (rows_of("x", a[0], c.rows, c.cols, dt, 1, &n.x, &n.ldx) ||
        matrix("out", a[5], c.rows, c.cols, i8 ? t_i8 : dt, 0, &c, (const void **)&n.y, &n.ldy) ||
        (a[1] != Py_None && vector("weight", a[1], c.cols, dt, &c, &n.weight)) ||
        (a[2] != Py_None && matrix("residual", a[2], c.rows, c.cols, dt, 1, &c, &n.residual, &n.ldr)) ||
        (a[4] != Py_None && matrix("h", a[4], c.rows, c.cols, dt, 0, &c, (const void **)&n.h, &n.ldh)) ||
        (a[6] != Py_None && vector("scale", a[6], c.rows, t_f32, &c, (const void **)&n.scale)) ||
        (a[7] != Py_None && vector("rstd", a[7], c.rows, t_f32, &c, (const void **)&n.rstd)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[8], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_rmsnorm(&n, s));
    return leave(before, st, "tcr_rmsnorm");
}

/* rmsnorm_backward(dy, h, weight, rstd, dh, dx, dweight, stream) */
static PyObject *rmsnorm_backward(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(8);
    Call c;
    tcr_norm_back_args n = {0};
    PyObject *dt;
    if (first("h", a[1], &c) || (n.dtype = float_type(a[1], &dt)) < 0) return NULL;
    n.rows = (size_t)c.rows;
    n.cols = (size_t)c.cols;
    if (matrix("dy", a[0], c.rows, c.cols, dt, 1, &c, &n.dy, &n.lddy) ||
        rows_of("h", a[1], c.rows, c.cols, dt, 1, &n.h, &n.ldh) ||
        (a[2] != Py_None && vector("weight", a[2], c.cols, dt, &c, &n.weight)) ||
        vector("rstd", a[3], c.rows, t_f32, &c, (const void **)&n.rstd) ||
        (a[4] != Py_None && matrix("dh", a[4], c.rows, c.cols, dt, 1, &c, &n.dh, &n.lddh)) ||
        matrix("dx", a[5], c.rows, c.cols, dt, 0, &c, (const void **)&n.dx, &n.lddx) ||
        (a[6] != Py_None && vector("dweight", a[6], c.cols, t_f32, &c, (const void **)&n.dweight)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[7], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_backward(&n, s));
    return leave(before, st, "tcr_rmsnorm_backward");
}

/* quantize_rows(x, gate, out, scale, stream) */
static PyObject *quantize_rows(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(5);
    Call c;
    PyObject *dt;
    int code;
    const void *x, *g = NULL, *q, *sc;
    size_t ldx, ldg = 0, ldq;
    if (first("x", a[0], &c) || (code = float_type(a[0], &dt)) < 0 ||
        rows_of("x", a[0], c.rows, c.cols, dt, 1, &x, &ldx) ||
        (a[1] != Py_None && matrix("gate", a[1], c.rows, c.cols, dt, 1, &c, &g, &ldg)) ||
        matrix("out", a[2], c.rows, c.cols, t_i8, 0, &c, &q, &ldq) ||
        vector("scale", a[3], c.rows, t_f32, &c, &sc))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[4], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_quantize(x, ldx, g, ldg, (void *)q, ldq, (float *)sc, (size_t)c.rows, (size_t)c.cols, code, s));
    return leave(before, st, "tcr_quantize_rows_i8");
}

/* dequantize_rows(q, scale, out, stream) */
static PyObject *dequantize_rows(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(4);
    Call c;
    PyObject *dt;
    int code;
    const void *q, *sc, *y;
    size_t ldq, ldy;
    if (first("q", a[0], &c) || (code = float_type(a[2], &dt)) < 0 ||
        rows_of("q", a[0], c.rows, c.cols, t_i8, 1, &q, &ldq) || vector("scale", a[1], c.rows, t_f32, &c, &sc) ||
        matrix("out", a[2], c.rows, c.cols, dt, 0, &c, &y, &ldy))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[3], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_dequantize(q, ldq, (const float *)sc, (void *)y, ldy, (size_t)c.rows, (size_t)c.cols, code, s));
    return leave(before, st, "tcr_dequantize_rows_i8");
}

/* gemm(A, W, scale_a, scale_w, out, stream) */
static PyObject *gemm(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(6);
    Call c, w;
    if (first("A", a[0], &c) || first("W", a[1], &w)) return NULL;
    if (w.dev != c.dev) {
        PyErr_Format(PyExc_ValueError, "W must be on cuda:%ld", c.dev);
        return NULL;
    }
    if (w.cols != c.cols) {
        PyErr_Format(PyExc_ValueError, "inner dimensions differ: (%zd, %zd) vs (%zd, %zd)", c.rows, c.cols, w.rows,
                     w.cols);
        return NULL;
    }
    PyObject *ot = PyObject_GetAttr(a[4], s_dtype);
    if (!ot) return NULL;
    const int code = ot == t_i32 ? TCR_I32 : float_code(ot);
    if (code < 0) PyErr_Format(PyExc_TypeError, "expected float16, bfloat16, float32 or int32, got %S", ot);
    Py_DECREF(ot);      /* torch keeps its types */
    if (code < 0) return NULL;
    if (code == TCR_I32 && (a[2] != Py_None || a[3] != Py_None)) {
        PyErr_SetString(PyExc_ValueError, "int32 sums take no scales");
        return NULL;
    }
    const void *pa, *pw, *pc, *sa = NULL, *sw = NULL;
    size_t lda, ldw, ldc;
    if (rows_of("A", a[0], c.rows, c.cols, t_i8, 0, &pa, &lda) ||
        rows_of("W", a[1], w.rows, w.cols, t_i8, 0, &pw, &ldw) ||
        matrix("out", a[4], c.rows, w.rows, ot, 0, &c, &pc, &ldc) ||
        (a[2] != Py_None && vector("scale_a", a[2], c.rows, t_f32, &c, &sa)) ||
        (a[3] != Py_None && vector("scale_w", a[3], w.rows, t_f32, &c, &sw)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[5], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_gemm(pa, lda, pw, ldw, (const float *)sa, (const float *)sw, (void *)pc, ldc, (size_t)c.rows,
                        (size_t)w.rows, (size_t)c.cols, code, s));
    return leave(before, st, "tcr_gemm_i8");
}

/* A call's dropout from p, seed, offset and state (an int64 tensor of two, or
 * None); *use: 0 where p is 0 and there is none. */
static int drop_rule(PyObject *const *a, const Call *c, tcr_drop *d, int *use)
{
    d->p = PyFloat_AsDouble(a[0]);
    if (d->p == -1.0 && PyErr_Occurred()) return -1;
    if (!(d->p >= 0.0 && d->p <= 1.0)) {
        PyErr_SetString(PyExc_ValueError, "p must be in 0 .. 1");
        return -1;
    }
    d->seed = PyLong_AsUnsignedLongLongMask(a[1]);
    if (PyErr_Occurred()) return -1;
    d->offset = PyLong_AsUnsignedLongLongMask(a[2]);
    if (PyErr_Occurred()) return -1;
    d->state = NULL;
    *use = d->p > 0.0;
    return a[3] == Py_None ? 0 : vector("state", a[3], 2, t_i64, c, (const void **)&d->state);
}

/* dropout(x, p, seed, offset, state, residual, out, stream) */
static PyObject *dropout(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_TRAINING(8);
    Call c;
    PyObject *dt;
    int code, use;
    tcr_drop d;
    const void *x, *r = NULL, *y;
    size_t ldx, ldr = 0, ldy;
    if (first("x", a[0], &c) || (code = float_type(a[0], &dt)) < 0 || drop_rule(a + 1, &c, &d, &use) ||
        rows_of("x", a[0], c.rows, c.cols, dt, 1, &x, &ldx) ||
        (a[5] != Py_None && matrix("residual", a[5], c.rows, c.cols, dt, 1, &c, &r, &ldr)) ||
        matrix("out", a[6], c.rows, c.cols, dt, 0, &c, &y, &ldy))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[7], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_dropout(x, ldx, r, ldr, (void *)y, ldy, (size_t)c.rows, (size_t)c.cols, &d, code, s));
    return leave(before, st, "tcr_dropout");
}

/* layernorm(x, weight, bias, residual, eps, p, seed, offset, state, h, out, scale, mean, rstd, stream) */
static PyObject *layernorm(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_TRAINING(15);
    Call c;
    tcr_layernorm_args n = {0};
    tcr_drop d;
    int use;
    PyObject *dt;
    if (first("x", a[0], &c) || (n.dtype = float_type(a[0], &dt)) < 0 || drop_rule(a + 5, &c, &d, &use)) return NULL;
    PyObject *ot = PyObject_GetAttr(a[10], s_dtype);
    if (!ot) return NULL;
    const int i8 = ot == t_i8;
    Py_DECREF(ot);
    n.y_dtype = i8 ? TCR_I8 : n.dtype;
    n.rows = (size_t)c.rows;
    n.cols = (size_t)c.cols;
    n.drop = use ? &d : NULL;
    const double eps = PyFloat_AsDouble(a[4]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    n.eps = (float)eps;
    if (rows_of("x", a[0], c.rows, c.cols, dt, 1, &n.x, &n.ldx) ||
        matrix("out", a[10], c.rows, c.cols, i8 ? t_i8 : dt, 0, &c, (const void **)&n.y, &n.ldy) ||
        (a[1] != Py_None && vector("weight", a[1], c.cols, dt, &c, &n.weight)) ||
        (a[2] != Py_None && vector("bias", a[2], c.cols, dt, &c, &n.bias)) ||
        (a[3] != Py_None && matrix("residual", a[3], c.rows, c.cols, dt, 1, &c, &n.residual, &n.ldr)) ||
        (a[9] != Py_None && matrix("h", a[9], c.rows, c.cols, dt, 0, &c, (const void **)&n.h, &n.ldh)) ||
        (a[11] != Py_None && vector("scale", a[11], c.rows, t_f32, &c, (const void **)&n.scale)) ||
        (a[12] != Py_None && vector("mean", a[12], c.rows, t_f32, &c, (const void **)&n.mean)) ||
        (a[13] != Py_None && vector("rstd", a[13], c.rows, t_f32, &c, (const void **)&n.rstd)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[14], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_layernorm(&n, s));
    return leave(before, st, "tcr_layernorm");
}

/* layernorm_backward(dy, h, weight, mean, rstd, dh, p, seed, offset, state, dx, dresidual, dweight, dbias, stream) */
static PyObject *layernorm_backward(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_TRAINING(15);
    Call c;
    tcr_layernorm_back_args n = {0};
    tcr_drop d;
    int use;
    PyObject *dt;
    if (first("h", a[1], &c) || (n.dtype = float_type(a[1], &dt)) < 0 || drop_rule(a + 6, &c, &d, &use)) return NULL;
    n.rows = (size_t)c.rows;
    n.cols = (size_t)c.cols;
    n.drop = use ? &d : NULL;
    if (matrix("dy", a[0], c.rows, c.cols, dt, 1, &c, &n.dy, &n.lddy) ||
        rows_of("h", a[1], c.rows, c.cols, dt, 1, &n.h, &n.ldh) ||
        (a[2] != Py_None && vector("weight", a[2], c.cols, dt, &c, &n.weight)) ||
        vector("mean", a[3], c.rows, t_f32, &c, (const void **)&n.mean) ||
        vector("rstd", a[4], c.rows, t_f32, &c, (const void **)&n.rstd) ||
        (a[5] != Py_None && matrix("dh", a[5], c.rows, c.cols, dt, 1, &c, &n.dh, &n.lddh)) ||
        (a[10] != Py_None && matrix("dx", a[10], c.rows, c.cols, dt, 0, &c, (const void **)&n.dx, &n.lddx)) ||
        (a[11] != Py_None &&
         matrix("dresidual", a[11], c.rows, c.cols, dt, 0, &c, (const void **)&n.dresidual, &n.lddr)) ||
        (a[12] != Py_None && vector("dweight", a[12], c.cols, t_f32, &c, (const void **)&n.dweight)) ||
        (a[13] != Py_None && vector("dbias", a[13], c.cols, t_f32, &c, (const void **)&n.dbias)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[14], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_layernorm_backward(&n, s));
    return leave(before, st, "tcr_layernorm_backward");
}

/* x and weight of the cross entropy: their device, shapes, type and rows. */
static int xent_inputs(PyObject *x, PyObject *weight, Call *c, Call *w, int *code, PyObject **dt, const void **px,
                       size_t *ldx, const void **pw, size_t *ldw)
{
    if (first("x", x, c) || first("weight", weight, w)) return -1;
    if (w->dev != c->dev) {
        PyErr_Format(PyExc_ValueError, "weight must be on cuda:%ld", c->dev);
        return -1;
    }
    if (w->cols != c->cols) {
        PyErr_Format(PyExc_ValueError, "inner dimensions differ: (%zd, %zd) vs (%zd, %zd)", c->rows, c->cols, w->rows,
                     w->cols);
        return -1;
    }
    if ((*code = float_type(x, dt)) < 0) return -1;
    if (*code == TCR_F32) {
        PyErr_Format(PyExc_TypeError, "expected float16 or bfloat16, got %S", *dt);
        return -1;
    }
    return rows_of("x", x, c->rows, c->cols, *dt, 1, px, ldx) || rows_of("weight", weight, w->rows, w->cols, *dt, 0, pw, ldw)
               ? -1
               : 0;
}

/* cross_entropy(x, weight, target, ignore_index, loss, lse, stream) */
static PyObject *cross_entropy(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_TRAINING(7);
    Call c, w;
    tcr_xent_args n = {0};
    PyObject *dt;
    if (xent_inputs(a[0], a[1], &c, &w, &n.dtype, &dt, &n.x, &n.ldx, &n.weight, &n.ldw)) return NULL;
    n.tokens = (size_t)c.rows;
    n.hidden = (size_t)c.cols;
    n.vocab = (size_t)w.rows;
    n.ignore_index = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred()) return NULL;
    if (vector("target", a[2], c.rows, t_i64, &c, (const void **)&n.target) ||
        vector("loss", a[4], c.rows, t_f32, &c, (const void **)&n.loss) ||
        (a[5] != Py_None && vector("lse", a[5], c.rows, t_f32, &c, (const void **)&n.lse)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[6], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_xent(&n, s));
    return leave(before, st, "tcr_cross_entropy");
}

/* cross_entropy_backward(dloss, x, weight, target, lse, ignore_index, dx, dweight, stream) */
static PyObject *cross_entropy_backward(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_TRAINING(9);
    Call c, w;
    tcr_xent_back_args n = {0};
    PyObject *dt, *v;
    if (xent_inputs(a[1], a[2], &c, &w, &n.dtype, &dt, &n.x, &n.ldx, &n.weight, &n.ldw)) return NULL;
    n.tokens = (size_t)c.rows;
    n.hidden = (size_t)c.cols;
    n.vocab = (size_t)w.rows;
    n.ignore_index = PyLong_AsLongLong(a[5]);
    if (PyErr_Occurred()) return NULL;
    /* dloss: contiguous, or one value expanded over the tokens */
    const Py_ssize_t dims = tuple_of(a[0], s_shape, 0, &v);
    if (dims < 0) return NULL;
    const int same = dims == 1 && PyLong_AsSsize_t(PyTuple_GET_ITEM(v, 0)) == c.rows;
    if (!same) PyErr_Format(PyExc_ValueError, "dloss must have shape (%zd,), got %S", c.rows, v);
    Py_DECREF(v);
    if (!same || tuple_of(a[0], s_stride, 1, &v) < 0) return NULL;
    const Py_ssize_t inc = PyLong_AsSsize_t(PyTuple_GET_ITEM(v, 0));
    Py_DECREF(v);
    if (c.rows > 1 && inc != 0 && inc != 1) {
        PyErr_SetString(PyExc_ValueError, "dloss must be contiguous or expanded from one value");
        return NULL;
    }
    n.inc_dloss = c.rows > 1 ? (size_t)inc : 1;
    if (on_device("dloss", a[0], &c) || typed("dloss", a[0], t_f32, (const void **)&n.dloss) ||
        vector("target", a[3], c.rows, t_i64, &c, (const void **)&n.target) ||
        vector("lse", a[4], c.rows, t_f32, &c, (const void **)&n.lse) ||
        (a[6] != Py_None && matrix("dx", a[6], c.rows, c.cols, dt, 0, &c, (const void **)&n.dx, &n.lddx)) ||
        (a[7] != Py_None && matrix("dweight", a[7], w.rows, w.cols, dt, 0, &c, (const void **)&n.dweight, &n.lddw)))
        return NULL;
    void *s;
    long before;
    if (stream_of(a[8], &c, &s) || enter_device(&c, &before)) return NULL;
    tcr_status st;
    UNLOCKED(st, f_xent_backward(&n, s));
    return leave(before, st, "tcr_cross_entropy_backward");
}

/* setup(float16, bfloat16, float32, int8, int32, raw_stream, get_device,
 *       set_device, error class, addresses of the five entry points) */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    if (nargs != 14) {
        PyErr_SetString(PyExc_TypeError, "setup takes 14 arguments");
        return NULL;
    }
    PyObject **slot[] = {&t_f16, &t_bf16, &t_f32, &t_i8, &t_i32, &raw_stream, &get_device, &set_device, &error_class};
    void *f[5];
    for (int i = 0; i < 5; i++) {
        f[i] = PyLong_AsVoidPtr(a[9 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    for (int i = 0; i < 9; i++) Py_XSETREF(*slot[i], Py_NewRef(a[i]));
    f_rmsnorm = (tcr_status(*)(const tcr_norm_args *, void *))f[0];
    f_backward = (tcr_status(*)(const tcr_norm_back_args *, void *))f[1];
    f_quantize = (tcr_status(*)(const void *, size_t, const void *, size_t, void *, size_t, float *, size_t, size_t,
                                int, void *))f[2];
    f_dequantize = (tcr_status(*)(const void *, size_t, const float *, void *, size_t, size_t, size_t, int, void *))f[3];
    f_gemm = (tcr_status(*)(const void *, size_t, const void *, size_t, const float *, const float *, void *, size_t,
                            size_t, size_t, size_t, int, void *))f[4];
    Py_RETURN_NONE;
}

/* setup_training(int64, addresses of the five entry points of dropout, the layer
 * norm and the cross entropy): after setup() */
static PyObject *setup_training(PyObject *self, PyObject *const *a, Py_ssize_t nargs)
{
    (void)self;
    WANT_ARGS(6);
    void *f[5];
    for (int i = 0; i < 5; i++) {
        f[i] = PyLong_AsVoidPtr(a[1 + i]);
        if (PyErr_Occurred()) return NULL;
    }
    Py_XSETREF(t_i64, Py_NewRef(a[0]));
    f_dropout = (tcr_status(*)(const void *, size_t, const void *, size_t, void *, size_t, size_t, size_t,
                               const tcr_drop *, int, void *))f[0];
    f_layernorm = (tcr_status(*)(const tcr_layernorm_args *, void *))f[1];
    f_layernorm_backward = (tcr_status(*)(const tcr_layernorm_back_args *, void *))f[2];
    f_xent = (tcr_status(*)(const tcr_xent_args *, void *))f[3];
    f_xent_backward = (tcr_status(*)(const tcr_xent_back_args *, void *))f[4];
    Py_RETURN_NONE;
}

#define FAST(f) {#f, (PyCFunction)(void (*)(void))f, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(setup),         FAST(rmsnorm),         FAST(rmsnorm_backward),
                                FAST(quantize_rows), FAST(dequantize_rows), FAST(gemm),
                                FAST(dropout),       FAST(layernorm),       FAST(layernorm_backward),
                                FAST(cross_entropy), FAST(cross_entropy_backward), FAST(setup_training),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tcrbind", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tcrbind(void)
{
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (!s_shape || !s_dtype || !s_stride || !s_data_ptr || !s_get_device || !s_cuda_stream) return NULL;
    return PyModule_Create(&module);
}
