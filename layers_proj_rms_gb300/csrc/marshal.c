/* Argument marshalling of the sub-layer edge operators (q/k norm + rotation,
 * router, sort, dispatch, combine) and of the experts' products in 8-bit
 * floating point for the Python binding: checks the torch
 * tensors it is given (type, dtype, shape, contiguity, device), takes their
 * device pointers and calls the library's C entry points.  It does what
 * _lib.py does for the other entry points, in C because these operators are
 * also called on single tokens, where the call costs more than the kernel: on
 * the GB300's Arm host a q/k call took 9.9 us through Python and ctypes, of
 * which the launch is 2, and a sort call 5.6; here they take 5.4 and 4.2.
 *
 * Needs Python's headers alone.  A tensor is looked at through its attributes,
 * nothing is kept between calls, and the interpreter lock is released during
 * the library call. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/mhc.h"

enum { BF16 = MHC_BF16, FP16 = MHC_FP16, FP32 = MHC_FP32, I32, U8, E4M3, E5M2, NTYPES };

static PyObject *tensor_type, *dtypes[NTYPES];
static PyObject *s_shape, *s_dtype, *s_is_cuda, *s_is_contiguous, *s_data_ptr, *s_stride;

static const char *const type_names[NTYPES] = {"torch.bfloat16", "torch.float16", "torch.float32",
                                               "torch.int32", "torch.uint8",
                                               "torch.float8_e4m3fn", "torch.float8_e5m2"};

/* The entry points, in the order that setup() gets their addresses. */
static struct {
    __typeof__(&mhc_qk_norm_rope_fwd) qk_fwd;
    __typeof__(&mhc_qk_norm_rope_bwd) qk_bwd;
    __typeof__(&mhc_moe_router_fwd) router_fwd;
    __typeof__(&mhc_moe_router_bwd) router_bwd;
    __typeof__(&mhc_moe_sort) sort;
    __typeof__(&mhc_moe_dispatch_fwd) dispatch_fwd;
    __typeof__(&mhc_moe_dispatch_bwd) dispatch_bwd;
    __typeof__(&mhc_moe_combine_fwd) combine_fwd;
    __typeof__(&mhc_moe_combine_bwd) combine_bwd;
    __typeof__(&mhc_fp8_quant) fp8_quant;
    __typeof__(&mhc_fp8_swiglu_fwd) fp8_swiglu_fwd;
    __typeof__(&mhc_fp8_swiglu_bwd) fp8_swiglu_bwd;
    __typeof__(&mhc_fp8_gemm) fp8_gemm;
    __typeof__(&mhc_fp8_wgrad) fp8_wgrad;
    __typeof__(&mhc_moe_few_fwd) few_fwd;
} fn;

#define CALL(status, ...)                                             \
    Py_BEGIN_ALLOW_THREADS status = (int)(__VA_ARGS__);               \
    Py_END_ALLOW_THREADS

/* What the checks need of one tensor. */
typedef struct {
    PyObject *obj;   /* borrowed; NULL: None */
    const char *name;
    int code;        /* its type, -1: another */
    int nd;
    int64_t d[3];
    int64_t st[3];   /* strides, where asked for */
    int64_t numel;
    void *ptr;
} Tensor;

/* Reads type and shape; 0 and an exception on failure. */
static int look(PyObject *o, const char *name, Tensor *t)
{
    t->name = name;
    t->obj = NULL;
    t->code = -1;
    t->nd = 0;
    t->numel = 0;
    t->ptr = NULL;
    t->st[0] = t->st[1] = t->st[2] = 0;
    if (o == Py_None) return 1;
    if (!PyObject_TypeCheck(o, (PyTypeObject *)tensor_type)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", name);
        return 0;
    }
    t->obj = o;
    PyObject *dt = PyObject_GetAttr(o, s_dtype);
    if (!dt) return 0;
    for (int i = 0; i < NTYPES; ++i)
        if (dt == dtypes[i]) t->code = i;
    Py_DECREF(dt);
    PyObject *shape = PyObject_GetAttr(o, s_shape);
    if (!shape) return 0;
    t->nd = (int)PyTuple_Size(shape);
    t->numel = 1;
    for (int i = 0; i < t->nd; ++i) {
        const int64_t v = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
        if (i < 3) t->d[i] = v;
        t->numel *= v;
    }
    Py_DECREF(shape);
    return !PyErr_Occurred();
}

static int wrong_type(const Tensor *t, const char *expected)
{
    PyObject *dt = PyObject_GetAttr(t->obj, s_dtype);
    if (dt) PyErr_Format(PyExc_TypeError, "%s: dtype %S, expected %s", t->name, dt, expected);
    Py_XDECREF(dt);
    return 0;
}

static int wrong_shape(const Tensor *t, int nd, int64_t a, int64_t b, int64_t c)
{
    PyObject *shape = PyObject_GetAttr(t->obj, s_shape);
    if (shape && nd == 1)
        PyErr_Format(PyExc_ValueError, "%s: shape %S, expected (%lld,)", t->name, shape, (long long)a);
    else if (shape && nd == 2)
        PyErr_Format(PyExc_ValueError, "%s: shape %S, expected (%lld, %lld)", t->name, shape,
                     (long long)a, (long long)b);
    else if (shape)
        PyErr_Format(PyExc_ValueError, "%s: shape %S, expected (%lld, %lld, %lld)", t->name, shape,
                     (long long)a, (long long)b, (long long)c);
    Py_XDECREF(shape);
    return 0;
}

static int truth(const Tensor *t, PyObject *attr, int method)
{
    PyObject *v = method ? PyObject_CallMethodNoArgs(t->obj, attr) : PyObject_GetAttr(t->obj, attr);
    if (!v) return -1;
    const int r = PyObject_IsTrue(v);
    Py_DECREF(v);
    return r;
}

/* Device pointer of a tensor that has passed its other checks. */
static int point(Tensor *t)
{
    if (t->numel == 0) return 1;
    const int cuda = truth(t, s_is_cuda, 0);
    if (cuda < 0) return 0;
    if (!cuda) {
        PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", t->name);
        return 0;
    }
    PyObject *p = PyObject_CallMethodNoArgs(t->obj, s_data_ptr);
    if (!p) return 0;
    t->ptr = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(p);
    Py_DECREF(p);
    return !PyErr_Occurred();
}

static int contiguous(Tensor *t)
{
    const int c = truth(t, s_is_contiguous, 1);
    if (c < 0) return 0;
    if (!c) {
        PyErr_Format(PyExc_ValueError, "%s must be contiguous", t->name);
        return 0;
    }
    return point(t);
}

static int given(const Tensor *t)
{
    if (!t->obj) PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor", t->name);
    return t->obj != NULL;
}

/* An activation of any type and nd dimensions; sets *code. */
static int activation(Tensor *t, int nd, int *code)
{
    if (!given(t)) return 0;
    if (t->code != BF16 && t->code != FP16 && t->code != FP32)
        return wrong_type(t, "bfloat16, float16 or float32");
    *code = t->code;
    if (t->nd != nd) {
        PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", t->name, nd);
        return 0;
    }
    return 1;
}

/* A contiguous tensor of this type and shape (nd 1 or 2); `opt`: may be None. */
static int exact(Tensor *t, int code, int nd, int64_t a, int64_t b, int opt)
{
    if (opt && !t->obj) return 1;
    if (!given(t)) return 0;
    if (t->code != code) return wrong_type(t, type_names[code]);
    if (t->nd != nd || t->d[0] != a || (nd > 1 && t->d[1] != b)) return wrong_shape(t, nd, a, b, 0);
    return contiguous(t);
}

/* A [T, H, D] tensor or view with any token and head stride; None where H = 0. */
static int heads(Tensor *t, int code, int64_t T, int64_t H, int64_t D)
{
    if (!t->obj && H == 0) return 1;
    if (!given(t)) return 0;
    if (t->code != code) return wrong_type(t, type_names[code]);
    if (t->nd != 3 || t->d[0] != T || t->d[1] != H || t->d[2] != D) return wrong_shape(t, 3, T, H, D);
    PyObject *st = PyObject_CallMethodNoArgs(t->obj, s_stride);
    if (!st) return 0;
    for (int i = 0; i < 3; ++i) t->st[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(st, i));
    Py_DECREF(st);
    if (PyErr_Occurred()) return 0;
    if (t->st[2] != 1 && D > 1) {
        PyErr_Format(PyExc_ValueError, "%s: the elements of a head must be contiguous", t->name);
        return 0;
    }
    if (t->numel == 0) t->st[0] = t->st[1] = 0;
    return point(t);
}

static int nargs(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return n == want;
}

static int whole(PyObject *o, int64_t *v)
{
    *v = PyLong_AsLongLong(o);
    return !(*v == -1 && PyErr_Occurred());
}

static int real(PyObject *o, float *v)
{
    const double d = PyFloat_AsDouble(o);
    *v = (float)d;
    return !(d == -1.0 && PyErr_Occurred());
}

static int handle(PyObject *o, mhc_stream_t *s)
{
    *s = (mhc_stream_t)(uintptr_t)PyLong_AsUnsignedLongLong(o);
    return !PyErr_Occurred();
}

/* What the two q/k calls share: shapes, gammas, table, positions. */
typedef struct {
    Tensor q, k, gq, gk, cos, sin, pos;
    int code, inter;
    int64_t T, Hq, Hk, D, R, P;
    float eps;
    mhc_stream_t stream;
} Qk;

static int three(const Tensor *t)
{
    if (t->obj && t->nd != 3) PyErr_Format(PyExc_ValueError, "%s must be a [T, H, D] tensor", t->name);
    return !t->obj || t->nd == 3;
}

/* a: q, k, gamma_q, gamma_k, cos, sin, pos, eps; then inter and the stream */
static int qk_args(PyObject *const *a, PyObject *inter, PyObject *stream, Qk *x)
{
    if (!look(a[0], "q", &x->q) || !look(a[1], "k", &x->k) || !look(a[2], "gamma_q", &x->gq) ||
        !look(a[3], "gamma_k", &x->gk) || !look(a[4], "cos", &x->cos) || !look(a[5], "sin", &x->sin) ||
        !look(a[6], "pos", &x->pos))
        return 0;
    Tensor *one = x->q.obj ? &x->q : &x->k;
    if (!one->obj) {
        PyErr_SetString(PyExc_ValueError, "q and k are both None");
        return 0;
    }
    if (!three(&x->q) || !three(&x->k) || !activation(one, 3, &x->code)) return 0;
    x->T = one->d[0];
    x->D = one->d[2];
    x->Hq = x->q.obj ? x->q.d[1] : 0;
    x->Hk = x->k.obj ? x->k.d[1] : 0;
    x->R = x->P = 0;
    if (x->cos.obj) {
        if (x->cos.nd != 2) {
            PyErr_SetString(PyExc_ValueError, "cos must be a [P, R/2] tensor");
            return 0;
        }
        x->P = x->cos.d[0];
        x->R = 2 * x->cos.d[1];
    }
    x->inter = PyObject_IsTrue(inter);
    if (x->Hq > INT32_MAX || x->Hk > INT32_MAX || x->D > INT32_MAX || x->R > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "a head count or size does not fit 32 bits");
        return 0;
    }
    return x->inter >= 0 && heads(&x->q, x->code, x->T, x->Hq, x->D) &&
           heads(&x->k, x->code, x->T, x->Hk, x->D) && exact(&x->gq, FP32, 1, x->D, 0, 1) &&
           exact(&x->gk, FP32, 1, x->D, 0, 1) && exact(&x->cos, FP32, 2, x->P, x->R / 2, 1) &&
           exact(&x->sin, FP32, 2, x->P, x->R / 2, 1) && exact(&x->pos, I32, 1, x->T, 0, 1) &&
           real(a[7], &x->eps) && handle(stream, &x->stream);
}

/* (q, k, gamma_q, gamma_k, cos, sin, pos, eps, q_out, k_out, interleaved, stream) -> status */
static PyObject *py_qk_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Qk x;
    Tensor qo, ko;
    if (!nargs(n, 12) || !qk_args(a, a[10], a[11], &x) || !look(a[8], "q_out", &qo) ||
        !look(a[9], "k_out", &ko) || !heads(&qo, x.code, x.T, x.Hq, x.D) ||
        !heads(&ko, x.code, x.T, x.Hk, x.D))
        return NULL;
    const int64_t st[8] = {x.q.st[0], x.q.st[1], x.k.st[0], x.k.st[1],
                           qo.st[0],  qo.st[1],  ko.st[0],  ko.st[1]};
    int status;
    CALL(status, fn.qk_fwd(x.q.ptr, x.k.ptr, (mhc_dtype)x.code, st, x.gq.ptr, x.gk.ptr, x.cos.ptr,
                           x.sin.ptr, x.pos.ptr, x.T, (int)x.Hq, (int)x.Hk, (int)x.D, (int)x.R, x.P,
                           x.inter, x.eps, qo.ptr, ko.ptr, x.stream))
    return PyLong_FromLong(status);
}

/* (dq_out, dk_out, q, k, gamma_q, gamma_k, cos, sin, pos, eps, dq, dk, dgamma_q,
 *  dgamma_k, ws, interleaved, stream) -> status */
static PyObject *py_qk_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Qk x;
    Tensor uq, uk, dq, dk, dgq, dgk, ws;
    if (!nargs(n, 17) || !qk_args(a + 2, a[15], a[16], &x) || !look(a[0], "dq_out", &uq) ||
        !look(a[1], "dk_out", &uk) || !look(a[10], "dq", &dq) || !look(a[11], "dk", &dk) ||
        !look(a[12], "dgamma_q", &dgq) || !look(a[13], "dgamma_k", &dgk) || !look(a[14], "ws", &ws) ||
        !heads(&uq, x.code, x.T, x.Hq, x.D) || !heads(&uk, x.code, x.T, x.Hk, x.D) ||
        !heads(&dq, x.code, x.T, x.Hq, x.D) || !heads(&dk, x.code, x.T, x.Hk, x.D) ||
        !exact(&dgq, FP32, 1, x.D, 0, 1) || !exact(&dgk, FP32, 1, x.D, 0, 1) ||
        !exact(&ws, U8, 1, ws.numel, 0, 1))
        return NULL;
    const int64_t st[12] = {uq.st[0],  uq.st[1],  uk.st[0], uk.st[1], x.q.st[0], x.q.st[1],
                            x.k.st[0], x.k.st[1], dq.st[0], dq.st[1], dk.st[0],  dk.st[1]};
    int status;
    CALL(status,
         fn.qk_bwd(uq.ptr, uk.ptr, x.q.ptr, x.k.ptr, (mhc_dtype)x.code, st, x.gq.ptr, x.gk.ptr,
                   x.cos.ptr, x.sin.ptr, x.pos.ptr, x.T, (int)x.Hq, (int)x.Hk, (int)x.D, (int)x.R,
                   x.P, x.inter, x.eps, dq.ptr, dk.ptr, dgq.ptr, dgk.ptr, ws.ptr, (size_t)ws.numel,
                   x.stream))
    return PyLong_FromLong(status);
}

/* Sizes that the C entry points take as int. */
static int small(int64_t v, const char *name)
{
    if (v > INT32_MAX || v < INT32_MIN) PyErr_Format(PyExc_ValueError, "%s does not fit 32 bits", name);
    return v <= INT32_MAX && v >= INT32_MIN;
}

static int matrix(const Tensor *t)
{
    if (!given(t)) return 0;
    if (t->nd != 2) PyErr_Format(PyExc_ValueError, "%s must have 2 dimensions", t->name);
    return t->nd == 2;
}

/* (logits, score, renorm, scale, ids, w, stream) -> status */
static PyObject *py_router_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor l, ids, w;
    int code, renorm, status;
    int64_t score;
    float scale;
    mhc_stream_t s;
    if (!nargs(n, 7) || !look(a[0], "logits", &l) || !look(a[4], "ids", &ids) || !look(a[5], "w", &w) ||
        !activation(&l, 2, &code) || !contiguous(&l) || !matrix(&ids))
        return NULL;
    const int64_t T = l.d[0], E = l.d[1], k = ids.d[1];
    if (!exact(&ids, I32, 2, T, k, 0) || !exact(&w, FP32, 2, T, k, 0) || !whole(a[1], &score) ||
        (renorm = PyObject_IsTrue(a[2])) < 0 || !real(a[3], &scale) || !handle(a[6], &s) ||
        !small(E, "E") || !small(k, "k") || !small(score, "score"))
        return NULL;
    CALL(status, fn.router_fwd(l.ptr, (mhc_dtype)code, T, (int)E, (int)k, (mhc_score)score, renorm,
                               scale, ids.ptr, w.ptr, s))
    return PyLong_FromLong(status);
}

/* (dw, logits, ids, score, renorm, scale, dlogits, stream) -> status */
static PyObject *py_router_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor dw, l, ids, dl;
    int code, renorm, status;
    int64_t score;
    float scale;
    mhc_stream_t s;
    if (!nargs(n, 8) || !look(a[0], "dw", &dw) || !look(a[1], "logits", &l) || !look(a[2], "ids", &ids) ||
        !look(a[6], "dlogits", &dl) || !activation(&l, 2, &code) || !contiguous(&l) || !matrix(&ids))
        return NULL;
    const int64_t T = l.d[0], E = l.d[1], k = ids.d[1];
    if (!exact(&dw, FP32, 2, T, k, 0) || !exact(&ids, I32, 2, T, k, 0) ||
        !exact(&dl, code, 2, T, E, 0) || !whole(a[3], &score) ||
        (renorm = PyObject_IsTrue(a[4])) < 0 || !real(a[5], &scale) || !handle(a[7], &s) ||
        !small(E, "E") || !small(k, "k") || !small(score, "score"))
        return NULL;
    CALL(status, fn.router_bwd(dw.ptr, l.ptr, (mhc_dtype)code, ids.ptr, T, (int)E, (int)k,
                               (mhc_score)score, renorm, scale, dl.ptr, s))
    return PyLong_FromLong(status);
}

/* (ids, align, counts, offsets, row_of, slot_of, stream) -> status */
static PyObject *py_sort(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor ids, counts, offsets, row, slot;
    int64_t align;
    mhc_stream_t s;
    int status;
    if (!nargs(n, 7) || !look(a[0], "ids", &ids) || !look(a[2], "counts", &counts) ||
        !look(a[3], "offsets", &offsets) || !look(a[4], "row_of", &row) ||
        !look(a[5], "slot_of", &slot) || !matrix(&ids) || !given(&counts) || !given(&slot))
        return NULL;
    const int64_t T = ids.d[0], k = ids.d[1], E = counts.nd ? counts.d[0] : 0;
    const int64_t R = slot.nd ? slot.d[0] : 0;
    if (!exact(&ids, I32, 2, T, k, 0) || !exact(&counts, I32, 1, E, 0, 0) ||
        !exact(&offsets, I32, 1, E + 1, 0, 0) || !exact(&row, I32, 2, T, k, 0) ||
        !exact(&slot, I32, 1, R, 0, 0) || !whole(a[1], &align) || !handle(a[6], &s) ||
        !small(k, "k") || !small(E, "E") || !small(align, "align"))
        return NULL;
    CALL(status, fn.sort(ids.ptr, T, (int)k, (int)E, (int)align, R, counts.ptr, offsets.ptr, row.ptr,
                         slot.ptr, s))
    return PyLong_FromLong(status);
}

/* (x, row_of, slot_of, xs, stream) -> status */
static PyObject *py_dispatch_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor x, row, slot, xs;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 5) || !look(a[0], "x", &x) || !look(a[1], "row_of", &row) ||
        !look(a[2], "slot_of", &slot) || !look(a[3], "xs", &xs) || !activation(&x, 2, &code) ||
        !contiguous(&x) || !matrix(&row) || !matrix(&xs))
        return NULL;
    const int64_t T = x.d[0], C = x.d[1], k = row.d[1], R = xs.d[0];
    if (!exact(&row, I32, 2, T, k, 0) || !exact(&slot, I32, 1, R, 0, 0) ||
        !exact(&xs, code, 2, R, C, 0) || !handle(a[4], &s) || !small(k, "k"))
        return NULL;
    CALL(status, fn.dispatch_fwd(x.ptr, (mhc_dtype)code, row.ptr, slot.ptr, T, (int)k, R, C, xs.ptr, s))
    return PyLong_FromLong(status);
}

/* (dxs, row_of, dx, stream) -> status */
static PyObject *py_dispatch_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor dxs, row, dx;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 4) || !look(a[0], "dxs", &dxs) || !look(a[1], "row_of", &row) ||
        !look(a[2], "dx", &dx) || !activation(&dxs, 2, &code) || !contiguous(&dxs) || !matrix(&row))
        return NULL;
    const int64_t R = dxs.d[0], C = dxs.d[1], T = row.d[0], k = row.d[1];
    if (!exact(&row, I32, 2, T, k, 0) || !exact(&dx, code, 2, T, C, 0) || !handle(a[3], &s) ||
        !small(k, "k"))
        return NULL;
    CALL(status, fn.dispatch_bwd(dxs.ptr, (mhc_dtype)code, row.ptr, T, (int)k, R, C, dx.ptr, s))
    return PyLong_FromLong(status);
}

/* (ys, w, row_of, f, stream) -> status */
static PyObject *py_combine_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor ys, w, row, f;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 5) || !look(a[0], "ys", &ys) || !look(a[1], "w", &w) || !look(a[2], "row_of", &row) ||
        !look(a[3], "f", &f) || !activation(&ys, 2, &code) || !contiguous(&ys) || !matrix(&row))
        return NULL;
    const int64_t R = ys.d[0], C = ys.d[1], T = row.d[0], k = row.d[1];
    if (!exact(&w, FP32, 2, T, k, 1) || !exact(&row, I32, 2, T, k, 0) ||
        !exact(&f, code, 2, T, C, 0) || !handle(a[4], &s) || !small(k, "k"))
        return NULL;
    CALL(status, fn.combine_fwd(ys.ptr, (mhc_dtype)code, w.ptr, row.ptr, T, (int)k, R, C, f.ptr, s))
    return PyLong_FromLong(status);
}

/* (df, ys, w, row_of, slot_of, dys, dw, stream) -> status */
static PyObject *py_combine_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor df, ys, w, row, slot, dys, dw;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 8) || !look(a[0], "df", &df) || !look(a[1], "ys", &ys) || !look(a[2], "w", &w) ||
        !look(a[3], "row_of", &row) || !look(a[4], "slot_of", &slot) || !look(a[5], "dys", &dys) ||
        !look(a[6], "dw", &dw) || !activation(&dys, 2, &code) || !contiguous(&dys) || !matrix(&row))
        return NULL;
    const int64_t R = dys.d[0], C = dys.d[1], T = row.d[0], k = row.d[1];
    if (!exact(&df, code, 2, T, C, 0) || !exact(&ys, code, 2, R, C, 1) ||
        !exact(&w, FP32, 2, T, k, 1) || !exact(&row, I32, 2, T, k, 0) ||
        !exact(&slot, I32, 1, R, 0, 0) || !exact(&dw, FP32, 2, T, k, 1) || !handle(a[7], &s) ||
        !small(k, "k"))
        return NULL;
    CALL(status, fn.combine_bwd(df.ptr, ys.ptr, (mhc_dtype)code, w.ptr, row.ptr, slot.ptr, T, (int)k, R,
                                C, dys.ptr, dw.ptr, s))
    return PyLong_FromLong(status);
}

/* A contiguous [G, a, b] tensor of this type, [a, b] where nd is 2; `opt`: may be None. */
static int batch(Tensor *t, int code, int nd, int64_t G, int64_t a, int64_t b, int opt)
{
    if (nd == 2) return exact(t, code, 2, a, b, opt);
    if (opt && !t->obj) return 1;
    if (!given(t)) return 0;
    if (t->code != code) return wrong_type(t, type_names[code]);
    if (t->nd != 3 || t->d[0] != G || t->d[1] != a || t->d[2] != b) return wrong_shape(t, 3, G, a, b);
    return contiguous(t);
}

/* An 8-bit matrix of nd dimensions; sets *format. */
static int eight(Tensor *t, int nd, int *format)
{
    if (!given(t)) return 0;
    if (t->code != E4M3 && t->code != E5M2) return wrong_type(t, "float8_e4m3fn or float8_e5m2");
    *format = t->code == E5M2 ? MHC_E5M2 : MHC_E4M3;
    if (t->nd != nd) PyErr_Format(PyExc_ValueError, "%s must have %d dimensions", t->name, nd);
    return t->nd == nd;
}

static int64_t blocks(int64_t n) { return (n + 127) / 128; }

/* q, s, qt, st of a quantisation of [G, R, C] ([R, C] where nd is 2). */
typedef struct {
    Tensor q, s, qt, st;
    int format;
} Quant;

static int quantised(PyObject *const *a, Quant *x, int nd, int64_t G, int64_t R, int64_t C, int tiles)
{
    if (!look(a[0], "q", &x->q) || !look(a[1], "s", &x->s) || !look(a[2], "qt", &x->qt) ||
        !look(a[3], "st", &x->st))
        return 0;
    x->format = MHC_E4M3;
    const Tensor *one = x->q.obj ? &x->q : &x->qt;
    if (one->obj && !eight((Tensor *)one, nd, &x->format)) return 0;
    const int code = x->format == MHC_E5M2 ? E5M2 : E4M3;
    return batch(&x->q, code, nd, G, R, C, 1) && batch(&x->qt, code, nd, G, C, R, 1) &&
           batch(&x->s, FP32, nd, G, blocks(C), tiles ? blocks(R) : R, !x->q.obj) &&
           batch(&x->st, FP32, nd, G, blocks(R), tiles ? blocks(C) : C, !x->qt.obj);
}

/* (x, q, s, qt, st, tiles, stream) -> status */
static PyObject *py_fp8_quant(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor x;
    Quant o;
    int code, tiles, status;
    mhc_stream_t s;
    if (!nargs(n, 7) || !look(a[0], "x", &x) || !given(&x) || (tiles = PyObject_IsTrue(a[5])) < 0 ||
        !activation(&x, x.nd == 3 ? 3 : 2, &code) || !contiguous(&x))
        return NULL;
    const int64_t G = x.nd == 3 ? x.d[0] : 1, R = x.d[x.nd - 2], C = x.d[x.nd - 1];
    if (!quantised(a + 1, &o, x.nd, G, R, C, tiles) || !handle(a[6], &s)) return NULL;
    CALL(status, fn.fp8_quant(x.ptr, (mhc_dtype)code, G, R, C, (mhc_fp8)o.format, tiles, o.q.ptr,
                              o.s.ptr, o.qt.ptr, o.st.ptr, s))
    return PyLong_FromLong(status);
}

/* h [R, 2F] */
static int gate_up(Tensor *h, int *code)
{
    if (!activation(h, 2, code) || !contiguous(h)) return 0;
    if (h->d[1] % 2) PyErr_Format(PyExc_ValueError, "h: its %lld columns are no two halves",
                                  (long long)h->d[1]);
    return h->d[1] % 2 == 0;
}

/* (h, a, q, s, qt, st, stream) -> status */
static PyObject *py_fp8_swiglu_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor h, y;
    Quant o;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 7) || !look(a[0], "h", &h) || !look(a[1], "a", &y) || !gate_up(&h, &code)) return NULL;
    const int64_t R = h.d[0], F = h.d[1] / 2;
    if (!exact(&y, code, 2, R, F, 1) || !quantised(a + 2, &o, 2, 1, R, F, 0) || !handle(a[6], &s))
        return NULL;
    CALL(status, fn.fp8_swiglu_fwd(h.ptr, (mhc_dtype)code, R, F, (mhc_fp8)o.format, y.ptr, o.q.ptr,
                                   o.s.ptr, o.qt.ptr, o.st.ptr, s))
    return PyLong_FromLong(status);
}

/* (da, h, dh, q, s, qt, st, stream) -> status */
static PyObject *py_fp8_swiglu_bwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor da, h, y;
    Quant o;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 8) || !look(a[0], "da", &da) || !look(a[1], "h", &h) || !look(a[2], "dh", &y) ||
        !gate_up(&h, &code))
        return NULL;
    const int64_t R = h.d[0], F = h.d[1] / 2;
    if (!exact(&da, code, 2, R, F, 0) || !exact(&y, code, 2, R, 2 * F, 1) ||
        !quantised(a + 3, &o, 2, 1, R, 2 * F, 0) || !handle(a[7], &s))
        return NULL;
    CALL(status, fn.fp8_swiglu_bwd(da.ptr, h.ptr, (mhc_dtype)code, R, F, (mhc_fp8)o.format, y.ptr,
                                   o.q.ptr, o.s.ptr, o.qt.ptr, o.st.ptr, s))
    return PyLong_FromLong(status);
}

/* (a, sa, b, sb, offsets, out, stream) -> status */
static PyObject *py_fp8_gemm(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor x, sx, w, sw, off, out;
    int fa, fb, code, status;
    mhc_stream_t s;
    if (!nargs(n, 7) || !look(a[0], "a", &x) || !look(a[1], "sa", &sx) || !look(a[2], "b", &w) ||
        !look(a[3], "sb", &sw) || !look(a[4], "offsets", &off) || !look(a[5], "out", &out) ||
        !eight(&x, 2, &fa) || !eight(&w, 3, &fb) || !activation(&out, 2, &code) || !contiguous(&x) ||
        !contiguous(&w))
        return NULL;
    const int64_t R = x.d[0], K = x.d[1], G = w.d[0], N = w.d[1];
    if (!batch(&w, w.code, 3, G, N, K, 0) || !exact(&sx, FP32, 2, blocks(K), R, 0) ||
        !batch(&sw, FP32, 3, G, blocks(K), blocks(N), 0) || !exact(&off, I32, 1, G + 1, 0, 1) ||
        !exact(&out, code, 2, R, N, 0) || !handle(a[6], &s))
        return NULL;
    CALL(status, fn.fp8_gemm(x.ptr, (mhc_fp8)fa, sx.ptr, w.ptr, (mhc_fp8)fb, sw.ptr, off.ptr, G, R, N,
                             K, (mhc_dtype)code, out.ptr, s))
    return PyLong_FromLong(status);
}

/* (at, sat, bt, sbt, offsets, out, stream) -> status */
static PyObject *py_fp8_wgrad(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor x, sx, w, sw, off, out;
    int fa, fb, code, status;
    mhc_stream_t s;
    if (!nargs(n, 7) || !look(a[0], "at", &x) || !look(a[1], "sat", &sx) || !look(a[2], "bt", &w) ||
        !look(a[3], "sbt", &sw) || !look(a[4], "offsets", &off) || !look(a[5], "out", &out) ||
        !eight(&x, 2, &fa) || !eight(&w, 2, &fb) || !activation(&out, 3, &code) || !contiguous(&x))
        return NULL;
    const int64_t M = x.d[0], R = x.d[1], G = out.d[0], N = w.d[0];
    if (!exact(&w, w.code, 2, N, R, 0) || !exact(&sx, FP32, 2, blocks(R), M, 0) ||
        !exact(&sw, FP32, 2, blocks(R), N, 0) || !exact(&off, I32, 1, G + 1, 0, 1) ||
        !batch(&out, code, 3, G, M, N, 0) || !handle(a[6], &s))
        return NULL;
    CALL(status, fn.fp8_wgrad(x.ptr, (mhc_fp8)fa, sx.ptr, w.ptr, (mhc_fp8)fb, sw.ptr, off.ptr, G, R, M,
                              N, (mhc_dtype)code, out.ptr, s))
    return PyLong_FromLong(status);
}

/* (x, ids, w, w1, w2, f, ws, s1, s2, stream) -> status */
static PyObject *py_few_fwd(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    Tensor x, ids, w, w1, w2, f, ws, s1, s2;
    int code, status;
    mhc_stream_t s;
    if (!nargs(n, 10) || !look(a[0], "x", &x) || !look(a[1], "ids", &ids) || !look(a[2], "w", &w) ||
        !look(a[3], "w1", &w1) || !look(a[4], "w2", &w2) || !look(a[5], "f", &f) ||
        !look(a[6], "ws", &ws) || !look(a[7], "s1", &s1) || !look(a[8], "s2", &s2) ||
        !activation(&x, 2, &code) || !contiguous(&x) || !matrix(&ids) || !given(&w1) || !given(&w2))
        return NULL;
    const int64_t T = x.d[0], C = x.d[1], k = ids.d[1];
    if (w2.nd != 3) {
        PyErr_SetString(PyExc_ValueError, "w2 must have 3 dimensions");
        return NULL;
    }
    const int64_t E = w2.d[0], F = w2.d[2];
    const int wc = s1.obj || s2.obj ? E4M3 : code;
    if (!exact(&ids, I32, 2, T, k, 0) || !exact(&w, FP32, 2, T, k, 0) ||
        !batch(&w1, wc, 3, E, 2 * F, C, 0) || !batch(&w2, wc, 3, E, C, F, 0) ||
        !batch(&s1, FP32, 3, E, blocks(C), blocks(2 * F), wc != E4M3) ||
        !batch(&s2, FP32, 3, E, blocks(F), blocks(C), wc != E4M3) || !exact(&f, code, 2, T, C, 0) ||
        !exact(&ws, U8, 1, ws.numel, 0, 1) || !handle(a[9], &s) || !small(k, "k") || !small(E, "E"))
        return NULL;
    CALL(status, fn.few_fwd(x.ptr, (mhc_dtype)code, ids.ptr, w.ptr, w1.ptr, s1.ptr, w2.ptr, s2.ptr, T,
                            (int)k, (int)E, C, F, f.ptr, ws.ptr, (size_t)ws.numel, s))
    return PyLong_FromLong(status);
}

/* setup(torch.Tensor, (the dtypes in the order of type_names), (entry points' addresses)) */
static PyObject *py_setup(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *type, *types, *entries;
    if (!PyArg_ParseTuple(args, "OO!O!", &type, &PyTuple_Type, &types, &PyTuple_Type, &entries))
        return NULL;
    const Py_ssize_t ne = (Py_ssize_t)(sizeof fn / sizeof(void *));
    if (!PyType_Check(type) || PyTuple_GET_SIZE(types) != NTYPES || PyTuple_GET_SIZE(entries) != ne) {
        PyErr_SetString(PyExc_TypeError, "setup: a type, its dtypes and the entry points' addresses");
        return NULL;
    }
    void *p[sizeof fn / sizeof(void *)];
    for (Py_ssize_t i = 0; i < ne; ++i)
        p[i] = (void *)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(entries, i));
    if (PyErr_Occurred()) return NULL;
    memcpy(&fn, p, sizeof fn);
    Py_INCREF(type);
    Py_XSETREF(tensor_type, type);
    for (int i = 0; i < NTYPES; ++i) {
        PyObject *d = PyTuple_GET_ITEM(types, i);
        Py_INCREF(d);
        Py_XSETREF(dtypes[i], d);
    }
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, NULL},
    ENTRY(qk_fwd), ENTRY(qk_bwd), ENTRY(router_fwd), ENTRY(router_bwd), ENTRY(sort),
    ENTRY(dispatch_fwd), ENTRY(dispatch_bwd), ENTRY(combine_fwd), ENTRY(combine_bwd),
    ENTRY(fp8_quant), ENTRY(fp8_swiglu_fwd), ENTRY(fp8_swiglu_bwd), ENTRY(fp8_gemm),
    ENTRY(fp8_wgrad), ENTRY(few_fwd),
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_stride = PyUnicode_InternFromString("stride");
    if (!s_shape || !s_dtype || !s_is_cuda || !s_is_contiguous || !s_data_ptr || !s_stride) return NULL;
    return PyModule_Create(&module);
}
