/*
 * kda_fastcall.c -- argument checks and calls of the 8-bit operators' Python
 * binding, as a small CPython extension.
 *
 * A decode step's norm or projection takes 2-4 us on the GPU, less than the
 * interpreter needs to read the shapes, types, devices and pointers of its
 * six tensors one attribute at a time and to marshal them through ctypes
 * (3.6 us of a 6.5 us call). The functions here make the same checks and the
 * same library calls. They know torch only through the objects that setup()
 * is given.
 *
 * Each returns the library's status (0 = KDA_OK), or -1 where the tensors live
 * on another device than the current one and no stream of theirs was named: the
 * caller makes that device current and calls again.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef int (*add_rmsnorm_fn)(const void *, const void *, const float *, void *, void *, float *, int64_t, int, int,
                              int, float, void *);
typedef int (*gated_rmsnorm_fn)(const void *, const void *, const float *, void *, float *, int64_t, int, int, int,
                                int, float, void *);
typedef int (*linear_fn)(const void *, const float *, const void *, const float *, void *, int64_t, int, int, int64_t,
                         int64_t, int64_t, int, void *);

static struct {
    add_rmsnorm_fn add_rmsnorm;
    gated_rmsnorm_fn gated_rmsnorm;
    linear_fn linear;
    PyObject *f32, *bf16, *f8;            /* torch dtypes */
    PyObject *get_device, *raw_stream;    /* current device index; device index -> stream handle */
    int ready;
} S;

static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_stride, *n_cuda_stream,
    *n_device_index;

enum { DT_F32 = 0, DT_BF16 = 1, DT_F8 = 2, DT_OTHER = -1 };

typedef struct {
    int64_t dim[4];
    int nd, dt, contiguous;
    long dev;
    void *p;
} Tensor;

static int long_of(PyObject *o, long long *v) { /* takes the reference */
    if (o == NULL) return 0;
    *v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*v == -1 && PyErr_Occurred());
}

/* Shape, dtype, device and pointer of a tensor, and with `whole` whether it is contiguous. */
static int look(PyObject *t, Tensor *r, int whole) {
    PyObject *o = PyObject_GetAttr(t, n_shape);
    if (o == NULL) return 0;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) > 4) {
        Py_DECREF(o);
        PyErr_SetString(PyExc_ValueError, "shape mismatch");
        return 0;
    }
    r->nd = (int)PyTuple_GET_SIZE(o);
    for (int i = 0; i < r->nd; ++i) {
        r->dim[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        if (r->dim[i] == -1 && PyErr_Occurred()) {
            Py_DECREF(o);
            return 0;
        }
    }
    Py_DECREF(o);
    if ((o = PyObject_GetAttr(t, n_dtype)) == NULL) return 0;
    r->dt = o == S.f32 ? DT_F32 : o == S.bf16 ? DT_BF16 : o == S.f8 ? DT_F8 : DT_OTHER;
    Py_DECREF(o);
    long long v;
    if (!long_of(PyObject_CallMethodNoArgs(t, n_get_device), &v)) return 0;
    r->dev = (long)v;
    r->contiguous = 1;
    if (whole) {
        if ((o = PyObject_CallMethodNoArgs(t, n_is_contiguous)) == NULL) return 0;
        r->contiguous = PyObject_IsTrue(o);
        Py_DECREF(o);
        if (r->contiguous < 0) return 0;
    }
    if ((o = PyObject_CallMethodNoArgs(t, n_data_ptr)) == NULL) return 0;
    r->p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return !(r->p == NULL && PyErr_Occurred());
}

static int is_shape(const Tensor *t, int nd, int64_t a, int64_t b, int64_t c) {
    return t->nd == nd && t->dim[0] == a && (nd < 2 || t->dim[1] == b) && (nd < 3 || t->dim[2] == c);
}

static PyObject *bad(PyObject *kind, const char *what) {
    PyErr_SetString(kind, what);
    return NULL;
}
static const char SHAPE[] = "shape mismatch", CODES[] = "8-bit codes must be torch.float8_e4m3fn",
                  FLOATS[] = "scales and norm weights must be float32",
                  DTYPE[] = "unsupported dtype; use float32 or bfloat16";

/* Every tensor on one CUDA device, those that have to be contiguous so. */
static int one_device(const Tensor *t, const Tensor *const *others, int n) {
    int same = 1, whole = t->contiguous;
    for (int i = 0; i < n; ++i) {
        same = same && others[i]->dev == t->dev;
        whole = whole && others[i]->contiguous;
    }
    if (t->dev >= 0 && same && whole) return 1;
    PyErr_SetString(PyExc_ValueError, t->dev < 0 ? "tensors must be on a CUDA device"
                                      : !same    ? "tensors must be on one CUDA device"
                                                 : "tensors must be contiguous");
    return 0;
}

/* Handle of `stream`, or of the current stream of device `dev` where it is None. 1: found, 0: error set (a
 * stream of another device among them, where the kernels would run beside the tensors' memory), -1: a default
 * stream (whose handle, 0, names no device) of a device that is not the current one, or None there. */
static int find_stream(PyObject *stream, long dev, void **handle) {
    PyObject *o;
    *handle = NULL;
    if (stream != Py_None) {
        long long on;
        if (long_of(PyObject_GetAttr(stream, n_device_index), &on)) {
            if (on != dev) {
                PyErr_SetString(PyExc_ValueError, "stream must be on the tensors' device");
                return 0;
            }
        } else if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear(); /* a stream that does not say */
        } else {
            return 0;
        }
        if ((o = PyObject_GetAttr(stream, n_cuda_stream)) == NULL) return 0;
        *handle = PyLong_AsVoidPtr(o);
        Py_DECREF(o);
        if (*handle != NULL) return 1;
        if (PyErr_Occurred()) return 0;
    }
    long long cur;
    if (!long_of(PyObject_CallNoArgs(S.get_device), &cur)) return 0;
    if (cur != dev) return -1;
    if (stream != Py_None) return 1;
    PyObject *d = PyLong_FromLong(dev);
    if (d == NULL) return 0;
    o = PyObject_CallOneArg(S.raw_stream, d);
    Py_DECREF(d);
    if (o == NULL) return 0;
    *handle = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return *handle == NULL && PyErr_Occurred() ? 0 : 1;
}

static int arity(Py_ssize_t got, Py_ssize_t want) {
    if (!S.ready) {
        PyErr_SetString(PyExc_RuntimeError, "setup() has not been called");
        return 0;
    }
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return 0;
    }
    return 1;
}

/* (x, weight, y, scales, residual, sum_out, eps, stream) */
static PyObject *add_rmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 8)) return NULL;
    Tensor x, w, y, s, r = {.p = NULL}, so = {.p = NULL};
    const int has_r = a[4] != Py_None, has_so = a[5] != Py_None;
    if (!look(a[0], &x, 1) || !look(a[1], &w, 1) || !look(a[2], &y, 1) || !look(a[3], &s, 1) ||
        (has_r && !look(a[4], &r, 1)) || (has_so && !look(a[5], &so, 1)))
        return NULL;
    if (x.nd != 2) return bad(PyExc_ValueError, SHAPE);
    const int64_t T = x.dim[0], N = x.dim[1];
    if (!is_shape(&w, 1, N, 0, 0) || !is_shape(&y, 2, T, N, 0) || !is_shape(&s, 2, (N + 127) / 128, T, 0) ||
        (has_r && !is_shape(&r, 2, T, N, 0)) || (has_so && !is_shape(&so, 2, T, N, 0)) || N > INT32_MAX)
        return bad(PyExc_ValueError, SHAPE);
    if (y.dt != DT_F8) return bad(PyExc_TypeError, CODES);
    if (w.dt != DT_F32 || s.dt != DT_F32) return bad(PyExc_TypeError, FLOATS);
    if (has_r && has_so && r.dt != so.dt) return bad(PyExc_TypeError, "sum_out must have residual's dtype");
    const int res = has_r ? r.dt : has_so ? so.dt : x.dt;
    if ((x.dt != DT_F32 && x.dt != DT_BF16) || (res != DT_F32 && res != DT_BF16)) return bad(PyExc_TypeError, DTYPE);
    const Tensor *others[] = {&w, &y, &s, has_r ? &r : &w, has_so ? &so : &w};
    if (!one_device(&x, others, 5)) return NULL;
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    void *h = NULL;
    const int found = find_stream(a[7], x.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = S.add_rmsnorm(x.p, r.p, w.p, so.p, y.p, s.p, T, (int)N, x.dt, res, (float)eps, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (o, gate, weight, y, scales, act code, eps, stream) */
static PyObject *gated_rmsnorm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 8)) return NULL;
    Tensor o, g, w, y, s;
    if (!look(a[0], &o, 1) || !look(a[1], &g, 1) || !look(a[2], &w, 1) || !look(a[3], &y, 1) || !look(a[4], &s, 1))
        return NULL;
    if (o.nd != 3) return bad(PyExc_ValueError, SHAPE);
    const int64_t T = o.dim[0], H = o.dim[1], D = o.dim[2];
    if (!is_shape(&g, 3, T, H, D) || !is_shape(&y, 3, T, H, D) || !is_shape(&w, 1, D, 0, 0) ||
        !is_shape(&s, 2, (H * D + 127) / 128, T, 0) || H > INT32_MAX || D > INT32_MAX)
        return bad(PyExc_ValueError, SHAPE);
    if (g.dt != o.dt) return bad(PyExc_TypeError, "gate must have o's dtype");
    if (y.dt != DT_F8) return bad(PyExc_TypeError, CODES);
    if (w.dt != DT_F32 || s.dt != DT_F32) return bad(PyExc_TypeError, FLOATS);
    if (o.dt != DT_F32 && o.dt != DT_BF16) return bad(PyExc_TypeError, DTYPE);
    const Tensor *others[] = {&g, &w, &y, &s};
    if (!one_device(&o, others, 4)) return NULL;
    const long act = PyLong_AsLong(a[5]);
    if (act == -1 && PyErr_Occurred()) return NULL;
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    void *h = NULL;
    const int found = find_stream(a[7], o.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = S.gated_rmsnorm(o.p, g.p, w.p, y.p, s.p, T, (int)H, (int)D, o.dt, (int)act, (float)eps, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* Row stride of a matrix whose rows are contiguous; a single row's is its length. */
static int row_stride(PyObject *t, const Tensor *d, int64_t *ld) {
    PyObject *o = PyObject_CallMethodNoArgs(t, n_stride);
    if (o == NULL) return 0;
    const int64_t outer = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0)), inner = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1));
    Py_DECREF(o);
    if (inner != 1 && d->dim[1] > 1) {
        PyErr_SetString(PyExc_ValueError, "rows must be contiguous");
        return 0;
    }
    *ld = d->dim[0] > 1 ? outer : d->dim[1];
    return 1;
}

/* (a, a_scales, w, w_scales, y, stream) */
static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 6)) return NULL;
    Tensor x, sa, w, sw, y;
    if (!look(a[0], &x, 0) || !look(a[1], &sa, 1) || !look(a[2], &w, 0) || !look(a[3], &sw, 1) || !look(a[4], &y, 0))
        return NULL;
    if (x.nd != 2 || w.nd != 2) return bad(PyExc_ValueError, SHAPE);
    const int64_t M = x.dim[0], K = x.dim[1], N = w.dim[0], kb = (K + 127) / 128;
    if (w.dim[1] != K || !is_shape(&y, 2, M, N, 0) || !is_shape(&sa, 2, kb, M, 0) ||
        !is_shape(&sw, 2, (N + 127) / 128, kb, 0) || N > INT32_MAX || K > INT32_MAX)
        return bad(PyExc_ValueError, SHAPE);
    if (x.dt != DT_F8 || w.dt != DT_F8) return bad(PyExc_TypeError, CODES);
    if (sa.dt != DT_F32 || sw.dt != DT_F32) return bad(PyExc_TypeError, FLOATS);
    if (y.dt != DT_F32 && y.dt != DT_BF16) return bad(PyExc_TypeError, DTYPE);
    const Tensor *others[] = {&sa, &w, &sw, &y};
    if (!one_device(&x, others, 4)) return NULL;
    int64_t lda, ldw, ldy;
    if (!row_stride(a[0], &x, &lda) || !row_stride(a[2], &w, &ldw) || !row_stride(a[4], &y, &ldy)) return NULL;
    void *h = NULL;
    const int found = find_stream(a[5], x.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = S.linear(x.p, sa.p, w.p, sw.p, y.p, M, (int)N, (int)K, lda, ldw, ldy, y.dt, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (address of kda_add_rmsnorm_fp8, of kda_gated_rmsnorm_fp8, of kda_fp8_linear, torch.float32, torch.bfloat16,
 * torch.float8_e4m3fn, current device index (callable), device index -> stream handle (callable)) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *p[3], *o[5];
    if (!PyArg_ParseTuple(args, "OOOOOOOO", &p[0], &p[1], &p[2], &o[0], &o[1], &o[2], &o[3], &o[4])) return NULL;
    void *f[3];
    for (int i = 0; i < 3; ++i)
        if ((f[i] = PyLong_AsVoidPtr(p[i])) == NULL)
            return PyErr_Occurred() ? NULL : bad(PyExc_ValueError, "a function's address is NULL");
    S.add_rmsnorm = (add_rmsnorm_fn)f[0];
    S.gated_rmsnorm = (gated_rmsnorm_fn)f[1];
    S.linear = (linear_fn)f[2];
    PyObject **slot[5] = {&S.f32, &S.bf16, &S.f8, &S.get_device, &S.raw_stream};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*slot[i], o[i]);
    }
    S.ready = 1;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Library functions and torch objects that the calls use."},
    {"add_rmsnorm", (PyCFunction)(void (*)(void))add_rmsnorm, METH_FASTCALL, "kda_add_rmsnorm_fp8"},
    {"gated_rmsnorm", (PyCFunction)(void (*)(void))gated_rmsnorm, METH_FASTCALL, "kda_gated_rmsnorm_fp8"},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, "kda_fp8_linear"},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "kda_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit_kda_fastcall(void) {
    struct {
        PyObject **name;
        const char *text;
    } names[] = {{&n_dtype, "dtype"},       {&n_shape, "shape"},       {&n_get_device, "get_device"},
                 {&n_is_contiguous, "is_contiguous"}, {&n_data_ptr, "data_ptr"}, {&n_stride, "stride"},
                 {&n_cuda_stream, "cuda_stream"}, {&n_device_index, "device_index"}};
    for (size_t i = 0; i < sizeof(names) / sizeof(names[0]); ++i)
        if ((*names[i].name = PyUnicode_InternFromString(names[i].text)) == NULL) return NULL;
    return PyModule_Create(&module);
}
