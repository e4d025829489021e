/*
 * kda_fastcall.c -- argument checks and calls of the Python binding of the 8-bit
 * operators and of the softmax-attention layers', as a small CPython extension.
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
#include <math.h>
#include <stdint.h>

typedef int (*add_rmsnorm_fn)(const void *, const void *, const float *, void *, void *, float *, int64_t, int, int,
                              int, float, void *);
typedef int (*gated_rmsnorm_fn)(const void *, const void *, const float *, void *, float *, int64_t, int, int, int,
                                int, float, void *);
typedef int (*linear_fn)(const void *, const float *, const void *, const float *, void *, int64_t, int, int, int64_t,
                         int64_t, int64_t, int, void *);

typedef int (*norm_rope_fn)(const void *, const void *, void *, void *, const float *, const float *, const int64_t *,
                            const double *, int64_t, int, int, int, int, int64_t, int64_t, int64_t, int64_t, int, float,
                            int, void *);
typedef int (*kv4_append_fn)(const void *, const void *, void *, const int32_t *, const int64_t *, const int64_t *, int,
                             int64_t, int, int, int, int64_t, int, int64_t, int64_t, int64_t, int, void *);
typedef int (*kv4_read_fn)(const void *, const int32_t *, const int64_t *, const int64_t *, void *, void *, int, int64_t,
                           int, int, int, int64_t, int, int64_t, int64_t, int64_t, int, void *);
typedef int (*kv4_attention_fn)(const void *, const void *, const int32_t *, const int64_t *, const int64_t *, void *,
                                float *, int, int64_t, int, int, int, int, int64_t, int, int64_t, int64_t, int64_t, float,
                                int, int64_t, int, void *, size_t, void *);
typedef size_t (*kv4_space_fn)(int, int64_t, int, int, int, int, int, int, int64_t, int);

static struct {
    add_rmsnorm_fn add_rmsnorm;
    gated_rmsnorm_fn gated_rmsnorm;
    linear_fn linear;
    norm_rope_fn norm_rope;
    kv4_append_fn kv4_append;
    kv4_read_fn kv4_read;
    kv4_attention_fn kv4_attention;
    kv4_space_fn kv4_space;
    PyObject *f32, *bf16, *f8, *f64, *i64, *i32, *u8; /* torch dtypes */
    PyObject *get_device, *raw_stream;    /* current device index; device index -> stream handle */
    int ready;
} S;

static PyObject *n_dtype, *n_shape, *n_get_device, *n_is_contiguous, *n_data_ptr, *n_stride, *n_cuda_stream,
    *n_device_index;

enum { DT_F32 = 0, DT_BF16 = 1, DT_F8 = 2, DT_F64, DT_I64, DT_I32, DT_U8, DT_OTHER = -1 };

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
    r->dt = o == S.f32 ? DT_F32 : o == S.bf16 ? DT_BF16 : o == S.f8 ? DT_F8 : o == S.i64 ? DT_I64 : o == S.i32 ? DT_I32
          : o == S.u8 ? DT_U8 : o == S.f64 ? DT_F64 : DT_OTHER;
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

/* Token stride of a [T,H,D] tensor whose heads and channels are contiguous. */
static int token_stride(PyObject *t, const Tensor *d, int64_t *ld) {
    PyObject *o = PyObject_CallMethodNoArgs(t, n_stride);
    if (o == NULL) return 0;
    int64_t st[3];
    for (int i = 0; i < 3; ++i) st[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    Py_DECREF(o);
    if (PyErr_Occurred()) return 0;
    if ((st[2] != 1 && d->dim[2] > 1) || (st[1] != d->dim[2] && d->dim[1] > 1)) {
        PyErr_SetString(PyExc_ValueError, "heads must be contiguous");
        return 0;
    }
    *ld = d->dim[0] > 1 ? st[0] : d->dim[1] * d->dim[2];
    return 1;
}

/* An optional tensor: looked at where it is there; p = NULL, dev = -2 and contiguous where it is None. */
static int look_at(PyObject *t, Tensor *r, int whole) {
    if (t != Py_None) return look(t, r, whole);
    *r = (Tensor){.p = NULL, .dt = DT_OTHER, .dev = -2, .contiguous = 1};
    return 1;
}
/* Like one_device, skipping what is absent. */
static int one_device_of(const Tensor *t, const Tensor *const *others, int n) {
    const Tensor *there[12];
    int m = 0;
    for (int i = 0; i < n; ++i)
        if (others[i]->dev != -2) there[m++] = others[i];
    return one_device(t, there, m);
}

/* (q, k, q_out, k_out, positions, inv_freq, q_weight, k_weight, eps, interleaved, stream) */
static PyObject *norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 11)) return NULL;
    Tensor q, k, qo, ko, pos, fr, qw, kw;
    if (!look(a[0], &q, 0) || !look_at(a[1], &k, 0) || !look(a[2], &qo, 0) || !look_at(a[3], &ko, 0) ||
        !look_at(a[4], &pos, 1) || !look_at(a[5], &fr, 1) || !look_at(a[6], &qw, 1) || !look_at(a[7], &kw, 1))
        return NULL;
    const int has_k = a[1] != Py_None, turns = a[5] != Py_None;
    if (has_k != (a[3] != Py_None) || turns != (a[4] != Py_None))
        return bad(PyExc_ValueError, "k and k_out, positions and inv_freq go together");
    if (q.nd != 3 || (has_k && k.nd != 3)) return bad(PyExc_ValueError, SHAPE);
    const int64_t T = q.dim[0], Hq = q.dim[1], D = q.dim[2], Hk = has_k ? k.dim[1] : 0, R = turns ? 2 * fr.dim[0] : 0;
    if (!is_shape(&qo, 3, T, Hq, D) || (has_k && (!is_shape(&k, 3, T, Hk, D) || !is_shape(&ko, 3, T, Hk, D))) ||
        (turns && (fr.nd != 1 || !is_shape(&pos, 1, T, 0, 0))) || (a[6] != Py_None && !is_shape(&qw, 1, D, 0, 0)) ||
        (a[7] != Py_None && !is_shape(&kw, 1, D, 0, 0)) || Hq > INT32_MAX || Hk > INT32_MAX || D > INT32_MAX ||
        R > INT32_MAX)
        return bad(PyExc_ValueError, SHAPE);
    if (qo.dt != q.dt || (has_k && (k.dt != q.dt || ko.dt != q.dt)))
        return bad(PyExc_TypeError, "q, k and the outputs must have one dtype");
    if (q.dt != DT_F32 && q.dt != DT_BF16) return bad(PyExc_TypeError, DTYPE);
    if (turns && pos.dt != DT_I64) return bad(PyExc_TypeError, "positions must be int64");
    if (turns && fr.dt != DT_F64) return bad(PyExc_TypeError, "inv_freq must be float64");
    if ((a[6] != Py_None && qw.dt != DT_F32) || (a[7] != Py_None && kw.dt != DT_F32)) return bad(PyExc_TypeError, FLOATS);
    const Tensor *others[] = {&k, &qo, &ko, &pos, &fr, &qw, &kw};
    if (!one_device_of(&q, others, 7)) return NULL;
    int64_t ld[4] = {0, 0, 0, 0};
    if (!token_stride(a[0], &q, ld) || (has_k && !token_stride(a[1], &k, ld + 1)) || !token_stride(a[2], &qo, ld + 2) ||
        (has_k && !token_stride(a[3], &ko, ld + 3)))
        return NULL;
    const double eps = PyFloat_AsDouble(a[8]);
    if (eps == -1.0 && PyErr_Occurred()) return NULL;
    const int inter = PyObject_IsTrue(a[9]);
    if (inter < 0) return NULL;
    void *h = NULL;
    const int found = find_stream(a[10], q.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = S.norm_rope(q.p, k.p, qo.p, ko.p, qw.p, kw.p, pos.p, fr.p, T, (int)Hq, (int)Hk, (int)D, (int)R, ld[0], ld[1], ld[2],
                     ld[3], inter, (float)eps, q.dt, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* A cache, the sequences in it and a tensor x [T,H,D] of new tokens. */
typedef struct {
    Tensor cache, table, lens, cu;
    int64_t B, T, Hk, D, pages, cols, table_stride;
    int page;
} Cached;

static int look_cached(PyObject *cache, PyObject *table, PyObject *lens, PyObject *cu, const Tensor *x, Cached *c) {
    if (!look(cache, &c->cache, 1) || !look(table, &c->table, 0) || !look(lens, &c->lens, 1) || !look_at(cu, &c->cu, 1))
        return 0;
    if (c->cache.nd != 4 || c->table.nd != 2 || c->lens.nd != 1 || x->nd != 3) return bad(PyExc_ValueError, SHAPE) != NULL;
    c->pages = c->cache.dim[0];
    c->Hk = c->cache.dim[1];
    c->B = c->lens.dim[0];
    c->T = x->dim[0];
    c->D = x->dim[2];
    c->cols = c->table.dim[1];
    if (c->cache.dim[3] != 18 * c->D || c->table.dim[0] != c->B || (cu != Py_None && !is_shape(&c->cu, 1, c->B + 1, 0, 0)) ||
        c->Hk > INT32_MAX || c->D > INT32_MAX || c->B > INT32_MAX || c->cols > INT32_MAX || c->cache.dim[2] > 1 << 20 ||
        x->dim[1] > INT32_MAX)
        return bad(PyExc_ValueError, SHAPE) != NULL;
    c->page = 16 * (int)c->cache.dim[2];
    if (c->cache.dt != DT_U8) return bad(PyExc_TypeError, "cache must be uint8") != NULL;
    if (c->table.dt != DT_I32) return bad(PyExc_TypeError, "block_table must be int32") != NULL;
    if (c->lens.dt != DT_I64 || (cu != Py_None && c->cu.dt != DT_I64))
        return bad(PyExc_TypeError, "lens and cu_seqlens must be int64") != NULL;
    if (x->dt != DT_F32 && x->dt != DT_BF16) return bad(PyExc_TypeError, DTYPE) != NULL;
    return row_stride(table, &c->table, &c->table_stride);
}

/* (k, v, cache, block_table, lens, cu_seqlens, stream, read) */
static PyObject *kv4_rows(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 8)) return NULL;
    Tensor k, v;
    Cached c;
    if (!look(a[0], &k, 0) || !look(a[1], &v, 0) || !look_cached(a[2], a[3], a[4], a[5], &k, &c)) return NULL;
    if (k.dim[1] != c.Hk || !is_shape(&v, 3, k.dim[0], k.dim[1], k.dim[2])) return bad(PyExc_ValueError, SHAPE);
    if (k.dt != v.dt) return bad(PyExc_TypeError, "k and v must have one dtype");
    const Tensor *others[] = {&v, &c.cache, &c.table, &c.lens, &c.cu};
    if (!one_device_of(&k, others, 5)) return NULL;
    int64_t ks, vs;
    if (!token_stride(a[0], &k, &ks) || !token_stride(a[1], &v, &vs)) return NULL;
    void *h = NULL;
    const int found = find_stream(a[6], k.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    int st;
    Py_BEGIN_ALLOW_THREADS
    if (a[7] == Py_True)
        st = S.kv4_read(c.cache.p, c.table.p, c.lens.p, c.cu.p, k.p, v.p, (int)c.B, c.T, (int)c.Hk, (int)c.D, c.page, c.pages,
                        (int)c.cols, c.table_stride, ks, vs, k.dt, h);
    else
        st = S.kv4_append(k.p, v.p, c.cache.p, c.table.p, c.lens.p, c.cu.p, (int)c.B, c.T, (int)c.Hk, (int)c.D, c.page,
                          c.pages, (int)c.cols, c.table_stride, ks, vs, k.dt, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (q, cache, block_table, lens, out, cu_seqlens, scale or None, causal, window, lse, workspace, stream). With no
 * workspace where one is needed: its size as a negative number below -1. */
static PyObject *kv4_attention(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    if (!arity(n, 12)) return NULL;
    Tensor q, out, lse, ws;
    Cached c;
    if (!look(a[0], &q, 0) || !look(a[4], &out, 0) || !look_at(a[9], &lse, 1) || !look_at(a[10], &ws, 1) ||
        !look_cached(a[1], a[2], a[3], a[5], &q, &c))
        return NULL;
    const int64_t Hq = q.dim[1];
    if (!is_shape(&out, 3, c.T, Hq, c.D) || (a[9] != Py_None && !is_shape(&lse, 2, c.T, Hq, 0)))
        return bad(PyExc_ValueError, SHAPE);
    if (out.dt != q.dt) return bad(PyExc_TypeError, "out must have q's dtype");
    if (a[9] != Py_None && lse.dt != DT_F32) return bad(PyExc_TypeError, "lse must be float32");
    if (a[10] != Py_None && ws.dt != DT_U8) return bad(PyExc_TypeError, "workspace must be uint8");
    const Tensor *others[] = {&out, &lse, &ws, &c.cache, &c.table, &c.lens, &c.cu};
    if (!one_device_of(&q, others, 7)) return NULL;
    int64_t qs, os;
    if (!token_stride(a[0], &q, &qs) || !token_stride(a[4], &out, &os)) return NULL;
    const double scale = a[6] == Py_None ? 1.0 / sqrt((double)c.D) : PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    const int causal = PyObject_IsTrue(a[7]);
    if (causal < 0) return NULL;
    const int64_t window = PyLong_AsLongLong(a[8]);
    if (window == -1 && PyErr_Occurred()) return NULL;
    void *h = NULL;
    const int found = find_stream(a[11], q.dev, &h);
    if (found == 0) return NULL;
    if (found < 0) return PyLong_FromLong(-1);
    size_t size = 1;
    if (a[10] == Py_None) {
        const size_t need = S.kv4_space((int)c.B, c.T, (int)Hq, (int)c.Hk, (int)c.D, c.page, (int)c.cols,
                                        a[5] != Py_None, window, q.dt);
        if (need > 0) {  /* of the current device, which has to be the tensors' */
            long long cur;
            if (!long_of(PyObject_CallNoArgs(S.get_device), &cur)) return NULL;
            return PyLong_FromLongLong(cur == q.dev ? -(long long)need : -1);
        }
        size = 0;
    }
    for (int i = 0; a[10] != Py_None && i < ws.nd; ++i) size *= (size_t)ws.dim[i];
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = S.kv4_attention(q.p, c.cache.p, c.table.p, c.lens.p, c.cu.p, out.p, lse.p, (int)c.B, c.T, (int)Hq, (int)c.Hk,
                         (int)c.D, c.page, c.pages, (int)c.cols, c.table_stride, qs, os, (float)scale, causal, window, q.dt,
                         ws.p, size, h);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* (addresses of kda_add_rmsnorm_fp8, kda_gated_rmsnorm_fp8, kda_fp8_linear, kda_qk_norm_rope, kda_kv4_append,
 * kda_kv4_read, kda_kv4_attention, kda_kv4_attention_workspace_bytes; torch's float32, bfloat16, float8_e4m3fn,
 * float64, int64, int32, uint8; current device index (callable), device index -> stream handle (callable)) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    enum { FNS = 8, OBJECTS = 9 };
    PyObject **slot[OBJECTS] = {&S.f32, &S.bf16, &S.f8, &S.f64, &S.i64, &S.i32, &S.u8, &S.get_device, &S.raw_stream};
    if (PyTuple_GET_SIZE(args) != FNS + OBJECTS) return bad(PyExc_TypeError, "wrong number of arguments");
    void *f[FNS];
    for (int i = 0; i < FNS; ++i)
        if ((f[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, i))) == NULL)
            return PyErr_Occurred() ? NULL : bad(PyExc_ValueError, "a function's address is NULL");
    S.add_rmsnorm = (add_rmsnorm_fn)f[0];
    S.gated_rmsnorm = (gated_rmsnorm_fn)f[1];
    S.linear = (linear_fn)f[2];
    S.norm_rope = (norm_rope_fn)f[3];
    S.kv4_append = (kv4_append_fn)f[4];
    S.kv4_read = (kv4_read_fn)f[5];
    S.kv4_attention = (kv4_attention_fn)f[6];
    S.kv4_space = (kv4_space_fn)f[7];
    for (int i = 0; i < OBJECTS; ++i) {
        PyObject *o = PyTuple_GET_ITEM(args, FNS + i);
        Py_INCREF(o);
        Py_XSETREF(*slot[i], o);
    }
    S.ready = 1;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "Library functions and torch objects that the calls use."},
    {"add_rmsnorm", (PyCFunction)(void (*)(void))add_rmsnorm, METH_FASTCALL, "kda_add_rmsnorm_fp8"},
    {"gated_rmsnorm", (PyCFunction)(void (*)(void))gated_rmsnorm, METH_FASTCALL, "kda_gated_rmsnorm_fp8"},
    {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, "kda_fp8_linear"},
    {"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, "kda_qk_norm_rope"},
    {"kv4_rows", (PyCFunction)(void (*)(void))kv4_rows, METH_FASTCALL, "kda_kv4_append and kda_kv4_read"},
    {"kv4_attention", (PyCFunction)(void (*)(void))kv4_attention, METH_FASTCALL, "kda_kv4_attention"},
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
