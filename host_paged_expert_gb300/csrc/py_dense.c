/*
 * The Python binding of the dense operators: checks torch tensors, allocates
 * results and workspaces through torch, and calls libpe's C ABI.
 *
 * It is native because a decode step makes these calls with one token: the
 * same checks and the marshalling through ctypes took 12 us a call on the
 * Grace host, six times the norm's time on the GPU.  Tensors are read through
 * their Python attributes, so nothing here depends on torch's C++ interface.
 * dense.py documents the functions; arguments arrive by position.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "pe.h"

static struct {
    PyObject *empty, *stream, *device;           /* torch.empty; current stream handle and device */
    PyObject *bf16, *f16, *f32, *e4m3, *u8;      /* torch dtypes (compared by identity) */
    PyObject *acts, *bad, *elsewhere, *rmsnorm;  /* name -> pe_act; raises; reruns elsewhere; result type */
} G;
static PyObject *s_shape, *s_stride, *s_dtype, *s_device, *s_get_device, *s_data_ptr, *kw_empty;

typedef struct {
    PyObject* dt; /* borrowed: torch keeps its dtypes */
    Py_ssize_t nd;
    long long d[2], s[2];
    long dev;
    void* p;
} Ten;

static PyObject* bad(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyObject* msg = PyUnicode_FromFormatV(fmt, ap);
    va_end(ap);
    if (!msg) return NULL;
    PyObject* r = PyObject_CallFunction(G.bad, "iN", status, msg); /* raises */
    Py_XDECREF(r);
    return NULL;
}
static PyObject* failed(pe_status st) { return bad(st, "%s", pe_last_error(NULL)); }

static int pair(PyObject* t, Py_ssize_t* nd, long long* v) {
    if (!t) return -1;
    if (!PyTuple_Check(t)) {
        Py_DECREF(t);
        PyErr_SetString(PyExc_TypeError, "want a torch tensor");
        return -1;
    }
    const Py_ssize_t n = PyTuple_GET_SIZE(t);
    if (nd) *nd = n;
    for (Py_ssize_t i = 0; i < n && i < 2; ++i) v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
    Py_DECREF(t);
    return PyErr_Occurred() ? -1 : 0;
}

static int load(PyObject* o, Ten* t) {
    t->d[0] = t->d[1] = t->s[0] = t->s[1] = 1;
    if (pair(PyObject_GetAttr(o, s_shape), &t->nd, t->d) || pair(PyObject_CallMethodNoArgs(o, s_stride), NULL, t->s)) return -1;
    PyObject* v = PyObject_GetAttr(o, s_dtype);
    if (!v) return -1;
    t->dt = v;
    Py_DECREF(v);
    if (!(v = PyObject_CallMethodNoArgs(o, s_get_device))) return -1;
    t->dev = PyLong_AsLong(v);
    Py_DECREF(v);
    if (!(v = PyObject_CallMethodNoArgs(o, s_data_ptr))) return -1;
    t->p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

static int mismatch(const Ten* t, const char* name, PyObject* dt, long long r, long long c, long dev) {
    if (c < 0)
        bad(PE_ERR_INVALID, "%s: want contiguous %R [%lld] on cuda:%ld, got %R, %zd-d [%lld, %lld], strides (%lld, %lld), on device %ld",
            name, dt, r, dev, t->dt, t->nd, t->d[0], t->d[1], t->s[0], t->s[1], t->dev);
    else
        bad(PE_ERR_INVALID, "%s: want %R [%lld, %lld] on cuda:%ld, got %R, %zd-d [%lld, %lld], strides (%lld, %lld), on device %ld", name,
            dt, r, c, dev, t->dt, t->nd, t->d[0], t->d[1], t->s[0], t->s[1], t->dev);
    return -1;
}

/* x, the first operand: a CUDA matrix. */
static int load_matrix(PyObject* o, Ten* t, const char* name) {
    if (load(o, t)) return -1;
    if (t->nd != 2 || t->dev < 0) {
        bad(PE_ERR_INVALID, "%s: want a CUDA matrix [rows, features], got %zd-d on device %ld", name, t->nd, t->dev);
        return -1;
    }
    return 0;
}
/* Unit column stride; the pitch of a single row is never used (a view of one
 * row may state any), so it becomes the row's length. */
static int pitched(Ten* t, const char* name) {
    if (t->s[1] != 1 && t->d[0] && t->d[1] > 1) {
        bad(PE_ERR_INVALID, "%s: columns must be contiguous", name);
        return -1;
    }
    if (t->d[0] <= 1) t->s[0] = t->d[1];
    return 0;
}
static int load_rows(PyObject* o, Ten* t, const char* name, PyObject* dt, long long r, long long c, long dev) {
    if (load(o, t)) return -1;
    if (t->dt != dt || t->nd != 2 || t->d[0] != r || t->d[1] != c || t->dev != dev) return mismatch(t, name, dt, r, c, dev);
    return pitched(t, name);
}
/* A contiguous [r, c] tensor, or [r] where c < 0. */
static int whole(const Ten* t, const char* name, PyObject* dt, long long r, long long c, long dev) {
    const int two = c >= 0;
    int ok = t->dt == dt && t->nd == 1 + two && t->d[0] == r && (!two || t->d[1] == c) && t->dev == dev;
    if (ok && r && (!two || c)) {
        if (two) ok = (t->s[1] == 1 || c == 1) && (t->s[0] == c || r == 1);
        else ok = t->s[0] == 1 || r == 1;
    }
    return ok ? 0 : mismatch(t, name, dt, r, c, dev);
}
static int load_whole(PyObject* o, Ten* t, const char* name, PyObject* dt, long long r, long long c, long dev) {
    return load(o, t) || whole(t, name, dt, r, c, dev);
}

/* torch.empty(r[, c], dtype=dt, device=device) and its pointer. */
static PyObject* empty(long long r, long long c, PyObject* dt, PyObject* device, void** p) {
    PyObject* a[4];
    Py_ssize_t n = 0;
    a[n++] = PyLong_FromLongLong(r);
    if (c >= 0) a[n++] = PyLong_FromLongLong(c);
    a[n] = dt;
    a[n + 1] = device;
    PyObject* t = PyObject_Vectorcall(G.empty, a, n, kw_empty);
    for (Py_ssize_t i = 0; i < n; ++i) Py_XDECREF(a[i]);
    if (!t) return NULL;
    PyObject* v = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!v) {
        Py_DECREF(t);
        return NULL;
    }
    *p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return t;
}

static int elem_of(PyObject* dt, const char* name) {
    if (dt == G.bf16) return PE_ELEM_BF16;
    if (dt == G.f16) return PE_ELEM_F16;
    bad(PE_ERR_INVALID, "%s: %R is neither bf16 nor fp16", name, dt);
    return -1;
}
static int act_of(PyObject* name) {
    PyObject* v = PyDict_GetItemWithError(G.acts, name);
    if (v) return (int)PyLong_AsLong(v);
    if (!PyErr_Occurred()) bad(PE_ERR_INVALID, "unknown activation %R; one of %S", name, G.acts);
    return -1;
}

/* Whether the call belongs to another stream or device than the current
 * ones (1), which Python then makes current; -1: an exception. */
static int away(PyObject* stream, long dev) {
    if (stream != Py_None) return 1;
    PyObject* v = PyObject_CallNoArgs(G.device);
    if (!v) return -1;
    const long cur = PyLong_AsLong(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : cur != dev;
}
static PyObject* go_there(PyObject* self, const char* name, long dev, PyObject* const* args, Py_ssize_t n) {
    PyObject* fn = PyObject_GetAttrString(self, name);
    if (!fn) return NULL;
    PyObject* rest = PyTuple_New(n - 1); /* without the stream, the last one */
    if (!rest) {
        Py_DECREF(fn);
        return NULL;
    }
    for (Py_ssize_t i = 0; i < n - 1; ++i) PyTuple_SET_ITEM(rest, i, Py_NewRef(args[i]));
    return PyObject_CallFunction(G.elsewhere, "NlON", fn, dev, args[n - 1], rest);
}
static int current(long dev, void** st) {
    PyObject* d = PyLong_FromLong(dev);
    PyObject* v = d ? PyObject_CallOneArg(G.stream, d) : NULL;
    Py_XDECREF(d);
    if (!v) return -1;
    *st = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return PyErr_Occurred() ? -1 : 0;
}

#define WANT(N)                                                                                   \
    do {                                                                                          \
        if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);          \
    } while (0)
#define THERE(NAME, DEV)                                        \
    do {                                                        \
        const int a_ = away(args[n - 1], DEV);                  \
        if (a_ < 0) return NULL;                                \
        if (a_) return go_there(self, NAME, DEV, args, n);      \
    } while (0)
/* Rows and features are 32-bit in the C ABI. */
#define FITS(V)                                                                                          \
    do {                                                                                                 \
        if ((V) > INT32_MAX) return bad(PE_ERR_RANGE, "a dimension of %lld is too large", (long long)(V)); \
    } while (0)
#define CALL(X)                             \
    do {                                    \
        pe_status st_;                      \
        Py_BEGIN_ALLOW_THREADS st_ = (X);   \
        Py_END_ALLOW_THREADS if (st_) {     \
            failed(st_);                    \
            goto out;                       \
        }                                   \
    } while (0)
#define NEW(VAR, PTR, R, C, DT)                                \
    do {                                                       \
        if (!(VAR = empty(R, C, DT, device, &PTR))) goto out;  \
    } while (0)

/* rms_norm(x, weight, residual, eps, y, quant, save, stream) */
static PyObject* f_rms_norm(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(8);
    Ten x, w, r = {0};
    if (load_matrix(args[0], &x, "x")) return NULL;
    THERE("rms_norm", x.dev);
    const long long rows = x.d[0], hidden = x.d[1];
    FITS(rows);
    FITS(hidden);
    const int elem = elem_of(x.dt, "x");
    const double eps = PyFloat_AsDouble(args[3]);
    const int want_y = PyObject_IsTrue(args[4]), quant = PyObject_IsTrue(args[5]), save = PyObject_IsTrue(args[6]);
    if (elem < 0 || want_y < 0 || quant < 0 || save < 0 || PyErr_Occurred() || pitched(&x, "x") ||
        load_whole(args[1], &w, "weight", x.dt, hidden, -1, x.dev))
        return NULL;
    const int add = args[2] != Py_None;
    if (add && load_rows(args[2], &r, "residual", x.dt, rows, hidden, x.dev)) return NULL;
    PyObject *device = PyObject_GetAttr(args[0], s_device), *res = NULL;
    PyObject *y = NULL, *sum = NULL, *codes = NULL, *scale = NULL, *rstd = NULL;
    void *yp = NULL, *tp = NULL, *cp = NULL, *sp = NULL, *dp = NULL, *st;
    if (!device) return NULL;
    if (want_y) NEW(y, yp, rows, hidden, x.dt);
    if (add) NEW(sum, tp, rows, hidden, x.dt);
    else sum = Py_NewRef(args[0]);
    if (quant) {
        NEW(codes, cp, rows, hidden, G.e4m3);
        NEW(scale, sp, rows, (hidden + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP, G.f32);
    }
    if (save) NEW(rstd, dp, rows, -1, G.f32);
    if (current(x.dev, &st)) goto out;
    CALL(pe_rms_norm(x.p, x.s[0], r.p, r.s[0], w.p, (float)eps, yp, tp, cp, sp, dp, (int32_t)rows, (int32_t)hidden, elem, st));
    PyObject* a[5] = {y ? y : Py_None, sum, codes ? codes : Py_None, scale ? scale : Py_None, rstd ? rstd : Py_None};
    res = PyObject_Vectorcall(G.rmsnorm, a, 5, NULL);
out:
    Py_DECREF(device);
    Py_XDECREF(y);
    Py_XDECREF(sum);
    Py_XDECREF(codes);
    Py_XDECREF(scale);
    Py_XDECREF(rstd);
    return res;
}

/* rms_norm_backward(dy, sum, weight, rstd, dsum, stream) */
static PyObject* f_rms_norm_backward(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(6);
    Ten dy, s, w, rs, ds = {0};
    if (load_matrix(args[1], &s, "sum")) return NULL;
    THERE("rms_norm_backward", s.dev);
    const long long rows = s.d[0], hidden = s.d[1];
    FITS(rows);
    FITS(hidden);
    const int elem = elem_of(s.dt, "sum");
    if (elem < 0 || pitched(&s, "sum") || load_rows(args[0], &dy, "dy", s.dt, rows, hidden, s.dev) ||
        load_whole(args[2], &w, "weight", s.dt, hidden, -1, s.dev) || load_whole(args[3], &rs, "rstd", G.f32, rows, -1, s.dev) ||
        (args[4] != Py_None && load_rows(args[4], &ds, "dsum", s.dt, rows, hidden, s.dev)))
        return NULL;
    PyObject *device = PyObject_GetAttr(args[1], s_device), *res = NULL, *dx = NULL, *dw = NULL, *ws = NULL;
    void *xp, *wp, *kp, *st;
    if (!device) return NULL;
    const size_t bytes = pe_rms_norm_backward_workspace((int32_t)rows, (int32_t)hidden);
    NEW(dx, xp, rows, hidden, s.dt);
    NEW(dw, wp, hidden, -1, s.dt);
    NEW(ws, kp, (long long)bytes, -1, G.u8);
    if (current(s.dev, &st)) goto out;
    CALL(pe_rms_norm_backward(dy.p, dy.s[0], ds.p, ds.s[0], s.p, s.s[0], w.p, rs.p, xp, wp, kp, bytes, (int32_t)rows, (int32_t)hidden,
                              elem, st));
    res = PyTuple_Pack(2, dx, dw);
out:
    Py_DECREF(device);
    Py_XDECREF(dx);
    Py_XDECREF(dw);
    Py_XDECREF(ws);
    return res;
}

/* linear(x, weight, bias, act, residual, x_scale, w_scale, out_dtype, save, stream) */
static PyObject* f_linear(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(10);
    Ten x, w, b = {0}, r = {0}, xs = {0}, wsc = {0};
    if (load_matrix(args[0], &x, "x")) return NULL;
    THERE("linear", x.dev);
    const int act = act_of(args[3]), save = PyObject_IsTrue(args[8]);
    if (act < 0 || save < 0 || load(args[1], &w)) return NULL;
    const long long rows = x.d[0], k = x.d[1], outs = w.d[0];
    FITS(rows);
    FITS(k);
    FITS(outs);
    if (pitched(&x, "x") || whole(&w, "weight", x.dt, outs, k, x.dev)) return NULL;
    PyObject *dt = x.dt, *odt = args[7];
    if (dt == G.e4m3) {
        if (args[5] == Py_None || args[6] == Py_None) return bad(PE_ERR_INVALID, "E4M3 x and weight need x_scale and w_scale");
        const long long kg = (k + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP, ng = (outs + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP;
        if (load_whole(args[5], &xs, "x_scale", G.f32, rows, kg, x.dev) || load_whole(args[6], &wsc, "w_scale", G.f32, ng, kg, x.dev))
            return NULL;
        /* the 16-bit type: the residual's, the bias's, the result's, else bf16 */
        if (args[4] != Py_None || args[2] != Py_None) {
            Ten t;
            if (load(args[4] != Py_None ? args[4] : args[2], &t)) return NULL;
            dt = t.dt;
        } else {
            dt = odt != Py_None && odt != G.f32 ? odt : G.bf16;
        }
    } else if (args[5] != Py_None || args[6] != Py_None) {
        return bad(PE_ERR_INVALID, "scales go with E4M3 x and weight");
    }
    const int elem = elem_of(dt, "x");
    if (elem < 0) return NULL;
    int oelem = elem;
    if (odt == Py_None) odt = dt;
    else if (odt == G.f32) oelem = PE_ELEM_F32;
    else if (odt != dt) return bad(PE_ERR_INVALID, "out_dtype: want %R or torch.float32, got %R", dt, odt);
    if ((args[2] != Py_None && load_whole(args[2], &b, "bias", dt, outs, -1, x.dev)) ||
        (args[4] != Py_None && load_rows(args[4], &r, "residual", dt, rows, outs, x.dev)))
        return NULL;
    PyObject *device = PyObject_GetAttr(args[0], s_device), *res = NULL, *y = NULL, *z = NULL;
    void *yp, *zp = NULL, *st;
    if (!device) return NULL;
    NEW(y, yp, rows, outs, odt);
    if (save && act) NEW(z, zp, rows, outs, dt);
    if (current(x.dev, &st)) goto out;
    CALL(pe_linear(x.p, x.s[0], xs.p, w.p, wsc.p, b.p, r.p, r.s[0], yp, oelem, zp, act, (int32_t)rows, (int32_t)k, (int32_t)outs, elem,
                   st));
    res = save ? PyTuple_Pack(2, y, z ? z : Py_None) : Py_NewRef(y);
out:
    Py_DECREF(device);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return res;
}

/* linear_backward(dy, x, weight, z, act, bias, stream) */
static PyObject* f_linear_backward(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(7);
    Ten dy, x, w, z = {0};
    if (load_matrix(args[1], &x, "x")) return NULL;
    THERE("linear_backward", x.dev);
    const int act = act_of(args[4]), bias = PyObject_IsTrue(args[5]);
    if (act < 0 || bias < 0 || load(args[2], &w)) return NULL;
    const long long rows = x.d[0], k = x.d[1], outs = w.d[0];
    FITS(rows);
    FITS(k);
    FITS(outs);
    const int elem = elem_of(x.dt, "x");
    if (elem < 0 || pitched(&x, "x") || load_rows(args[0], &dy, "dy", x.dt, rows, outs, x.dev) ||
        whole(&w, "weight", x.dt, outs, k, x.dev))
        return NULL;
    if (act) {
        if (args[3] == Py_None) return bad(PE_ERR_INVALID, "act %R needs the z that linear(save=True) returned", args[4]);
        if (load_whole(args[3], &z, "z", x.dt, rows, outs, x.dev)) return NULL;
    }
    PyObject *device = PyObject_GetAttr(args[1], s_device), *res = NULL, *dx = NULL, *dw = NULL, *db = NULL, *ws = NULL;
    void *xp, *wp, *bp = NULL, *kp, *st;
    if (!device) return NULL;
    const size_t bytes = pe_linear_backward_workspace((int32_t)rows, (int32_t)outs, act);
    NEW(dx, xp, rows, k, x.dt);
    NEW(dw, wp, outs, k, x.dt);
    if (bias) NEW(db, bp, outs, -1, x.dt);
    NEW(ws, kp, (long long)bytes, -1, G.u8);
    if (current(x.dev, &st)) goto out;
    CALL(pe_linear_backward(dy.p, dy.s[0], x.p, x.s[0], w.p, z.p, act, xp, wp, bp, kp, bytes, (int32_t)rows, (int32_t)k, (int32_t)outs,
                            elem, st));
    res = PyTuple_Pack(3, dx, dw, db ? db : Py_None);
out:
    Py_DECREF(device);
    Py_XDECREF(dx);
    Py_XDECREF(dw);
    Py_XDECREF(db);
    Py_XDECREF(ws);
    return res;
}

/* gated_ffn(x, w13, w2, act, residual, save, stream) */
static PyObject* f_gated_ffn(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(7);
    Ten x, w13, w2, r = {0};
    if (load_matrix(args[0], &x, "x")) return NULL;
    THERE("gated_ffn", x.dev);
    const int act = act_of(args[3]), save = PyObject_IsTrue(args[5]), elem = act < 0 ? -1 : elem_of(x.dt, "x");
    if (elem < 0 || save < 0 || load(args[2], &w2)) return NULL;
    const long long rows = x.d[0], h = x.d[1], i = w2.nd ? w2.d[w2.nd > 1] : 0;
    FITS(rows);
    FITS(h);
    FITS(2 * i);
    if (pitched(&x, "x") || load_whole(args[1], &w13, "w13", x.dt, 2 * i, h, x.dev) ||
        whole(&w2, "w2", x.dt, h, i, x.dev) ||
        (args[4] != Py_None && load_rows(args[4], &r, "residual", x.dt, rows, h, x.dev)))
        return NULL;
    PyObject *device = PyObject_GetAttr(args[0], s_device), *res = NULL, *y = NULL, *gu = NULL, *ws = NULL;
    void *yp, *gp = NULL, *kp, *st;
    if (!device) return NULL;
    const size_t bytes = pe_gated_ffn_workspace((int32_t)rows, (int32_t)i);
    NEW(y, yp, rows, h, x.dt);
    if (save) NEW(gu, gp, rows, 2 * i, x.dt);
    NEW(ws, kp, (long long)bytes, -1, G.u8);
    if (current(x.dev, &st)) goto out;
    CALL(pe_gated_ffn(x.p, x.s[0], w13.p, w2.p, r.p, r.s[0], yp, gp, act, kp, bytes, (int32_t)rows, (int32_t)h, (int32_t)i, elem, st));
    res = save ? PyTuple_Pack(2, y, gu) : Py_NewRef(y);
out:
    Py_DECREF(device);
    Py_XDECREF(y);
    Py_XDECREF(gu);
    Py_XDECREF(ws);
    return res;
}

/* gated_ffn_backward(dy, x, w13, w2, gu, act, stream) */
static PyObject* f_gated_ffn_backward(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(7);
    Ten dy, x, w13, w2, gu;
    if (load_matrix(args[1], &x, "x")) return NULL;
    THERE("gated_ffn_backward", x.dev);
    const int act = act_of(args[5]), elem = act < 0 ? -1 : elem_of(x.dt, "x");
    if (elem < 0 || load(args[3], &w2)) return NULL;
    const long long rows = x.d[0], h = x.d[1], i = w2.nd ? w2.d[w2.nd > 1] : 0;
    FITS(rows);
    FITS(h);
    FITS(2 * i);
    if (pitched(&x, "x") || load_rows(args[0], &dy, "dy", x.dt, rows, h, x.dev) ||
        load_whole(args[2], &w13, "w13", x.dt, 2 * i, h, x.dev) || whole(&w2, "w2", x.dt, h, i, x.dev) ||
        load_whole(args[4], &gu, "gu", x.dt, rows, 2 * i, x.dev))
        return NULL;
    PyObject *device = PyObject_GetAttr(args[1], s_device), *res = NULL, *dx = NULL, *d13 = NULL, *d2 = NULL, *ws = NULL;
    void *xp, *p13, *p2, *kp, *st;
    if (!device) return NULL;
    const size_t bytes = pe_gated_ffn_backward_workspace((int32_t)rows, (int32_t)i);
    NEW(dx, xp, rows, h, x.dt);
    NEW(d13, p13, 2 * i, h, x.dt);
    NEW(d2, p2, h, i, x.dt);
    NEW(ws, kp, (long long)bytes, -1, G.u8);
    if (current(x.dev, &st)) goto out;
    CALL(pe_gated_ffn_backward(dy.p, dy.s[0], x.p, x.s[0], w13.p, w2.p, gu.p, act, xp, p13, p2, kp, bytes, (int32_t)rows, (int32_t)h,
                               (int32_t)i, elem, st));
    res = PyTuple_Pack(3, dx, d13, d2);
out:
    Py_DECREF(device);
    Py_XDECREF(dx);
    Py_XDECREF(d13);
    Py_XDECREF(d2);
    Py_XDECREF(ws);
    return res;
}

/* setup(empty, stream, device, bf16, f16, f32, e4m3, u8, acts, bad, elsewhere, rmsnorm) */
static PyObject* f_setup(PyObject* self, PyObject* const* args, Py_ssize_t n) {
    WANT(12);
    PyObject** to[12] = {&G.empty, &G.stream, &G.device, &G.bf16, &G.f16,       &G.f32,
                         &G.e4m3,  &G.u8,     &G.acts,   &G.bad,  &G.elsewhere, &G.rmsnorm};
    for (int i = 0; i < 12; ++i) Py_XSETREF(*to[i], Py_NewRef(args[i]));
    Py_RETURN_NONE;
}

#define M(NAME) {#NAME, (PyCFunction)(void (*)(void))f_##NAME, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {M(setup),           M(rms_norm),  M(rms_norm_backward),  M(linear),
                                M(linear_backward), M(gated_ffn), M(gated_ffn_backward), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__dense(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_device = PyUnicode_InternFromString("device");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    kw_empty = s_dtype && s_device ? PyTuple_Pack(2, s_dtype, s_device) : NULL;
    if (!kw_empty || !s_shape || !s_stride || !s_get_device || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
