// The Python binding of the dense operators: checks torch tensors, allocates
// results and workspaces, and calls libpe's C ABI.
//
// It is native because a decode step makes these calls with one token.  On
// the Grace host a linear call took 11.9 us of marshalling through ctypes and
// 8.8 us with tensors read and allocated through their Python attributes; its
// kernel takes 3.  So tensors are read and made in C++.  dense.py documents
// the functions; arguments arrive by position, the stream last.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdio.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pe.h"

namespace {

// name -> pe_act, format; raises; reruns elsewhere; result types
PyObject *g_acts, *g_formats, *g_raise, *g_elsewhere, *g_rmsnorm, *g_routing;

using Type = at::ScalarType;
constexpr Type kBF16 = at::kBFloat16, kF16 = at::kHalf, kF32 = at::kFloat, kE4M3 = at::kFloat8_e4m3fn, kU8 = at::kByte,
               kI32 = at::kInt, kE8M0 = at::kFloat8_e8m0fnu;

struct Raised {};  // a Python exception is set

[[noreturn]] void bad(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    PyObject* msg = PyUnicode_FromFormatV(fmt, ap);
    va_end(ap);
    if (msg) Py_XDECREF(PyObject_CallFunction(g_raise, "iN", status, msg));
    throw Raised();
}

// A tensor as the calls see it: at most two dimensions, three for the weights of groups.
struct Ten {
    Type dt{};
    int64_t nd = 0, d0 = 1, d1 = 1, s0 = 1, s1 = 1, d2 = 1;
    bool packed = false;  // contiguous
    int dev = -1;
    void* p = nullptr;
    bool there = false;
};

Ten load(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s: want a tensor, got %s", name, Py_TYPE(o)->tp_name);
        throw Raised();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided) bad(PE_ERR_INVALID, "%s: want a dense tensor", name);
    // a result without a graph would drop the tensor's gradient without a word
    if (t.requires_grad() && c10::GradMode::is_enabled())
        bad(PE_ERR_INVALID, "%s requires grad, and these calls record none: detach it, or call under torch.no_grad() or inside a "
                            "torch.autograd.Function", name);
    Ten r;
    r.there = true;
    r.dt = t.scalar_type();
    r.nd = t.dim();
    const auto d = t.sizes(), s = t.strides();
    if (r.nd > 0) r.d0 = d[0], r.s0 = s[0];
    if (r.nd > 1) r.d1 = d[1], r.s1 = s[1];
    if (r.nd > 2) r.d2 = d[2], r.packed = t.is_contiguous();
    r.dev = t.is_cuda() ? t.get_device() : -1;
    r.p = t.numel() ? t.data_ptr() : nullptr;
    return r;
}

[[noreturn]] void mismatch(const Ten& t, const char* name, const char* how, Type dt, int64_t r, int64_t c) {
    char want[64];
    if (c < 0) snprintf(want, sizeof want, "[%lld]", (long long)r);
    else snprintf(want, sizeof want, "[%lld, %lld]", (long long)r, (long long)c);
    bad(PE_ERR_INVALID, "%s: want %s%s %s, got %s, %d-d [%lld, %lld], strides (%lld, %lld)", name, how, c10::toString(dt), want,
        c10::toString(t.dt), (int)t.nd, (long long)t.d0, (long long)t.d1, (long long)t.s0, (long long)t.s1);
}

// Unit column stride; the pitch of a single row is never used (a view of one
// row may state any), so it becomes the row's length.
void pitched(Ten& t, const char* name) {
    if (t.s1 != 1 && t.d0 && t.d1 > 1) bad(PE_ERR_INVALID, "%s: columns must be contiguous", name);
    if (t.d0 <= 1) t.s0 = t.d1;
}

// Features are 32-bit in the C ABI.
void fits(int64_t v) {
    if (v > INT32_MAX) bad(PE_ERR_RANGE, "a dimension of %lld is too large", (long long)v);
}

// x, the first operand.
Ten matrix(PyObject* o, const char* name) {
    Ten t = load(o, name);
    if (t.nd != 2) bad(PE_ERR_INVALID, "%s: want a matrix [rows, features], got %d-d", name, (int)t.nd);
    if (t.d0 > PE_MAX_ROWS) bad(PE_ERR_RANGE, "%s: a number of rows of %lld is too large, at most %d", name, (long long)t.d0, PE_MAX_ROWS);
    fits(t.d1);
    pitched(t, name);
    return t;
}
Ten rows_of(PyObject* o, const char* name, Type dt, int64_t r, int64_t c) {
    Ten t = load(o, name);
    if (t.dt != dt || t.nd != 2 || t.d0 != r || t.d1 != c) mismatch(t, name, "", dt, r, c);
    pitched(t, name);
    return t;
}
// A contiguous [r, c] tensor, or [r] where c < 0.
void whole(const Ten& t, const char* name, Type dt, int64_t r, int64_t c = -1) {
    const bool two = c >= 0;
    bool ok = t.dt == dt && t.nd == 1 + two && t.d0 == r && (!two || t.d1 == c);
    if (ok && r && (!two || c)) ok = two ? (t.s1 == 1 || c == 1) && (t.s0 == c || r == 1) : t.s0 == 1 || r == 1;
    if (!ok) mismatch(t, name, "contiguous ", dt, r, c);
}
Ten whole_of(PyObject* o, const char* name, Type dt, int64_t r, int64_t c = -1) {
    const Ten t = load(o, name);
    whole(t, name, dt, r, c);
    return t;
}

// The weights of groups: contiguous [g, r, c].
void packed(const Ten& t, const char* name, Type dt, int64_t g, int64_t r, int64_t c) {
    if (t.dt == dt && t.nd == 3 && t.d0 == g && t.d1 == r && t.d2 == c && t.packed) return;
    bad(PE_ERR_INVALID, "%s: want contiguous %s [%lld, %lld, %lld], got %s, %d-d [%lld, %lld, %lld]%s", name, c10::toString(dt), (long long)g,
        (long long)r, (long long)c, c10::toString(t.dt), (int)t.nd, (long long)t.d0, (long long)t.d1, (long long)t.d2,
        t.nd == 3 && !t.packed ? ", not contiguous" : "");
}
// The offsets of groups, [g + 1].
Ten offsets_of(PyObject* o, int64_t groups) {
    if (groups < 1) bad(PE_ERR_INVALID, "no groups of weights");
    fits(groups);
    return whole_of(o, "offsets", kI32, groups + 1);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
}

int elem_of(Type dt, const char* name) {
    if (dt == kBF16) return PE_ELEM_BF16;
    if (dt == kF16) return PE_ELEM_F16;
    bad(PE_ERR_INVALID, "%s: %s is neither bf16 nor fp16", name, c10::toString(dt));
}
int act_of(PyObject* name) {
    PyObject* v = PyDict_GetItemWithError(g_acts, name);
    if (v) return (int)PyLong_AsLong(v);
    if (PyErr_Occurred()) throw Raised();
    bad(PE_ERR_INVALID, "unknown activation %R; one of %S", name, g_acts);
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised();
    return v;
}

// Every tensor on x's CUDA device (checked last, so that a wrong shape or
// type is what a call hears of first).
void together(const Ten& x, std::initializer_list<const Ten*> others) {
    if (x.dev < 0) bad(PE_ERR_INVALID, "want CUDA tensors");
    for (const Ten* t : others)
        if (t->there && t->dev != x.dev) bad(PE_ERR_INVALID, "tensors on device %d and device %d", x.dev, t->dev);
}

// Whether the call belongs to another stream or device than the current ones,
// which Python then makes current before it calls again.
bool away(PyObject* stream, int dev) { return stream != Py_None || c10::cuda::current_device() != dev; }
PyObject* go_there(PyObject* self, const char* name, int dev, PyObject* const* args, Py_ssize_t n) {
    PyObject* fn = PyObject_GetAttrString(self, name);
    PyObject* rest = fn ? PyTuple_New(n - 1) : nullptr;  // without the stream
    if (!rest) {
        Py_XDECREF(fn);
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n - 1; ++i) PyTuple_SET_ITEM(rest, i, Py_NewRef(args[i]));
    return PyObject_CallFunction(g_elsewhere, "NiON", fn, dev, args[n - 1], rest);
}
void* current(int dev) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

// torch.empty on device dev, without the dispatcher.
at::Tensor empty(int dev, Type dt, int64_t r, int64_t c = -1, int64_t c2 = -1) {
    const int64_t d[3] = {r, c, c2};
    return at::Tensor(at::detail::empty_cuda(at::IntArrayRef(d, c < 0 ? 1 : c2 < 0 ? 2 : 3), dt, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev),
                                             std::nullopt));
}
void* ptr(const at::Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; }
PyObject* wrap(const at::Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }

// The interpreter lock is let go for the C call, and held again before anything
// that it throws goes on.
struct NoGil {
    PyThreadState* const saved = PyEval_SaveThread();
    ~NoGil() { PyEval_RestoreThread(saved); }
};
template <typename F>
void call(F&& f) {
    pe_status st;
    {
        NoGil go;
        st = f();
    }
    if (st) bad(st, "%s", pe_last_error(nullptr));
}

PyObject* tuple(std::initializer_list<const at::Tensor*> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const at::Tensor* t : ts) PyTuple_SET_ITEM(r, i++, wrap(*t));
    return r;
}

using Args = PyObject* const*;

// rms_norm(x, weight, residual, eps, y, quant, save, stream)
PyObject* rms_norm(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x");
    const int64_t rows = x.d0, hidden = x.d1;
    const int elem = elem_of(x.dt, "x");
    const Ten w = whole_of(args[1], "weight", x.dt, hidden);
    const Ten r = args[2] == Py_None ? Ten() : rows_of(args[2], "residual", x.dt, rows, hidden);
    const double eps = PyFloat_AsDouble(args[3]);
    if (PyErr_Occurred()) throw Raised();
    const bool want_y = truth(args[4]), quant = truth(args[5]), save = truth(args[6]);
    together(x, {&w, &r});
    if (away(args[7], x.dev)) return go_there(self, "rms_norm", x.dev, args, n);
    at::Tensor y, sum, codes, scale, rstd;
    if (want_y) y = empty(x.dev, x.dt, rows, hidden);
    if (r.there) sum = empty(x.dev, x.dt, rows, hidden);
    if (quant) {
        codes = empty(x.dev, kE4M3, rows, hidden);
        scale = empty(x.dev, kF32, rows, (hidden + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP);
    }
    if (save) rstd = empty(x.dev, kF32, rows);
    call([&] {
        return pe_rms_norm(x.p, x.s0, r.p, r.s0, w.p, (float)eps, ptr(y), ptr(sum), ptr(codes), (float*)ptr(scale), (float*)ptr(rstd),
                           (int32_t)rows, (int32_t)hidden, elem, current(x.dev));
    });
    PyObject* a[5] = {wrap(y), r.there ? wrap(sum) : Py_NewRef(args[0]), wrap(codes), wrap(scale), wrap(rstd)};
    PyObject* res = PyObject_Vectorcall(g_rmsnorm, a, 5, nullptr);
    for (PyObject* o : a) Py_XDECREF(o);
    return res;
}

// rms_norm_backward(dy, sum, weight, rstd, dsum, stream)
PyObject* rms_norm_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten s = matrix(args[1], "sum");
    const int64_t rows = s.d0, hidden = s.d1;
    const int elem = elem_of(s.dt, "sum");
    const Ten dy = rows_of(args[0], "dy", s.dt, rows, hidden);
    const Ten w = whole_of(args[2], "weight", s.dt, hidden), rstd = whole_of(args[3], "rstd", kF32, rows);
    const Ten ds = args[4] == Py_None ? Ten() : rows_of(args[4], "dsum", s.dt, rows, hidden);
    together(s, {&dy, &w, &rstd, &ds});
    if (away(args[5], s.dev)) return go_there(self, "rms_norm_backward", s.dev, args, n);
    const size_t bytes = pe_rms_norm_backward_workspace((int32_t)rows, (int32_t)hidden);
    const at::Tensor dx = empty(s.dev, s.dt, rows, hidden), dw = empty(s.dev, s.dt, hidden), ws = empty(s.dev, kU8, (int64_t)bytes);
    call([&] {
        return pe_rms_norm_backward(dy.p, dy.s0, ds.p, ds.s0, s.p, s.s0, w.p, (const float*)rstd.p, ptr(dx), ptr(dw), ptr(ws), bytes,
                                    (int32_t)rows, (int32_t)hidden, elem, current(s.dev));
    });
    return tuple({&dx, &dw});
}

// linear(x, weight, bias, act, residual, x_scale, w_scale, out_dtype, save, stream)
PyObject* linear(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), w = load(args[1], "weight");
    const int act = act_of(args[3]);
    const bool save = truth(args[8]);
    const int64_t rows = x.d0, k = x.d1, outs = w.d0;
    fits(outs);
    whole(w, "weight", x.dt, outs, k);
    const bool odt_given = args[7] != Py_None;
    if (odt_given && !THPDtype_Check(args[7])) {
        PyErr_SetString(PyExc_TypeError, "out_dtype: want a torch dtype");
        throw Raised();
    }
    Type dt = x.dt, odt = odt_given ? reinterpret_cast<THPDtype*>(args[7])->scalar_type : kF32;
    Ten xs, ws;
    if (dt == kE4M3) {
        if (args[5] == Py_None || args[6] == Py_None) bad(PE_ERR_INVALID, "E4M3 x and weight need x_scale and w_scale");
        const int64_t kg = (k + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP;
        xs = whole_of(args[5], "x_scale", kF32, rows, kg);
        ws = whole_of(args[6], "w_scale", kF32, (outs + PE_SCALE_GROUP - 1) / PE_SCALE_GROUP, kg);
        // the 16-bit type: the residual's, the bias's, the result's, else bf16
        dt = args[4] != Py_None ? load(args[4], "residual").dt
             : args[2] != Py_None ? load(args[2], "bias").dt
             : odt_given && odt != kF32 ? odt
                                        : kBF16;
    } else if (args[5] != Py_None || args[6] != Py_None) {
        bad(PE_ERR_INVALID, "scales go with E4M3 x and weight");
    }
    const int elem = elem_of(dt, "x");
    if (!odt_given) odt = dt;
    if (odt != dt && odt != kF32)
        bad(PE_ERR_INVALID, "out_dtype: want %s or torch.float32, got %s", c10::toString(dt), c10::toString(odt));
    const Ten b = args[2] == Py_None ? Ten() : whole_of(args[2], "bias", dt, outs);
    const Ten r = args[4] == Py_None ? Ten() : rows_of(args[4], "residual", dt, rows, outs);
    together(x, {&w, &xs, &ws, &b, &r});
    if (away(args[9], x.dev)) return go_there(self, "linear", x.dev, args, n);
    const at::Tensor y = empty(x.dev, odt, rows, outs);
    at::Tensor z;
    if (save && act) z = empty(x.dev, dt, rows, outs);
    call([&] {
        return pe_linear(x.p, x.s0, (const float*)xs.p, w.p, (const float*)ws.p, b.p, r.p, r.s0, ptr(y), odt == dt ? elem : PE_ELEM_F32,
                         ptr(z), act, (int32_t)rows, (int32_t)k, (int32_t)outs, elem, current(x.dev));
    });
    return save ? tuple({&y, &z}) : wrap(y);
}

// linear_backward(dy, x, weight, z, act, bias, stream)
PyObject* linear_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[1], "x"), w = load(args[2], "weight");
    const int act = act_of(args[4]);
    const bool bias = truth(args[5]);
    const int64_t rows = x.d0, k = x.d1, outs = w.d0;
    fits(outs);
    const int elem = elem_of(x.dt, "x");
    whole(w, "weight", x.dt, outs, k);
    const Ten dy = rows_of(args[0], "dy", x.dt, rows, outs);
    if (act && args[3] == Py_None) bad(PE_ERR_INVALID, "act %R needs the z that linear(save=True) returned", args[4]);
    const Ten z = act ? whole_of(args[3], "z", x.dt, rows, outs) : Ten();
    together(x, {&w, &dy, &z});
    if (away(args[6], x.dev)) return go_there(self, "linear_backward", x.dev, args, n);
    const size_t bytes = pe_linear_backward_workspace((int32_t)rows, (int32_t)outs, act);
    const at::Tensor dx = empty(x.dev, x.dt, rows, k), dw = empty(x.dev, x.dt, outs, k), ws = empty(x.dev, kU8, (int64_t)bytes);
    at::Tensor db;
    if (bias) db = empty(x.dev, x.dt, outs);
    call([&] {
        return pe_linear_backward(dy.p, dy.s0, x.p, x.s0, w.p, z.p, act, ptr(dx), ptr(dw), ptr(db), ptr(ws), bytes, (int32_t)rows,
                                  (int32_t)k, (int32_t)outs, elem, current(x.dev));
    });
    return tuple({&dx, &dw, &db});
}

// gated_ffn(x, w13, w2, act, residual, save, stream)
PyObject* gated_ffn(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), w2 = load(args[2], "w2");
    const int act = act_of(args[3]), elem = elem_of(x.dt, "x");
    const bool save = truth(args[5]);
    const int64_t rows = x.d0, h = x.d1, i = w2.nd == 2 ? w2.d1 : w2.d0;
    fits(2 * i);
    const Ten w13 = whole_of(args[1], "w13", x.dt, 2 * i, h);
    whole(w2, "w2", x.dt, h, i);
    const Ten r = args[4] == Py_None ? Ten() : rows_of(args[4], "residual", x.dt, rows, h);
    together(x, {&w13, &w2, &r});
    if (away(args[6], x.dev)) return go_there(self, "gated_ffn", x.dev, args, n);
    const size_t bytes = pe_gated_ffn_workspace((int32_t)rows, (int32_t)i);
    const at::Tensor y = empty(x.dev, x.dt, rows, h), ws = empty(x.dev, kU8, (int64_t)bytes);
    at::Tensor gu;
    if (save) gu = empty(x.dev, x.dt, rows, 2 * i);
    call([&] {
        return pe_gated_ffn(x.p, x.s0, w13.p, w2.p, r.p, r.s0, ptr(y), ptr(gu), act, ptr(ws), bytes, (int32_t)rows, (int32_t)h, (int32_t)i,
                            elem, current(x.dev));
    });
    return save ? tuple({&y, &gu}) : wrap(y);
}

// gated_ffn_backward(dy, x, w13, w2, gu, act, stream)
PyObject* gated_ffn_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[1], "x"), w2 = load(args[3], "w2");
    const int act = act_of(args[5]), elem = elem_of(x.dt, "x");
    const int64_t rows = x.d0, h = x.d1, i = w2.nd == 2 ? w2.d1 : w2.d0;
    fits(2 * i);
    const Ten dy = rows_of(args[0], "dy", x.dt, rows, h), w13 = whole_of(args[2], "w13", x.dt, 2 * i, h);
    whole(w2, "w2", x.dt, h, i);
    const Ten gu = whole_of(args[4], "gu", x.dt, rows, 2 * i);
    together(x, {&dy, &w13, &w2, &gu});
    if (away(args[6], x.dev)) return go_there(self, "gated_ffn_backward", x.dev, args, n);
    const size_t bytes = pe_gated_ffn_backward_workspace((int32_t)rows, (int32_t)i);
    const at::Tensor dx = empty(x.dev, x.dt, rows, h), d13 = empty(x.dev, x.dt, 2 * i, h), d2 = empty(x.dev, x.dt, h, i),
                     ws = empty(x.dev, kU8, (int64_t)bytes);
    call([&] {
        return pe_gated_ffn_backward(dy.p, dy.s0, x.p, x.s0, w13.p, w2.p, gu.p, act, ptr(dx), ptr(d13), ptr(d2), ptr(ws), bytes,
                                     (int32_t)rows, (int32_t)h, (int32_t)i, elem, current(x.dev));
    });
    return tuple({&dx, &d13, &d2});
}

// linear_w4(x, codes, scales, format, bias, act, residual, tensor_scale, out_dtype, stream)
PyObject* linear_w4(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), q = load(args[1], "codes"), sc = load(args[2], "scales");
    PyObject* f = PyDict_GetItemWithError(g_formats, args[3]);
    if (!f) {
        if (PyErr_Occurred()) throw Raised();
        bad(PE_ERR_INVALID, "unknown format %R; one of %S", args[3], g_formats);
    }
    const int fmt = (int)PyLong_AsLong(f), act = act_of(args[5]), elem = elem_of(x.dt, "x");
    const int64_t rows = x.d0, k = x.d1, outs = q.d0;
    fits(outs);
    if (k < 32 || k % 32) bad(PE_ERR_INVALID, "x: features must be a positive multiple of 32, got %lld", (long long)k);
    whole(q, "codes", kU8, outs, k / 2);
    // 8-bit scales may come as bytes
    const Type st = fmt == PE_INT4_GPTQ ? kF16 : fmt == PE_MXFP4 ? kE8M0 : kE4M3;
    const int64_t group = fmt == PE_INT4_GPTQ ? 128 : fmt == PE_MXFP4 ? 32 : 16;
    whole(sc, "scales", fmt != PE_INT4_GPTQ && sc.dt == kU8 ? kU8 : st, outs, (k + group - 1) / group);
    if ((fmt == PE_NVFP4) != (args[7] != Py_None)) bad(PE_ERR_INVALID, "tensor_scale goes with nvfp4, and nvfp4 with tensor_scale");
    const Ten ts = args[7] == Py_None ? Ten() : whole_of(args[7], "tensor_scale", kF32, 1);
    const Ten b = args[4] == Py_None ? Ten() : whole_of(args[4], "bias", x.dt, outs);
    const Ten r = args[6] == Py_None ? Ten() : rows_of(args[6], "residual", x.dt, rows, outs);
    Type odt = x.dt;
    if (args[8] != Py_None) {
        if (!THPDtype_Check(args[8])) {
            PyErr_SetString(PyExc_TypeError, "out_dtype: want a torch dtype");
            throw Raised();
        }
        odt = reinterpret_cast<THPDtype*>(args[8])->scalar_type;
        if (odt != x.dt && odt != kF32) bad(PE_ERR_INVALID, "out_dtype: want %s or torch.float32, got %s", c10::toString(x.dt), c10::toString(odt));
    }
    together(x, {&q, &sc, &ts, &b, &r});
    if (away(args[9], x.dev)) return go_there(self, "linear_w4", x.dev, args, n);
    const size_t bytes = pe_linear_four_bit_workspace((int32_t)rows, (int32_t)k, (int32_t)outs);
    const at::Tensor y = empty(x.dev, odt, rows, outs);
    at::Tensor ws;
    if (bytes) ws = empty(x.dev, kU8, (int64_t)bytes);
    call([&] {
        return pe_linear_four_bit(x.p, x.s0, q.p, sc.p, (const float*)ts.p, fmt, b.p, r.p, r.s0, ptr(y), odt == x.dt ? elem : PE_ELEM_F32, act,
                                  ptr(ws), bytes, (int32_t)rows, (int32_t)k, (int32_t)outs, elem, current(x.dev));
    });
    return wrap(y);
}

// route(logits, top_k, stream)
PyObject* route(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "logits");
    if (x.dt != kF32) mismatch(x, "logits", "", kF32, x.d0, x.d1);
    const int64_t k = integer(args[1]);
    if (k < 1 || k > x.d1) bad(PE_ERR_INVALID, "top_k: %lld of %lld experts", (long long)k, (long long)x.d1);
    together(x, {});
    if (away(args[2], x.dev)) return go_there(self, "route", x.dev, args, n);
    const size_t bytes = pe_route_workspace((int32_t)x.d0, (int32_t)x.d1);
    const at::Tensor ids = empty(x.dev, kI32, x.d0, k), w = empty(x.dev, kF32, x.d0, k), off = empty(x.dev, kI32, x.d1 + 1),
                     place = empty(x.dev, kI32, x.d0, k);
    at::Tensor ws;
    if (bytes) ws = empty(x.dev, kU8, (int64_t)bytes);
    call([&] {
        return pe_route((const float*)x.p, x.s0, (int32_t*)ptr(ids), (float*)ptr(w), (int32_t*)ptr(off), (int32_t*)ptr(place), ptr(ws), bytes,
                        (int32_t)x.d0, (int32_t)k, (int32_t)x.d1, current(x.dev));
    });
    PyObject* a[4] = {wrap(ids), wrap(w), wrap(off), wrap(place)};
    PyObject* res = PyObject_Vectorcall(g_routing, a, 4, nullptr);
    for (PyObject* o : a) Py_XDECREF(o);
    return res;
}

// route_backward(dweights, weights, ids, experts, stream)
PyObject* route_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten w = matrix(args[1], "weights");
    whole(w, "weights", kF32, w.d0, w.d1);
    const Ten d = whole_of(args[0], "dweights", kF32, w.d0, w.d1), ids = whole_of(args[2], "ids", kI32, w.d0, w.d1);
    const int64_t experts = integer(args[3]);
    if (w.d1 < 1 || experts < w.d1) bad(PE_ERR_INVALID, "experts: %lld for a choice of %lld", (long long)experts, (long long)w.d1);
    fits(experts);
    together(w, {&d, &ids});
    if (away(args[4], w.dev)) return go_there(self, "route_backward", w.dev, args, n);
    const at::Tensor dl = empty(w.dev, kF32, w.d0, experts);
    call([&] {
        return pe_route_backward((const float*)d.p, (const float*)w.p, (const int32_t*)ids.p, (float*)ptr(dl), (int32_t)w.d0, (int32_t)w.d1,
                                 (int32_t)experts, current(w.dev));
    });
    return wrap(dl);
}

// The rows of the entries, contiguous int32 [tokens, top_k].
Ten place_of(PyObject* o, int64_t tokens) {
    const Ten p = load(o, "place");
    whole(p, "place", kI32, tokens < 0 ? p.d0 : tokens, p.d1);
    fits(p.d1);
    if (p.d1 < 1) bad(PE_ERR_INVALID, "place: no entries per token");
    if (p.d0 > PE_MAX_ROWS) bad(PE_ERR_RANGE, "place: a number of tokens of %lld is too large, at most %d", (long long)p.d0, PE_MAX_ROWS);
    return p;
}

// expand_rows(x, place, rows, stream)
PyObject* expand_rows(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), p = place_of(args[1], x.d0);
    const int elem = elem_of(x.dt, "x");
    const int64_t rows = args[2] == Py_None ? p.d0 * p.d1 : integer(args[2]);
    if (rows < 0 || rows > PE_MAX_ROWS) bad(PE_ERR_RANGE, "rows: %lld, at most %d", (long long)rows, PE_MAX_ROWS);
    together(x, {&p});
    if (away(args[3], x.dev)) return go_there(self, "expand_rows", x.dev, args, n);
    const at::Tensor y = empty(x.dev, x.dt, rows, x.d1);
    call([&] {
        return pe_expand_rows(x.p, x.s0, (const int32_t*)p.p, ptr(y), (int32_t)x.d0, (int32_t)p.d1, (int32_t)rows, (int32_t)x.d1, elem,
                              current(x.dev));
    });
    return wrap(y);
}

// combine_rows(y, place, weights, residual, stream)
PyObject* combine_rows(PyObject* self, Args args, Py_ssize_t n) {
    const Ten y = matrix(args[0], "y"), p = place_of(args[1], -1);
    const int elem = elem_of(y.dt, "y");
    const Ten w = args[2] == Py_None ? Ten() : whole_of(args[2], "weights", kF32, p.d0, p.d1);
    const Ten r = args[3] == Py_None ? Ten() : rows_of(args[3], "residual", y.dt, p.d0, y.d1);
    together(y, {&p, &w, &r});
    if (away(args[4], y.dev)) return go_there(self, "combine_rows", y.dev, args, n);
    const at::Tensor out = empty(y.dev, y.dt, p.d0, y.d1);
    call([&] {
        return pe_combine_rows(y.p, y.s0, (const int32_t*)p.p, (const float*)w.p, r.p, r.s0, ptr(out), (int32_t)p.d0, (int32_t)p.d1,
                               (int32_t)y.d0, (int32_t)y.d1, elem, current(y.dev));
    });
    return wrap(out);
}

// combine_rows_backward(dout, y, place, weights, stream)
PyObject* combine_rows_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten y = matrix(args[1], "y"), p = place_of(args[2], -1);
    const int elem = elem_of(y.dt, "y");
    const Ten d = rows_of(args[0], "dout", y.dt, p.d0, y.d1), w = whole_of(args[3], "weights", kF32, p.d0, p.d1);
    together(y, {&d, &p, &w});
    if (away(args[4], y.dev)) return go_there(self, "combine_rows_backward", y.dev, args, n);
    const at::Tensor dy = empty(y.dev, y.dt, y.d0, y.d1), dw = empty(y.dev, kF32, p.d0, p.d1);
    call([&] {
        return pe_combine_rows_backward(d.p, d.s0, y.p, y.s0, (const int32_t*)p.p, (const float*)w.p, ptr(dy), (float*)ptr(dw), (int32_t)p.d0,
                                        (int32_t)p.d1, (int32_t)y.d0, (int32_t)y.d1, elem, current(y.dev));
    });
    return tuple({&dy, &dw});
}

// grouped_linear(x, weight, offsets, stream)
PyObject* grouped_linear(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), w = load(args[1], "weight");
    const int elem = elem_of(x.dt, "x");
    const int64_t rows = x.d0, k = x.d1, g = w.d0, outs = w.d1;
    fits(outs);
    packed(w, "weight", x.dt, g, outs, k);
    const Ten off = offsets_of(args[2], g);
    together(x, {&w, &off});
    if (away(args[3], x.dev)) return go_there(self, "grouped_linear", x.dev, args, n);
    const at::Tensor y = empty(x.dev, x.dt, rows, outs);
    call([&] {
        return pe_grouped_linear(x.p, x.s0, w.p, (const int32_t*)off.p, ptr(y), (int32_t)rows, (int32_t)g, (int32_t)k, (int32_t)outs, elem,
                                 current(x.dev));
    });
    return wrap(y);
}

// grouped_linear_backward(dy, x, weight, offsets, stream)
PyObject* grouped_linear_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[1], "x"), w = load(args[2], "weight");
    const int elem = elem_of(x.dt, "x");
    const int64_t rows = x.d0, k = x.d1, g = w.d0, outs = w.d1;
    fits(outs);
    packed(w, "weight", x.dt, g, outs, k);
    const Ten dy = rows_of(args[0], "dy", x.dt, rows, outs), off = offsets_of(args[3], g);
    together(x, {&w, &dy, &off});
    if (away(args[4], x.dev)) return go_there(self, "grouped_linear_backward", x.dev, args, n);
    const at::Tensor dx = empty(x.dev, x.dt, rows, k), dw = empty(x.dev, x.dt, g, outs, k);
    call([&] {
        return pe_grouped_linear_backward(dy.p, dy.s0, x.p, x.s0, w.p, (const int32_t*)off.p, ptr(dx), ptr(dw), (int32_t)rows, (int32_t)g,
                                          (int32_t)k, (int32_t)outs, elem, current(x.dev));
    });
    return tuple({&dx, &dw});
}

// w13 and w2 of groups, for x: (groups, intermediate)
std::pair<int64_t, int64_t> experts_of(const Ten& x, const Ten& w13, const Ten& w2) {
    const int64_t g = w2.d0, i = w2.d2;
    fits(2 * i);
    packed(w2, "w2", x.dt, g, x.d1, i);
    packed(w13, "w13", x.dt, g, 2 * i, x.d1);
    return {g, i};
}

// grouped_ffn(x, w13, w2, offsets, act, save, stream)
PyObject* grouped_ffn(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[0], "x"), w13 = load(args[1], "w13"), w2 = load(args[2], "w2");
    const int act = act_of(args[4]), elem = elem_of(x.dt, "x");
    const bool save = truth(args[5]);
    const auto [g, i] = experts_of(x, w13, w2);
    const int64_t groups = g, inter = i;
    const Ten off = offsets_of(args[3], groups);
    together(x, {&w13, &w2, &off});
    if (away(args[6], x.dev)) return go_there(self, "grouped_ffn", x.dev, args, n);
    const size_t bytes = pe_grouped_ffn_workspace((int32_t)x.d0, (int32_t)inter);
    const at::Tensor y = empty(x.dev, x.dt, x.d0, x.d1), ws = empty(x.dev, kU8, (int64_t)bytes);
    at::Tensor gu;
    if (save) gu = empty(x.dev, kF32, x.d0, 2 * inter);
    call([&] {
        return pe_grouped_ffn(x.p, x.s0, w13.p, w2.p, (const int32_t*)off.p, ptr(y), ptr(gu), act, ptr(ws), bytes, (int32_t)x.d0,
                              (int32_t)groups, (int32_t)x.d1, (int32_t)inter, elem, current(x.dev));
    });
    return save ? tuple({&y, &gu}) : wrap(y);
}

// grouped_ffn_backward(dy, x, w13, w2, gu, offsets, act, stream)
PyObject* grouped_ffn_backward(PyObject* self, Args args, Py_ssize_t n) {
    const Ten x = matrix(args[1], "x"), w13 = load(args[2], "w13"), w2 = load(args[3], "w2");
    const int act = act_of(args[6]), elem = elem_of(x.dt, "x");
    const auto [g, i] = experts_of(x, w13, w2);
    const int64_t groups = g, inter = i;
    const Ten dy = rows_of(args[0], "dy", x.dt, x.d0, x.d1), gu = whole_of(args[4], "gu", kF32, x.d0, 2 * inter);
    const Ten off = offsets_of(args[5], groups);
    together(x, {&dy, &w13, &w2, &gu, &off});
    if (away(args[7], x.dev)) return go_there(self, "grouped_ffn_backward", x.dev, args, n);
    const size_t bytes = pe_grouped_ffn_backward_workspace((int32_t)x.d0, (int32_t)inter);
    const at::Tensor dx = empty(x.dev, x.dt, x.d0, x.d1), d13 = empty(x.dev, x.dt, groups, 2 * inter, x.d1),
                     d2 = empty(x.dev, x.dt, groups, x.d1, inter), ws = empty(x.dev, kU8, (int64_t)bytes);
    call([&] {
        return pe_grouped_ffn_backward(dy.p, dy.s0, x.p, x.s0, w13.p, w2.p, gu.p, (const int32_t*)off.p, act, ptr(dx), ptr(d13), ptr(d2),
                                       ptr(ws), bytes, (int32_t)x.d0, (int32_t)groups, (int32_t)x.d1, (int32_t)inter, elem, current(x.dev));
    });
    return tuple({&dx, &d13, &d2});
}

// setup(acts, raise, elsewhere, rmsnorm, routing, formats)
PyObject* setup(PyObject*, Args args, Py_ssize_t) {
    PyObject** to[6] = {&g_acts, &g_raise, &g_elsewhere, &g_rmsnorm, &g_routing, &g_formats};
    for (int i = 0; i < 6; ++i) Py_XSETREF(*to[i], Py_NewRef(args[i]));
    Py_RETURN_NONE;
}

// Counts the arguments and turns C++ exceptions into Python's.
template <PyObject* (*F)(PyObject*, Args, Py_ssize_t), int N>
PyObject* entry(PyObject* self, Args args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments, got %zd", N, n);
    try {
        return F(self, args, n);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define M(F, N) \
    { #F, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {M(setup, 6),
                         M(rms_norm, 8),
                         M(rms_norm_backward, 6),
                         M(linear, 10),
                         M(linear_backward, 7),
                         M(gated_ffn, 7),
                         M(gated_ffn_backward, 7),
                         M(linear_w4, 10),
                         M(route, 3),
                         M(route_backward, 5),
                         M(expand_rows, 4),
                         M(combine_rows, 5),
                         M(combine_rows_backward, 5),
                         M(grouped_linear, 4),
                         M(grouped_linear_backward, 5),
                         M(grouped_ffn, 7),
                         M(grouped_ffn_backward, 8),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dense", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dense(void) { return PyModule_Create(&module); }
