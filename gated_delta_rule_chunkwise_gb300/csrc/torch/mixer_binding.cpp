// Native half of mixer.py: checks torch tensors, allocates outputs and workspaces, and calls
// the C entry points of include/ldn.h (ldn_add_rmsnorm*, ldn_short_conv*, ldn_ssm_*) on the
// current stream of the tensors' device.  No computation.  A call for a single token is a few
// microseconds of GPU work, and the same steps taken in Python cost several times that.
//
// Functions take positional arguments from mixer.py, which documents them.  They return None
// where the first tensor is on another device than the current one (the caller switches and
// comes back), and raise TypeError, ValueError or the package's LdnError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <algorithm>
#include <climits>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>
#include <utility>
#include <vector>

#include "../../../include/ldn.h"

namespace {

using at::Tensor;
using Shape = c10::IntArrayRef;

PyObject *g_error = nullptr;   // the package's LdnError

struct Refusal {
    PyObject *type;
    std::string what;
};

[[noreturn]] __attribute__((format(printf, 2, 3))) void refuse(PyObject *type, const char *format, ...)
{
    char what[512];
    va_list v;
    va_start(v, format);
    vsnprintf(what, sizeof what, format, v);
    va_end(v);
    throw Refusal{type, what};
}

// Around a function's body: refusals, and what torch throws (out of memory among it), become
// Python's exceptions.
#define ENTRY       \
    HANDLE_TH_ERRORS \
    try {
#define LEAVE                                           \
    }                                                   \
    catch (const Refusal &e)                            \
    {                                                   \
        PyErr_SetString(e.type, e.what.c_str());        \
        return nullptr;                                 \
    }                                                   \
    catch (const PythonError &)                         \
    {                                                   \
        return nullptr;                                 \
    }                                                   \
    END_HANDLE_TH_ERRORS

std::string text(Shape s)
{
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}

// A tensor argument; null for None.
const Tensor *tensor(PyObject *o, const char *name)
{
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return &THPVariable_Unpack(o);
}

const Tensor &must(const Tensor *t, const char *name)
{
    if (!t) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return *t;
}

struct Call {
    int dev;
    at::TensorOptions options;   // of the first tensor
    explicit Call(const Tensor &x) : dev(x.get_device()), options(x.options()) {}
    Tensor make(Shape shape, at::ScalarType type) const { return at::empty(shape, options.dtype(type).requires_grad(false)); }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

// Whether the first tensor is on the GPU, and on the current device.
bool here(const Tensor &x, const char *name)
{
    if (!x.is_cuda()) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
    return x.get_device() == c10::cuda::current_device();
}

int code(const Tensor &t, const char *name)
{
    if (t.scalar_type() == at::kFloat) return LDN_F32;
    if (t.scalar_type() == at::kBFloat16) return LDN_BF16;
    refuse(PyExc_TypeError, "%s must be float32 or bfloat16, got %s", name, c10::toString(t.scalar_type()));
}

// A dense tensor of this shape and type on the call's device.
void check(const Tensor &t, const char *name, Shape shape, at::ScalarType type, int dev)
{
    if (!t.is_cuda() || t.layout() != at::kStrided) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
    if (t.get_device() != dev)
        refuse(PyExc_ValueError, "%s is on cuda:%d, expected cuda:%d", name, (int)t.get_device(), dev);
    if (t.is_neg()) refuse(PyExc_ValueError, "%s is a negated view: its memory holds the other sign", name);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s has dtype %s, expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, text(t.sizes()).c_str(), text(shape).c_str());
}

// The address of a contiguous one; null for an absent one.
template <typename T = void>
T *address(const Tensor *t, const char *name, Shape shape, at::ScalarType type, int dev)
{
    if (!t) return nullptr;
    check(*t, name, shape, type, dev);
    if (!t->is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return (T *)t->data_ptr();
}

// Elements between the rows that the `lead` leading dimensions count, where the others are
// one contiguous row; -1 where rows have no constant distance.
int64_t row_distance(const Tensor &t, int64_t lead)
{
    const Shape n = t.sizes(), s = t.strides();
    const int64_t d = t.dim();
    int64_t width = 1;
    for (int64_t i = d; i-- > lead;) {
        if (n[i] != 1 && s[i] != width) return t.numel() ? -1 : width * n[i];
        width *= n[i];
    }
    if (!t.numel()) return width;   // no rows: no distance between them
    int64_t ld = width;
    bool set = false;
    for (int64_t i = lead, rows = 1; i-- > 0; rows *= n[i]) {
        if (n[i] == 1) continue;
        if (set && s[i] != rows * ld) return -1;
        if (!set) ld = s[i];
        set = true;
    }
    return ld < width ? -1 : ld;
}

struct Rows {
    void *p;
    long long ld;
};

Rows rows(const Tensor &t, const char *name, Shape shape, at::ScalarType type, int dev, int64_t lead)
{
    check(t, name, shape, type, dev);
    const int64_t ld = row_distance(t, lead);
    if (ld < 0)
        refuse(PyExc_ValueError, "%s has strides %s: rows must be contiguous and a constant distance apart", name,
                                text(t.strides()).c_str());
    return {t.data_ptr(), ld};
}

bool done(int status, const char *what)
{
    if (status == LDN_OK) return true;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return false;
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }

PyObject *tuple(std::initializer_list<PyObject *> items)   // takes the references
{
    PyObject *t = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject *o : items) PyTuple_SET_ITEM(t, i++, o);
    return t;
}

PyObject *kept(PyObject *o)
{
    Py_INCREF(o);
    return o;
}

// A dict of tensors; undefined ones as None.
PyObject *dict(std::initializer_list<std::pair<const char *, const Tensor *>> items)
{
    PyObject *d = PyDict_New();
    for (const auto &it : items) {
        PyObject *o = it.second && it.second->defined() ? wrap(*it.second) : kept(Py_None);
        PyDict_SetItemString(d, it.first, o);
        Py_DECREF(o);
    }
    return d;
}

// A tensor of the caller's that the call writes: a graph that saved its values is to notice.
void written(const Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A given output, checked, or a new one; `o` becomes a new reference to it.
template <typename T = void>
T *output(const Call &c, PyObject *&o, const char *name, Shape shape, at::ScalarType type)
{
    if (o != Py_None) {
        const Tensor *t = tensor(o, name);
        T *p = address<T>(t, name, shape, type, c.dev);
        written(*t);
        Py_INCREF(o);
        return p;
    }
    const Tensor t = c.make(shape, type);
    o = wrap(t);
    return (T *)t.data_ptr();
}

struct PythonError {};   // one is set

// These calls record no gradients.  Where a graph is being recorded and an argument wants one,
// the caller most likely meant autograd's form, and would otherwise see only that a gradient is
// missing.  The warning is the caller's of mixer.py's function.
void warn_without_gradient(PyObject *const *a, Py_ssize_t n, const char *name, bool recorded = true)
{
    if (!c10::GradMode::is_enabled()) return;
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!THPVariable_Check(a[i]) || !THPVariable_Unpack(a[i]).requires_grad()) continue;
        const int failed = recorded
            ? PyErr_WarnFormat(PyExc_UserWarning, 3, "%s: an argument requires a gradient and this call records none: "
                               "call autograd.%s, or this one under torch.no_grad()", name, name)
            : PyErr_WarnFormat(PyExc_UserWarning, 3, "%s: an argument requires a gradient and this call has none",
                               name);
        if (failed) throw PythonError{};
        return;
    }
}

int as_int(PyObject *o)
{
    const int v = PyLong_Check(o) ? (int)std::max(-1L, std::min(PyLong_AsLong(o), (long)INT_MAX)) : -1;
    if (!PyLong_Check(o)) refuse(PyExc_TypeError, "an int is wanted, got %s", Py_TYPE(o)->tp_name);
    if (PyErr_Occurred()) throw PythonError{};
    return v;
}
int truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw PythonError{};
    return v;
}
float as_float(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return (float)v;
}
// A size as the C entry points take it.
int size(int64_t n)
{
    if (n > INT_MAX) refuse(PyExc_ValueError, "a dimension of %lld is too large", (long long)n);
    return (int)n;
}

#define NEEDS(n)                                                                      \
    if (nargs != (n)) {                                                               \
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");                \
        return nullptr;                                                               \
    }

// ---- RMS norm with the residual's addition ----
// (x, residual, weight, eps, out, residual_out) -> (y, s); with (group, scale) appended
// (q, scale, s)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    if (nargs != 6 && nargs != 8) NEEDS(6);
    const bool eight = nargs == 8;
    const Tensor &x = must(tensor(a[0], "x"), "x"), *r = tensor(a[1], "residual"), *w = tensor(a[2], "weight");
    if (!here(x, "x")) Py_RETURN_NONE;
    if (x.dim() < 1) refuse(PyExc_ValueError, "x must have at least one dimension");
    if (eight) warn_without_gradient(a, nargs, "add_rmsnorm_e4m3", false);
    else warn_without_gradient(a, nargs, "add_rmsnorm");
    const Call c(x);
    const float eps = as_float(a[3]);
    const Shape shape = x.sizes();
    const int64_t D = shape.back(), n = D ? x.numel() / D : 0, wshape[] = {D};
    const int cx = code(x, "x");
    void *px = address(&x, "x", shape, x.scalar_type(), c.dev);
    float *pw = address<float>(&must(w, "weight"), "weight", Shape(wshape, 1), at::kFloat, c.dev);
    int cr = cx;
    void *pr = nullptr, *po = nullptr;
    if (r) {
        cr = code(*r, "residual");
        pr = address(r, "residual", shape, r->scalar_type(), c.dev);
    } else if (a[5] != Py_None) {
        refuse(PyExc_ValueError, "residual_out without residual");
    }
    int group = 0;
    std::vector<int64_t> sshape;
    if (eight) {
        group = as_int(a[6]);
        sshape.assign(shape.begin(), shape.end() - 1);
        if (group) sshape.push_back((D + 127) / 128);
    }
    // references are taken in this order and given up together on an error
    THPObjectPtr hold_s, hold_y, hold_scale;
    PyObject *s = r ? a[5] : a[0], *y = a[4], *scale = eight ? a[7] : Py_None;
    if (r) {
        po = output(c, s, "residual_out", shape, r->scalar_type());
        hold_s = s;
    } else {
        hold_s = kept(s);
    }
    void *py = output(c, y, "out", shape, eight ? at::kFloat8_e4m3fn : x.scalar_type());
    hold_y = y;
    int st;
    if (eight) {
        float *ps = output<float>(c, scale, "scale", sshape, at::kFloat);
        hold_scale = scale;
        st = ldn_add_rmsnorm_e4m3(px, pr, pw, py, ps, po, n, size(D), group, cx, cr, eps, c.stream());
    } else {
        st = ldn_add_rmsnorm(px, pr, pw, py, po, n, size(D), cx, cr, eps, c.stream());
    }
    if (!done(st, eight ? "ldn_add_rmsnorm_e4m3" : "ldn_add_rmsnorm")) return nullptr;
    if (eight) return tuple({hold_y.release(), hold_scale.release(), hold_s.release()});
    return tuple({hold_y.release(), hold_s.release()});
    LEAVE
}

// (dy, s, weight, dsum, eps) -> dict
PyObject *add_rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(5);
    const Tensor &dy = must(tensor(a[0], "dy"), "dy"), *s = tensor(a[1], "s"), *w = tensor(a[2], "weight"),
                 *dsum = tensor(a[3], "dsum");
    if (!here(dy, "dy")) Py_RETURN_NONE;
    if (dy.dim() < 1) refuse(PyExc_ValueError, "dy must have at least one dimension");
    const Call c(dy);
    const float eps = as_float(a[4]);
    const Shape shape = dy.sizes();
    const int64_t D = shape.back(), n = D ? dy.numel() / D : 0, wshape[] = {D};
    const int cx = code(dy, "dy"), cr = code(must(s, "s"), "s");
    void *pdy = address(&dy, "dy", shape, dy.scalar_type(), c.dev), *ps = address(s, "s", shape, s->scalar_type(), c.dev);
    float *pw = address<float>(&must(w, "weight"), "weight", Shape(wshape, 1), at::kFloat, c.dev);
    void *pd = address(dsum, "dsum", shape, s->scalar_type(), c.dev);
    const size_t need = ldn_add_rmsnorm_backward_workspace_size(n, size(D));
    const int64_t ws_n[] = {(int64_t)need};
    const Tensor dx = c.make(shape, dy.scalar_type()), dres = cx == cr ? dx : c.make(shape, s->scalar_type()),
                 dw = c.make(Shape(wshape, 1), at::kFloat), ws = c.make(Shape(ws_n, 1), at::kByte);
    if (!done(ldn_add_rmsnorm_backward(pdy, ps, pw, pd, dx.data_ptr(), cx == cr ? nullptr : dres.data_ptr(),
                                       (float *)dw.data_ptr(), n, size(D), cx, cr, eps, need ? ws.data_ptr() : nullptr,
                                       need, c.stream()), "ldn_add_rmsnorm_backward"))
        return nullptr;
    PyObject *d = dict({{"dx", &dx}, {"dweight", &dw}});
    if (cx == cr) {
        PyDict_SetItemString(d, "dresidual", PyDict_GetItemString(d, "dx"));   // the same tensor
    } else {
        PyObject *o = wrap(dres);
        PyDict_SetItemString(d, "dresidual", o);
        Py_DECREF(o);
    }
    return d;
    LEAVE
}

// ---- Short causal convolution ----
struct ConvIn {
    Rows x;
    float *w, *b;
    int64_t C, W;
    int code;
    ConvIn(const Call &c, const Tensor &t, const Tensor *weight, const Tensor *bias, int64_t lead)
    {
        if (t.dim() != lead + 1)
            refuse(PyExc_ValueError, "x must have %d dimensions, got %d", (int)lead + 1, (int)t.dim());
        code = ::code(t, "x");
        if (!weight || weight->dim() != 2) refuse(PyExc_TypeError, "weight must be a CUDA tensor [C, width]");
        C = t.size(lead);
        W = weight->size(1);
        const int64_t ws[] = {C, W}, bs[] = {C};
        x = rows(t, "x", t.sizes(), t.scalar_type(), c.dev, lead);
        w = address<float>(weight, "weight", Shape(ws, 2), at::kFloat, c.dev);
        b = address<float>(bias, "bias", Shape(bs, 1), at::kFloat, c.dev);
    }
};

// (x, weight, bias, state, lens, activation, out, state_out) -> (y, state_out)
PyObject *short_conv(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(8);
    const Tensor &x = must(tensor(a[0], "x"), "x");
    if (!here(x, "x")) Py_RETURN_NONE;
    warn_without_gradient(a, nargs, "short_conv");
    const Call c(x);
    const at::ScalarType t = x.scalar_type();
    const ConvIn in(c, x, tensor(a[1], "weight"), tensor(a[2], "bias"), 2);
    const int64_t B = x.size(0), T = x.size(1), ys[] = {B, T, in.C}, ss[] = {B, in.W - 1, in.C}, ls[] = {B};
    void *pst = address(tensor(a[3], "state"), "state", Shape(ss, 3), t, c.dev);
    int *pl = address<int>(tensor(a[4], "lens"), "lens", Shape(ls, 1), at::kInt, c.dev);
    PyObject *y = a[6], *so = a[7];
    THPObjectPtr hold_y, hold_s;
    void *py = output(c, y, "out", Shape(ys, 3), t);
    hold_y = y;
    void *ps = output(c, so, "state_out", Shape(ss, 3), t);
    hold_s = so;
    if (!done(ldn_short_conv(in.x.p, in.x.ld, in.w, in.b, pst, pl, py, ps, size(B), size(T), size(in.C), size(in.W),
                             truth(a[5]), in.code, c.stream()), "ldn_short_conv"))
        return nullptr;
    return tuple({hold_y.release(), hold_s.release()});
    LEAVE
}

// (x, weight, bias, state, activation, out, state_out) -> y
PyObject *short_conv_step(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(7);
    const Tensor &x = must(tensor(a[0], "x"), "x"), *so = tensor(a[6], "state_out");
    if (!here(x, "x")) Py_RETURN_NONE;
    const Call c(x);
    const at::ScalarType t = x.scalar_type();
    const ConvIn in(c, x, tensor(a[1], "weight"), tensor(a[2], "bias"), 1);
    const int64_t B = x.size(0), ys[] = {B, in.C}, ss[] = {B, in.W - 1, in.C};
    const Tensor *st = tensor(a[3], "state");
    void *pst = address(st, "state", Shape(ss, 3), t, c.dev);
    void *ps = so ? address(so, "state_out", Shape(ss, 3), t, c.dev) : pst;
    PyObject *y = a[5];
    void *py = output(c, y, "out", Shape(ys, 2), t);
    if (so || st) written(so ? *so : *st);
    THPObjectPtr hold_y(y);
    if (!done(ldn_short_conv_step(in.x.p, in.x.ld, in.w, in.b, pst, py, ps, size(B), size(in.C), size(in.W), truth(a[4]),
                                  in.code, c.stream()), "ldn_short_conv_step"))
        return nullptr;
    return hold_y.release();
    LEAVE
}

// (x, weight, bias, dy, state, dstate_out, lens, activation) -> dict
PyObject *short_conv_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(8);
    const Tensor &x = must(tensor(a[0], "x"), "x"), *bias = tensor(a[2], "bias"), *dy = tensor(a[3], "dy"),
                 *state = tensor(a[4], "state");
    if (!here(x, "x")) Py_RETURN_NONE;
    const Call c(x);
    const at::ScalarType t = x.scalar_type();
    const ConvIn in(c, x, tensor(a[1], "weight"), bias, 2);
    const int64_t B = x.size(0), T = x.size(1), ys[] = {B, T, in.C}, ss[] = {B, in.W - 1, in.C}, ls[] = {B},
                  ws_[] = {in.C, in.W};
    void *pst = address(state, "state", Shape(ss, 3), t, c.dev);
    void *pds = address(tensor(a[5], "dstate_out"), "dstate_out", Shape(ss, 3), t, c.dev);
    void *pdy = address(&must(dy, "dy"), "dy", Shape(ys, 3), t, c.dev);
    int *pl = address<int>(tensor(a[6], "lens"), "lens", Shape(ls, 1), at::kInt, c.dev);
    const size_t need = ldn_short_conv_backward_workspace_size(size(B), size(T), size(in.C), size(in.W));
    const int64_t nws[] = {(int64_t)(need ? need : 16)};
    Tensor dx = c.make(Shape(ys, 3), t), dw = c.make(Shape(ws_, 2), at::kFloat), ws = c.make(Shape(nws, 1), at::kByte), db,
           dst;
    if (bias) db = c.make(Shape(ws_, 1), at::kFloat);
    if (state) dst = c.make(Shape(ss, 3), t);
    if (!done(ldn_short_conv_backward(in.x.p, in.x.ld, in.w, in.b, pst, pl, pdy, pds, dx.data_ptr(),
                                      (float *)dw.data_ptr(), bias ? (float *)db.data_ptr() : nullptr,
                                      state ? dst.data_ptr() : nullptr, size(B), size(T), size(in.C), size(in.W),
                                      truth(a[7]), in.code, ws.data_ptr(), need, c.stream()),
              "ldn_short_conv_backward"))
        return nullptr;
    return dict({{"dx", &dx}, {"dweight", &dw}, {"dbias", &db}, {"dstate", &dst}});
    LEAVE
}

// ---- Selective state space scan ----
struct ScanIn {
    Rows u, d, B, C, z;
    float *A, *D, *bias;
    int64_t Dm, G, N;
    int code;
    Shape bshape;
    // u, delta, A, B, C, D, z, delta_bias from a[0]
    ScanIn(const Call &c, PyObject *const *a, int64_t lead)
    {
        const Tensor &tu = must(tensor(a[0], "u"), "u"), *td = tensor(a[1], "delta"), *tA = tensor(a[2], "A"),
                     *tB = tensor(a[3], "B"), *tC = tensor(a[4], "C"), *tD = tensor(a[5], "D"), *tz = tensor(a[6], "z"),
                     *tb = tensor(a[7], "delta_bias");
        const Shape s = tu.sizes();
        const at::ScalarType t = tu.scalar_type();
        if (tu.dim() != lead + 1)
            refuse(PyExc_ValueError, "u must have %d dimensions, got %d", (int)lead + 1, (int)tu.dim());
        code = ::code(tu, "u");
        if (!tB || tB->dim() != lead + 2)
            refuse(PyExc_ValueError, "B must be a CUDA tensor of %d dimensions", (int)lead + 2);
        bshape = tB->sizes();
        Dm = s[lead];
        G = bshape[lead];
        N = bshape[lead + 1];
        int64_t want[4] = {s[0], lead == 2 ? s[1] : G, lead == 2 ? G : N, N};
        const int64_t as[] = {Dm, N};
        u = rows(tu, "u", s, t, c.dev, lead);
        d = rows(must(td, "delta"), "delta", s, t, c.dev, lead);
        B = rows(*tB, "B", Shape(want, lead + 2), t, c.dev, lead);
        C = rows(must(tC, "C"), "C", Shape(want, lead + 2), t, c.dev, lead);
        z = tz ? rows(*tz, "z", s, t, c.dev, lead) : Rows{nullptr, Dm};
        A = address<float>(&must(tA, "A"), "A", Shape(as, 2), at::kFloat, c.dev);
        D = address<float>(tD, "D", Shape(as, 1), at::kFloat, c.dev);
        bias = address<float>(tb, "delta_bias", Shape(as, 1), at::kFloat, c.dev);
    }
};

// (u, delta, A, B, C, D, z, delta_bias, h0, delta_softplus, lens, save_states, out, h_final,
//  workspace) -> (y, h_final[, states])
PyObject *selective_scan(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(15);
    const Tensor &u = must(tensor(a[0], "u"), "u"), *given = tensor(a[14], "workspace");
    if (!here(u, "u")) Py_RETURN_NONE;
    warn_without_gradient(a, nargs, "selective_scan");
    const Call c(u);
    const at::ScalarType t = u.scalar_type();
    const ScanIn in(c, a, 2);
    const int64_t nb = u.size(0), T = u.size(1), hs[] = {nb, in.Dm, in.N}, ls[] = {nb},
                  cs[] = {nb, (T + 31) / 32, in.Dm, in.N};
    float *ph = address<float>(tensor(a[8], "h0"), "h0", Shape(hs, 3), at::kFloat, c.dev);
    int *pl = address<int>(tensor(a[10], "lens"), "lens", Shape(ls, 1), at::kInt, c.dev);
    const bool save = truth(a[11]);
    PyObject *y = a[12], *h = a[13];
    THPObjectPtr hold_y, hold_h;
    void *py = output(c, y, "out", u.sizes(), t);
    hold_y = y;
    float *pf = output<float>(c, h, "h_final", Shape(hs, 3), at::kFloat);
    hold_h = h;
    Tensor states, ws;
    if (save) states = c.make(Shape(cs, 4), at::kFloat);
    void *pws = nullptr;
    size_t nws = 0;
    if (given) {
        pws = address(given, "workspace", given->sizes(), at::kByte, c.dev);
        nws = (size_t)given->numel();
    } else if ((nws = ldn_ssm_scan_workspace_size(size(nb), size(T), size(in.Dm), size(in.N), size(in.G))) != 0) {
        const int64_t n[] = {(int64_t)nws};
        ws = c.make(Shape(n, 1), at::kByte);
        pws = ws.data_ptr();
    }
    if (!done(ldn_ssm_scan(in.u.p, in.u.ld, in.d.p, in.d.ld, in.A, in.B.p, in.B.ld, in.C.p, in.C.ld, in.D, in.z.p,
                           in.z.ld, in.bias, ph, pl, py, pf, save ? (float *)states.data_ptr() : nullptr, size(nb),
                           size(T), size(in.Dm), size(in.N), size(in.G), truth(a[9]), in.code, nws ? pws : nullptr, nws,
                           c.stream()), "ldn_ssm_scan"))
        return nullptr;
    if (save) return tuple({hold_y.release(), hold_h.release(), wrap(states)});
    return tuple({hold_y.release(), hold_h.release()});
    LEAVE
}

// (u, delta, A, B, C, D, z, delta_bias, h, delta_softplus, out, h_out) -> y
PyObject *selective_scan_step(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(12);
    const Tensor &u = must(tensor(a[0], "u"), "u"), *ho = tensor(a[11], "h_out");
    if (!here(u, "u")) Py_RETURN_NONE;
    const Call c(u);
    const ScanIn in(c, a, 1);
    const int64_t nb = u.size(0), hs[] = {nb, in.Dm, in.N};
    const Tensor &h = must(tensor(a[8], "h"), "h");
    float *ph = address<float>(&h, "h", Shape(hs, 3), at::kFloat, c.dev);
    float *po = ho ? address<float>(ho, "h_out", Shape(hs, 3), at::kFloat, c.dev) : ph;
    written(ho ? *ho : h);
    PyObject *y = a[10];
    void *py = output(c, y, "out", u.sizes(), u.scalar_type());
    THPObjectPtr hold_y(y);
    if (!done(ldn_ssm_step(in.u.p, in.u.ld, in.d.p, in.d.ld, in.A, in.B.p, in.B.ld, in.C.p, in.C.ld, in.D, in.z.p,
                           in.z.ld, in.bias, ph, po, py, size(nb), size(in.Dm), size(in.N), size(in.G), truth(a[9]),
                           in.code, c.stream()), "ldn_ssm_step"))
        return nullptr;
    return hold_y.release();
    LEAVE
}

// (u, delta, A, B, C, D, z, delta_bias, states, dy, dh_final, delta_softplus, lens) -> dict
PyObject *selective_scan_backward(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(13);
    const Tensor &u = must(tensor(a[0], "u"), "u");
    if (!here(u, "u")) Py_RETURN_NONE;
    const Call c(u);
    const at::ScalarType t = u.scalar_type();
    const ScanIn in(c, a, 2);
    const int64_t nb = u.size(0), T = u.size(1), hs[] = {nb, in.Dm, in.N}, ls[] = {nb},
                  cs[] = {nb, (T + 31) / 32, in.Dm, in.N}, as[] = {in.Dm, in.N};
    float *ps = address<float>(&must(tensor(a[8], "states"), "states"), "states", Shape(cs, 4), at::kFloat, c.dev);
    void *pdy = address(&must(tensor(a[9], "dy"), "dy"), "dy", u.sizes(), t, c.dev);
    float *pdh = address<float>(tensor(a[10], "dh_final"), "dh_final", Shape(hs, 3), at::kFloat, c.dev);
    int *pl = address<int>(tensor(a[12], "lens"), "lens", Shape(ls, 1), at::kInt, c.dev);
    Tensor du = c.make(u.sizes(), t), dd = c.make(u.sizes(), t), dA = c.make(Shape(as, 2), at::kFloat),
           dB = c.make(in.bshape, t), dC = c.make(in.bshape, t), dh0 = c.make(Shape(hs, 3), at::kFloat), dD, dz, db;
    if (in.D) dD = c.make(Shape(as, 1), at::kFloat);
    if (a[6] != Py_None) dz = c.make(u.sizes(), t);
    if (in.bias) db = c.make(Shape(as, 1), at::kFloat);
    auto p = [](const Tensor &x) { return x.defined() ? x.data_ptr() : nullptr; };
    const size_t need = ldn_ssm_backward_workspace_size(size(nb), size(T), size(in.Dm), size(in.N), size(in.G));
    const int64_t nws[] = {(int64_t)(need ? need : 16)};
    const Tensor ws = c.make(Shape(nws, 1), at::kByte);
    if (!done(ldn_ssm_backward(in.u.p, in.u.ld, in.d.p, in.d.ld, in.A, in.B.p, in.B.ld, in.C.p, in.C.ld, in.D, in.z.p,
                               in.z.ld, in.bias, ps, pl, pdy, pdh, p(du), p(dd), (float *)p(dA), p(dB), p(dC),
                               (float *)p(dD), p(dz), (float *)p(db), (float *)p(dh0), size(nb), size(T), size(in.Dm),
                               size(in.N), size(in.G), truth(a[11]), in.code, ws.data_ptr(), need, c.stream()),
              "ldn_ssm_backward"))
        return nullptr;
    return dict({{"du", &du}, {"ddelta", &dd}, {"dA", &dA}, {"dB", &dB}, {"dC", &dC}, {"dD", &dD}, {"dz", &dz},
                 {"ddelta_bias", &db}, {"dh0", &dh0}});
    LEAVE
}

// (t, lead) -> elements between rows, or -1
PyObject *py_row_distance(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    ENTRY
    NEEDS(2);
    return PyLong_FromLongLong(row_distance(must(tensor(a[0], "t"), "t"), as_int(a[1])));
    LEAVE
}

// (LdnError): the exception of a failed call
PyObject *set_error(PyObject *, PyObject *const *a, Py_ssize_t nargs)
{
    NEEDS(1);
    Py_INCREF(a[0]);
    Py_XSETREF(g_error, a[0]);
    Py_RETURN_NONE;
}

#define FAST(name, fn) {name, (PyCFunction)(void (*)(void))fn, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("add_rmsnorm", add_rmsnorm),
                         FAST("add_rmsnorm_backward", add_rmsnorm_backward),
                         FAST("short_conv", short_conv),
                         FAST("short_conv_step", short_conv_step),
                         FAST("short_conv_backward", short_conv_backward),
                         FAST("selective_scan", selective_scan),
                         FAST("selective_scan_step", selective_scan_step),
                         FAST("selective_scan_backward", selective_scan_backward),
                         FAST("row_distance", py_row_distance),
                         FAST("set_error", set_error),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ldn_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ldn_torch(void) { return PyModule_Create(&module); }
