// Python entry of the operators in train_api.cu (module ttm_torch): checks torch
// tensors, allocates outputs and workspaces with torch on the current stream, and
// calls the C ABI.  train.py documents the functions and is the only caller.
//
// Why compiled: a call of these operators takes the GPU a few microseconds, and
// marshalling it in Python took 12 (one output) to 27 (five allocations).
//
// Every function takes its arguments by position, None for an absent tensor.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <optional>
#include <string>
#include <vector>

#include "../../include/ttm.h"

namespace {

PyObject* g_error = nullptr;   // TTMError of the package

struct Failure {               // becomes TTMError(code, what)
    int code;
    std::string what;
};
struct WrongType {             // becomes TypeError
    std::string what;
};
struct PythonError {};         // already set

[[noreturn]] void bad(const std::string& what) { throw Failure{TTM_ERR_INVALID_ARG, what}; }

using Maybe = std::optional<at::Tensor>;

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!THPVariable_Check(o)) bad(std::string(what) + " must be a tensor");
    return THPVariable_Unpack(o);
}
Maybe maybe(PyObject* o, const char* what) {
    if (o == Py_None) return std::nullopt;
    return tensor(o, what);
}

int dtype_code(const at::Tensor& t, const char* what) {
    if (t.scalar_type() == at::kFloat) return TTM_F32;
    if (t.scalar_type() == at::kBFloat16) return TTM_BF16;
    throw WrongType{std::string(what) + " must be float32 or bfloat16"};
}

int narrow(int64_t v, const char* what) {
    if (v > INT_MAX) throw Failure{TTM_ERR_UNSUPPORTED, std::string(what) + ": a size of 2^31 or more"};
    return (int)v;
}

void* ptr(const Maybe& t) { return t ? t->data_ptr() : nullptr; }
float* fptr(const Maybe& t) { return t ? static_cast<float*>(t->data_ptr()) : nullptr; }

// A given tensor that has to be contiguous, of this type and shape, on this device.
void check(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev,
           const char* what) {
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || t.device() != dev)
        bad(std::string(what) + " must be contiguous, of the right dtype and shape and on the call's device");
}
void check(const Maybe& t, at::IntArrayRef shape, const at::Device& dev, const char* what) {
    if (t) check(*t, shape, at::kFloat, dev, what);
}

// Without the dispatcher, which takes longer than the allocation itself.
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
at::Tensor output(const Maybe& given, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev,
                  const char* what) {
    if (!given) return make(shape, type, dev);
    check(*given, shape, type, dev, what);
    return *given;
}
Maybe scratch(const Maybe& given, size_t need, const at::Device& dev) {
    if (given) {
        if (given->device() != dev || !given->is_contiguous())
            bad("workspace must be a contiguous tensor on the device of the call");
        return given;
    }
    if (!need) return std::nullopt;
    return make({(int64_t)need}, at::kByte, dev);
}
size_t bytes(const Maybe& t) { return t ? t->nbytes() : 0; }

void* current_stream(const at::Device& dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

void done(int code, const char* what) {
    if (code != TTM_OK) throw Failure{code, what};
}

// Elements between consecutive entries of the first `lead` dimensions taken as one; none when
// there is at most one entry.
std::optional<int64_t> one_stride(const at::Tensor& t, int64_t lead, const char* what) {
    std::optional<int64_t> step;
    int64_t size = 1;
    for (int64_t k = lead - 1; k >= 0; --k) {
        if (t.size(k) == 1) continue;
        if (!step) step = t.stride(k);
        else if (t.stride(k) != *step * size)
            bad(std::string(what) + ": the leading dimensions have no single stride");
        size *= t.size(k);
    }
    return step;
}

void strides(const at::Tensor& t, int64_t lead, int64_t inner, const char* what, long long& seq,
             long long& tok) {
    tok = t.size(lead) > 1 ? t.stride(lead) : inner;
    seq = one_stride(t, lead, what).value_or(t.size(lead) * tok);
}

// x [..., T, D] and its gate: of the same shape (per channel) or [..., T] fp32 (per token).
struct Glr {
    int N, T, D, dtype, gate;
    long long xs, xt, gs, gt;
    std::vector<int64_t> state;
};

Glr glr_shapes(const at::Tensor& x, const at::Tensor& g, const char* what) {
    Glr r;
    const int64_t lead = x.dim() - 2;
    if (lead < 0) bad(std::string(what) + ": expected [..., T, D]");
    const int64_t T = x.size(lead), D = x.size(lead + 1);
    int64_t N = 1;
    for (int64_t k = 0; k < lead; ++k) N *= x.size(k);
    r.dtype = dtype_code(x, what);
    if ((D > 1 && x.stride(lead + 1) != 1) || !x.is_cuda() || x.device() != g.device())
        bad(std::string(what) + ": channels must be contiguous, all tensors on one CUDA device");
    if (g.dim() == lead + 2) {
        if (g.sizes() != x.sizes() || g.scalar_type() != x.scalar_type() || (D > 1 && g.stride(lead + 1) != 1))
            bad(std::string(what) + ": a gate per channel has the shape, dtype and channel order of x");
        r.gate = TTM_GATE_CHANNEL;
    } else {
        if (g.sizes() != x.sizes().slice(0, lead + 1) || g.scalar_type() != at::kFloat)
            bad(std::string(what) + ": a gate per token is float32 of the shape of x without its last axis");
        r.gate = TTM_GATE_TOKEN;
    }
    r.N = narrow(N, what);
    r.T = narrow(T, what);
    r.D = narrow(D, what);
    strides(x, lead, D, what, r.xs, r.xt);
    strides(g, lead, r.gate == TTM_GATE_TOKEN ? 1 : D, what, r.gs, r.gt);
    r.state.assign(x.sizes().begin(), x.sizes().begin() + lead);
    r.state.push_back(D);
    return r;
}

PyObject* wrap(const Maybe& t) {
    if (t) return THPVariable_Wrap(*t);
    Py_RETURN_NONE;
}

PyObject* tuple(std::initializer_list<Maybe> ts) {
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) throw PythonError{};
    Py_ssize_t i = 0;
    for (const Maybe& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
    return r;
}

// (x, g, h0, h, h_last, workspace) -> (h, h_last)
PyObject* glr_fwd(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &g = tensor(a[1], "g");
    const Maybe h0 = maybe(a[2], "h0");
    const Glr s = glr_shapes(x, g, "glr_fwd");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(h0, s.state, dev, "h0");
    at::Tensor h = output(maybe(a[3], "h"), x.sizes(), x.scalar_type(), dev, "h");
    at::Tensor last = output(maybe(a[4], "h_last"), s.state, at::kFloat, dev, "h_last");
    const Maybe ws = scratch(maybe(a[5], "workspace"),
                             ttm_glr_workspace_size(s.N, s.T, s.D, s.dtype, s.gate, 0), dev);
    done(ttm_glr_fwd(s.N, s.T, s.D, s.dtype, s.gate, x.data_ptr(), s.xs, s.xt, g.data_ptr(), s.gs, s.gt,
                     fptr(h0), h.data_ptr(), static_cast<float*>(last.data_ptr()), ptr(ws), bytes(ws),
                     current_stream(dev)),
         "ttm_glr_fwd");
    return tuple({h, last});
}

// (g, h, dh, h0, dh_last, want_dh0, dx, dg, dh0, workspace) -> (dx, dg, dh0)
PyObject* glr_bwd(PyObject* const* a) {
    const at::Tensor &g = tensor(a[0], "g"), &h = tensor(a[1], "h"), &dh = tensor(a[2], "dh");
    const Maybe h0 = maybe(a[3], "h0"), dl = maybe(a[4], "dh_last");
    const Glr s = glr_shapes(dh, g, "glr_bwd");
    const at::Device dev = dh.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(h, dh.sizes(), dh.scalar_type(), dev, "h");
    check(h0, s.state, dev, "h0");
    check(dl, s.state, dev, "dh_last");
    at::Tensor dx = output(maybe(a[6], "dx"), dh.sizes(), dh.scalar_type(), dev, "dx");
    at::Tensor dg = output(maybe(a[7], "dg"), g.sizes(), g.scalar_type(), dev, "dg");
    Maybe d0;
    if (a[5] == Py_True) d0 = output(maybe(a[8], "dh0"), s.state, at::kFloat, dev, "dh0");
    const Maybe ws = scratch(maybe(a[9], "workspace"),
                             ttm_glr_workspace_size(s.N, s.T, s.D, s.dtype, s.gate, 1), dev);
    done(ttm_glr_bwd(s.N, s.T, s.D, s.dtype, s.gate, g.data_ptr(), s.gs, s.gt, h.data_ptr(), fptr(h0),
                     dh.data_ptr(), s.xs, s.xt, fptr(dl), dx.data_ptr(), dg.data_ptr(), fptr(d0), ptr(ws),
                     bytes(ws), current_stream(dev)),
         "ttm_glr_bwd");
    return tuple({dx, dg, d0});
}

// (x, g, state, h) -> h
PyObject* glr_step(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &g = tensor(a[1], "g"), &state = tensor(a[2], "state");
    const Glr s = glr_shapes(x, g, "glr_step");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(state, s.state, at::kFloat, dev, "state");
    at::Tensor h = output(maybe(a[3], "h"), x.sizes(), x.scalar_type(), dev, "h");
    done(ttm_glr_step(s.N, s.T, s.D, s.dtype, s.gate, x.data_ptr(), s.xs, s.xt, g.data_ptr(), s.gs, s.gt,
                      static_cast<float*>(state.data_ptr()), h.data_ptr(), current_stream(dev)),
         "ttm_glr_step");
    return wrap(h);
}

// Rows of x [..., D] and the elements between them.
void rows(const at::Tensor& x, const char* what, int& N, int& D, long long& step) {
    if (x.dim() < 1 || (x.size(-1) > 1 && x.stride(-1) != 1) || !x.is_cuda())
        bad(std::string(what) + ": expected a CUDA tensor [..., D] with a contiguous last axis");
    int64_t n = 1;
    for (int64_t k = 0; k + 1 < x.dim(); ++k) n *= x.size(k);
    N = narrow(n, what);
    D = narrow(x.size(-1), what);
    step = x.is_contiguous() ? D : one_stride(x, x.dim() - 1, what).value_or(D);
}

// (x, w, b, eps, y, mean, rstd, want_stats) -> (y, mean, rstd)
PyObject* layer_norm_fwd(PyObject* const* a) {
    const at::Tensor& x = tensor(a[0], "x");
    const Maybe w = maybe(a[1], "w"), b = maybe(a[2], "b");
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) throw PythonError{};
    int N, D;
    long long step;
    rows(x, "layer_norm_fwd", N, D, step);
    const int dt = dtype_code(x, "x");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(w, {D}, dev, "w");
    check(b, {D}, dev, "b");
    at::Tensor y = output(maybe(a[4], "y"), x.sizes(), x.scalar_type(), dev, "y");
    Maybe mean, rstd;
    if (a[7] == Py_True) {
        const at::IntArrayRef shape = x.sizes().slice(0, x.dim() - 1);
        mean = output(maybe(a[5], "mean"), shape, at::kFloat, dev, "mean");
        rstd = output(maybe(a[6], "rstd"), shape, at::kFloat, dev, "rstd");
    }
    done(ttm_layer_norm_fwd(N, D, dt, x.data_ptr(), step, fptr(w), fptr(b), (float)eps, y.data_ptr(),
                            fptr(mean), fptr(rstd), current_stream(dev)),
         "ttm_layer_norm_fwd");
    return tuple({y, mean, rstd});
}

// (dy, x, mean, rstd, w, want_dw, want_db, dx, dw, db, workspace) -> (dx, dw, db)
PyObject* layer_norm_bwd(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &mean = tensor(a[2], "mean"),
                     &rstd = tensor(a[3], "rstd");
    const Maybe w = maybe(a[4], "w");
    int N, D, n2, d2;
    long long step, dstep;
    rows(x, "layer_norm_bwd", N, D, step);
    const int dt = dtype_code(x, "x");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    if (dy.sizes() != x.sizes() || dy.scalar_type() != x.scalar_type() || dy.device() != dev)
        bad("layer_norm_bwd: dy must have the shape and dtype of x");
    rows(dy, "layer_norm_bwd", n2, d2, dstep);
    const at::IntArrayRef shape = x.sizes().slice(0, x.dim() - 1);
    check(mean, shape, at::kFloat, dev, "mean");
    check(rstd, shape, at::kFloat, dev, "rstd");
    check(w, {D}, dev, "w");
    at::Tensor dx = output(maybe(a[7], "dx"), x.sizes(), x.scalar_type(), dev, "dx");
    Maybe dw, db;
    if (a[5] == Py_True) dw = output(maybe(a[8], "dw"), {D}, at::kFloat, dev, "dw");
    if (a[6] == Py_True) db = output(maybe(a[9], "db"), {D}, at::kFloat, dev, "db");
    const Maybe ws =
        scratch(maybe(a[10], "workspace"), dw || db ? ttm_layer_norm_bwd_workspace_size(N, D) : 0, dev);
    done(ttm_layer_norm_bwd(N, D, dt, dy.data_ptr(), dstep, x.data_ptr(), step, fptr(w),
                            static_cast<float*>(mean.data_ptr()), static_cast<float*>(rstd.data_ptr()),
                            dx.data_ptr(), fptr(dw), fptr(db), ptr(ws), bytes(ws), current_stream(dev)),
         "ttm_layer_norm_bwd");
    return tuple({dx, dw, db});
}

// (G, coeffs: bytes of fp32 triples, eps, out, workspace) -> out
PyObject* orthogonalize(PyObject* const* a) {
    const at::Tensor& G = tensor(a[0], "G");
    char* c;
    Py_ssize_t n;
    if (PyBytes_AsStringAndSize(a[1], &c, &n) < 0) throw PythonError{};
    const double eps = PyFloat_AsDouble(a[2]);
    if (PyErr_Occurred()) throw PythonError{};
    const int dt = dtype_code(G, "G");
    if (G.dim() < 2 || !G.is_contiguous() || !G.is_cuda())
        bad("orthogonalize: expected a contiguous CUDA tensor [..., m, n]");
    const at::Device dev = G.device();
    const c10::cuda::CUDAGuard guard(dev);
    int64_t batch = 1;
    for (int64_t k = 0; k + 2 < G.dim(); ++k) batch *= G.size(k);
    const int b = narrow(batch, "G"), m = narrow(G.size(-2), "G"), w = narrow(G.size(-1), "G");
    at::Tensor out = output(maybe(a[3], "out"), G.sizes(), at::kBFloat16, dev, "out");
    const Maybe ws = scratch(maybe(a[4], "workspace"), ttm_orthogonalize_workspace_size(b, m, w), dev);
    done(ttm_orthogonalize(b, m, w, dt, G.data_ptr(), reinterpret_cast<const float*>(c), (int)(n / 12),
                           (float)eps, out.data_ptr(), ptr(ws), bytes(ws), current_stream(dev)),
         "ttm_orthogonalize");
    return wrap(out);
}

// No C++ exception leaves the module.
template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Failure& f) {
        PyObject* e = PyObject_CallFunction(g_error, "is", f.code, f.what.c_str());
        if (e) {
            PyErr_SetObject(g_error, e);
            Py_DECREF(e);
        }
    } catch (const WrongType& t) {
        PyErr_SetString(PyExc_TypeError, t.what.c_str());
    } catch (const PythonError&) {
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* type = nullptr;
        if (PyObject* torch = PyImport_ImportModule("torch")) {
            type = PyObject_GetAttrString(torch, "OutOfMemoryError");
            Py_DECREF(torch);
        }
        PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
        Py_XDECREF(type);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
    Py_XDECREF(g_error);
    Py_INCREF(type);
    g_error = type;
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, kArgs>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef g_methods[] = {method<glr_fwd, 6>("glr_fwd"),
                           method<glr_bwd, 10>("glr_bwd"),
                           method<glr_step, 4>("glr_step"),
                           method<layer_norm_fwd, 8>("layer_norm_fwd"),
                           method<layer_norm_bwd, 11>("layer_norm_bwd"),
                           method<orthogonalize, 5>("orthogonalize"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "ttm_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ttm_torch(void) { return PyModule_Create(&g_module); }
