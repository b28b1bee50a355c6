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

// x [..., T, C] with taps w [C, K]: sizes, strides and the shape of its state.
struct Conv {
    int N, T, C, K, dtype;
    long long xs, xt;
    std::vector<int64_t> state;
};

Conv conv_shapes(const at::Tensor& x, const at::Tensor& w, const Maybe& b, const char* what) {
    Conv r;
    const int64_t lead = x.dim() - 2;
    if (lead < 0) bad(std::string(what) + ": expected [..., T, C]");
    const int64_t C = x.size(lead + 1);
    r.dtype = dtype_code(x, what);
    if ((C > 1 && x.stride(lead + 1) != 1) || !x.is_cuda())
        bad(std::string(what) + ": expected a CUDA tensor with contiguous channels");
    if (w.dim() != 2) bad(std::string(what) + ": w must be [C, K]");
    const int64_t K = w.size(1);
    check(w, {C, K}, at::kFloat, x.device(), "w");
    check(b, {C}, x.device(), "b");
    int64_t N = 1;
    for (int64_t k = 0; k < lead; ++k) N *= x.size(k);
    r.N = narrow(N, what);
    r.T = narrow(x.size(lead), what);
    r.C = narrow(C, what);
    r.K = narrow(K, what);
    strides(x, lead, C, what, r.xs, r.xt);
    r.state.assign(x.sizes().begin(), x.sizes().begin() + lead);
    r.state.push_back(K - 1);
    r.state.push_back(C);
    return r;
}

void check_state(const Maybe& t, const Conv& c, const at::Tensor& x, const char* what) {
    if (t) check(*t, c.state, x.scalar_type(), x.device(), what);
}

// Document numbers [..., T] and the elements between sequences.
const int* documents(const Maybe& doc, const at::Tensor& x, long long& seq) {
    seq = 0;
    if (!doc) return nullptr;
    const int64_t lead = x.dim() - 2;
    if (doc->scalar_type() != at::kInt || doc->sizes() != x.sizes().slice(0, lead + 1) || doc->device() != x.device() ||
        (x.size(lead) > 1 && doc->stride(lead) != 1))
        bad("doc must be int32, of the shape of x without its last axis, tokens contiguous, on the call's device");
    seq = one_stride(*doc, lead, "doc").value_or(x.size(lead));
    return static_cast<const int*>(doc->data_ptr());
}

// (x, w, b, state0, doc, silu, want_state, y, state) -> (y, state)
PyObject* causal_conv_fwd(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
    const Maybe b = maybe(a[2], "b"), s0 = maybe(a[3], "state0"), doc = maybe(a[4], "doc");
    const Conv c = conv_shapes(x, w, b, "causal_conv_fwd");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check_state(s0, c, x, "state0");
    long long doc_seq;
    const int* ids = documents(doc, x, doc_seq);
    at::Tensor y = output(maybe(a[7], "y"), x.sizes(), x.scalar_type(), dev, "y");
    Maybe state;
    if (a[6] == Py_True) state = output(maybe(a[8], "state"), c.state, x.scalar_type(), dev, "state");
    done(ttm_causal_conv_fwd(c.N, c.T, c.C, c.K, c.dtype, a[5] == Py_True, x.data_ptr(), c.xs, c.xt,
                             static_cast<float*>(w.data_ptr()), fptr(b), ptr(s0), ids, doc_seq, y.data_ptr(), ptr(state),
                             current_stream(dev)),
         "ttm_causal_conv_fwd");
    return tuple({y, state});
}

// (dy, x, w, b, state0, doc, silu, dstate, want_dw, dx, dw, db, dstate0, workspace) -> (dx, dw, db, dstate0)
PyObject* causal_conv_bwd(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &w = tensor(a[2], "w");
    const Maybe b = maybe(a[3], "b"), s0 = maybe(a[4], "state0"), doc = maybe(a[5], "doc"), ds = maybe(a[7], "dstate");
    const Conv c = conv_shapes(x, w, b, "causal_conv_bwd");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check_state(s0, c, x, "state0");
    check_state(ds, c, x, "dstate");
    if (dy.sizes() != x.sizes() || dy.scalar_type() != x.scalar_type() || dy.device() != dev ||
        (c.C > 1 && dy.stride(-1) != 1))
        bad("causal_conv_bwd: dy must have the shape, dtype and channel order of x");
    long long doc_seq, ys, yt;
    const int* ids = documents(doc, x, doc_seq);
    strides(dy, x.dim() - 2, c.C, "causal_conv_bwd", ys, yt);
    const bool want = a[8] == Py_True;
    at::Tensor dx = output(maybe(a[9], "dx"), x.sizes(), x.scalar_type(), dev, "dx");
    Maybe dw, db, d0;
    if (want) dw = output(maybe(a[10], "dw"), w.sizes(), at::kFloat, dev, "dw");
    if (want && b) db = output(maybe(a[11], "db"), b->sizes(), at::kFloat, dev, "db");
    if (s0) d0 = output(maybe(a[12], "dstate0"), c.state, x.scalar_type(), dev, "dstate0");
    const Maybe ws = scratch(maybe(a[13], "workspace"), want ? ttm_causal_conv_bwd_workspace_size(c.C, c.K) : 0, dev);
    done(ttm_causal_conv_bwd(c.N, c.T, c.C, c.K, c.dtype, a[6] == Py_True, dy.data_ptr(), ys, yt, x.data_ptr(), c.xs,
                             c.xt, static_cast<float*>(w.data_ptr()), fptr(b), ptr(s0), ids, doc_seq, ptr(ds),
                             dx.data_ptr(), fptr(dw), fptr(db), ptr(d0), ptr(ws), bytes(ws), current_stream(dev)),
         "ttm_causal_conv_bwd");
    return tuple({dx, dw, db, d0});
}

// (x, w, state, b, silu, y) -> y
PyObject* causal_conv_step(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &state = tensor(a[2], "state");
    const Maybe b = maybe(a[3], "b");
    const Conv c = conv_shapes(x, w, b, "causal_conv_step");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(state, c.state, x.scalar_type(), dev, "state");
    at::Tensor y = output(maybe(a[5], "y"), x.sizes(), x.scalar_type(), dev, "y");
    done(ttm_causal_conv_step(c.N, c.T, c.C, c.K, c.dtype, a[4] == Py_True, x.data_ptr(), c.xs, c.xt,
                              static_cast<float*>(w.data_ptr()), fptr(b), state.data_ptr(), y.data_ptr(),
                              current_stream(dev)),
         "ttm_causal_conv_step");
    return wrap(y);
}

// x [..., D], W_in [D, 2F], W_out [F, D], all bf16 on one device.
struct Ffn {
    int N, D, F, act;
    long long step;
    std::vector<int64_t> wide;          // [..., 2F]
};

Ffn ffn_shapes(const at::Tensor& x, const at::Tensor& W_in, const at::Tensor& W_out, PyObject* act, const char* what) {
    Ffn r;
    if (x.scalar_type() != at::kBFloat16) throw WrongType{std::string(what) + ": tensors must be bfloat16"};
    rows(x, what, r.N, r.D, r.step);
    if (W_in.dim() != 2 || W_in.size(1) % 2) bad(std::string(what) + ": W_in must be [D, 2F]");
    const int64_t F = W_in.size(1) / 2;
    r.F = narrow(F, what);
    check(W_in, {r.D, 2 * F}, at::kBFloat16, x.device(), "W_in");
    check(W_out, {F, r.D}, at::kBFloat16, x.device(), "W_out");
    r.act = (int)PyLong_AsLong(act);
    if (PyErr_Occurred()) throw PythonError{};
    r.wide.assign(x.sizes().begin(), x.sizes().end() - 1);
    r.wide.push_back(2 * F);
    return r;
}

// Elements between the rows of a tensor that has the shape of x.
long long rows_like(const at::Tensor& t, const at::Tensor& x, const char* what) {
    if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != x.device())
        bad(std::string(what) + " must have the shape and dtype of x and be on its device");
    int n, d;
    long long step;
    rows(t, what, n, d, step);
    return step;
}

// (x, W_in, W_out, act, residual, want_gu, y, gu, workspace) -> (y, gu)
PyObject* gated_ffn_fwd(PyObject* const* a) {
    const at::Tensor &x = tensor(a[0], "x"), &W_in = tensor(a[1], "W_in"), &W_out = tensor(a[2], "W_out");
    const Ffn f = ffn_shapes(x, W_in, W_out, a[3], "gated_ffn_fwd");
    const Maybe res = maybe(a[4], "residual");
    const long long res_step = res ? rows_like(*res, x, "residual") : 0;
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor y = output(maybe(a[6], "y"), x.sizes(), at::kBFloat16, dev, "y");
    Maybe gu;
    if (a[5] == Py_True) gu = output(maybe(a[7], "gu"), f.wide, at::kBFloat16, dev, "gu");
    const Maybe ws = scratch(maybe(a[8], "workspace"), ttm_gated_ffn_workspace_size(f.N, f.D, f.F, 0), dev);
    done(ttm_gated_ffn_fwd(f.N, f.D, f.F, f.act, x.data_ptr(), f.step, W_in.data_ptr(), W_out.data_ptr(), ptr(res),
                           res_step, y.data_ptr(), ptr(gu), ptr(ws), bytes(ws), current_stream(dev)),
         "ttm_gated_ffn_fwd");
    return tuple({y, gu});
}

// (dy, x, gu, W_in, W_out, act, want_dx, want_dw, dx, dW_in, dW_out, workspace) -> (dx, dW_in, dW_out)
PyObject* gated_ffn_bwd(PyObject* const* a) {
    const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x"), &gu = tensor(a[2], "gu"),
                     &W_in = tensor(a[3], "W_in"), &W_out = tensor(a[4], "W_out");
    const Ffn f = ffn_shapes(x, W_in, W_out, a[5], "gated_ffn_bwd");
    const long long dy_step = rows_like(dy, x, "dy");
    const at::Device dev = x.device();
    const c10::cuda::CUDAGuard guard(dev);
    check(gu, f.wide, at::kBFloat16, dev, "gu");
    Maybe dx, dW_in, dW_out;
    if (a[6] == Py_True) dx = output(maybe(a[8], "dx"), x.sizes(), at::kBFloat16, dev, "dx");
    if (a[7] == Py_True) {
        dW_in = output(maybe(a[9], "dW_in"), W_in.sizes(), at::kBFloat16, dev, "dW_in");
        dW_out = output(maybe(a[10], "dW_out"), W_out.sizes(), at::kBFloat16, dev, "dW_out");
    }
    const Maybe ws = scratch(maybe(a[11], "workspace"), ttm_gated_ffn_workspace_size(f.N, f.D, f.F, 1), dev);
    done(ttm_gated_ffn_bwd(f.N, f.D, f.F, f.act, dy.data_ptr(), dy_step, x.data_ptr(), f.step, gu.data_ptr(),
                           W_in.data_ptr(), W_out.data_ptr(), ptr(dx), ptr(dW_in), ptr(dW_out), ptr(ws), bytes(ws),
                           current_stream(dev)),
         "ttm_gated_ffn_bwd");
    return tuple({dx, dW_in, dW_out});
}

// A list or tuple, held while it is read.
struct Items {
    PyObject* seq;
    Items(PyObject* o, const char* what) : seq(PySequence_Fast(o, "")) {
        if (!seq) {
            PyErr_Clear();
            bad(std::string(what) + " must be a list of tensors");
        }
    }
    ~Items() { Py_XDECREF(seq); }
    Items(const Items&) = delete;
    Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(seq); }
    PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(seq, i); }
};

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}

const float* scalar(const Maybe& t, const at::Device& dev, const char* what) {
    if (!t) return nullptr;
    if (t->numel() != 1 || t->scalar_type() != at::kFloat || t->device() != dev)
        bad(std::string(what) + " must be a float32 tensor of one value on the call's device");
    return static_cast<const float*>(t->data_ptr());
}

// Whole blocks of 256 moments; 8 bits when there are scales.
int64_t moments_of(const at::Tensor& m, const at::Tensor& v, const Maybe& ms, const Maybe& vs, const at::Device& dev) {
    const at::ScalarType type = ms ? at::kFloat8_e4m3fn : at::kFloat;
    const int64_t n = m.numel();
    if (ms.has_value() != vs.has_value() || n % 256) bad("state: not one of adamw_state");
    check(m, {n}, type, dev, "state m");
    check(v, {n}, type, dev, "state v");
    check(ms, {n / 256}, dev, "state m_scale");
    check(vs, {n / 256}, dev, "state v_scale");
    return n / 256;
}

// (params, grads, copies, m, v, m_scale, v_scale, step, lr, b1, b2, eps, weight_decay, grad_scale) -> None
PyObject* adamw_step(PyObject* const* a) {
    const Items params(a[0], "params"), grads(a[1], "grads");
    std::optional<Items> copies;
    if (a[2] != Py_None) copies.emplace(a[2], "copies");
    const Py_ssize_t n = params.size();
    if (grads.size() != n || (copies && copies->size() != n)) bad("adamw_step: as many grads and copies as params");
    const at::Tensor &m = tensor(a[3], "m"), &v = tensor(a[4], "v"), &step = tensor(a[7], "step");
    const Maybe ms = maybe(a[5], "m_scale"), vs = maybe(a[6], "v_scale"), gs = maybe(a[13], "grad_scale");
    if (!m.is_cuda()) bad("adamw_step: expected CUDA tensors");
    const at::Device dev = m.device();
    const int64_t blocks = moments_of(m, v, ms, vs, dev);
    check(step, {2}, at::kInt, dev, "state step");
    const float* scale = scalar(gs, dev, "grad_scale");
    Maybe lr_tensor;
    double lr = 0;
    if (THPVariable_Check(a[8]) && THPVariable_Unpack(a[8]).is_cuda()) lr_tensor = THPVariable_Unpack(a[8]);
    else lr = number(a[8]);
    const float* lr_at = scalar(lr_tensor, dev, "lr");
    std::vector<ttm_adamw_tensor> list((size_t)n);
    int64_t need = 0;
    for (Py_ssize_t i = 0; i < n; ++i) {
        const at::Tensor& p = tensor(params.at(i), "param");
        ttm_adamw_tensor& t = list[(size_t)i];
        t.n = p.numel();
        t.param_dtype = t.grad_dtype = dtype_code(p, "param");
        need += (t.n + 255) / 256;
        if (!p.is_contiguous() || p.device() != dev) bad("params must be contiguous and on the device of the state");
        t.param = p.data_ptr();
        t.grad = nullptr;
        t.copy = nullptr;
        if (grads.at(i) == Py_None) continue;
        const at::Tensor& g = tensor(grads.at(i), "grad");
        if (g.sizes() != p.sizes() || !g.is_contiguous() || g.device() != dev)
            bad("grads must be contiguous, of their parameter's shape and on its device");
        t.grad = g.data_ptr();
        t.grad_dtype = dtype_code(g, "grad");
        if (copies && copies->at(i) != Py_None) {
            const at::Tensor& c = tensor(copies->at(i), "copy");
            check(c, p.sizes(), at::kBFloat16, dev, "copies");
            t.copy = c.data_ptr();
        }
    }
    if (need != blocks) bad("adamw_step: the state is of other parameters");
    const c10::cuda::CUDAGuard guard(dev);
    done(ttm_adamw_step((int)n, list.data(), ms ? 8 : 32, m.data_ptr(), v.data_ptr(), fptr(ms), fptr(vs),
                        static_cast<int*>(step.data_ptr()), lr, lr_at, number(a[9]), number(a[10]), number(a[11]),
                        number(a[12]), scale, current_stream(dev)),
         "ttm_adamw_step");
    // autograd sees the parameters written in place
    auto written = [](PyObject* o) {
        const at::Tensor& t = THPVariable_Unpack(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    };
    for (Py_ssize_t i = 0; i < n; ++i) {
        if (!list[(size_t)i].grad) continue;
        written(params.at(i));
        if (list[(size_t)i].copy) written(copies->at(i));
    }
    Py_RETURN_NONE;
}

// (m, v, m_scale, v_scale) -> (m, v) in fp32
PyObject* adamw_moments(PyObject* const* a) {
    const at::Tensor &m = tensor(a[0], "m"), &v = tensor(a[1], "v");
    const Maybe ms = maybe(a[2], "m_scale"), vs = maybe(a[3], "v_scale");
    if (!m.is_cuda() || !ms) bad("adamw_moments: expected CUDA tensors in 8 bits with their scales");
    const at::Device dev = m.device();
    const c10::cuda::CUDAGuard guard(dev);
    const int64_t blocks = moments_of(m, v, ms, vs, dev);
    at::Tensor mo = make({blocks * 256}, at::kFloat, dev), vo = make({blocks * 256}, at::kFloat, dev);
    done(ttm_adamw_moments(blocks, m.data_ptr(), v.data_ptr(), fptr(ms), fptr(vs), static_cast<float*>(mo.data_ptr()),
                           static_cast<float*>(vo.data_ptr()), current_stream(dev)),
         "ttm_adamw_moments");
    return tuple({mo, vo});
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
                           method<causal_conv_fwd, 9>("causal_conv_fwd"),
                           method<causal_conv_bwd, 14>("causal_conv_bwd"),
                           method<causal_conv_step, 6>("causal_conv_step"),
                           method<gated_ffn_fwd, 9>("gated_ffn_fwd"),
                           method<gated_ffn_bwd, 12>("gated_ffn_bwd"),
                           method<adamw_step, 14>("adamw_step"),
                           method<adamw_moments, 4>("adamw_moments"),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "ttm_torch", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ttm_torch(void) { return PyModule_Create(&g_module); }
