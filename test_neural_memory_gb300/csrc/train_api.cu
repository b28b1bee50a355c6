// C ABI of the operators around the memory scan: host-side argument
// validation and launch.  Declarations and contract are in include/ttm.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ttm.h"
#include "train_ops.h"

namespace {

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

// No output may overlap an input or another output.
template <int NI, int NO>
bool outputs_clear(const Span (&ins)[NI], const Span (&outs)[NO]) {
    for (int i = 0; i < NO; ++i) {
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return false;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return false;
    }
    return true;
}

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

template <int N>
bool all_aligned16(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return false;
    return true;
}

bool dtype_ok(int dtype) { return dtype == TTM_F32 || dtype == TTM_BF16; }

// Bytes from the first to one past the last element of [N][T][D] values of es bytes
// with the given strides; 0 for an empty view, and `ok` is cleared when two rows
// would overlap or an offset leaves 62 bits.
size_t view_bytes(long long N, long long T, long long D, long long seq, long long tok, size_t es,
                  bool& ok) {
    if (N == 0 || T == 0) return 0;
    if ((T > 1 && tok < D) || (N > 1 && seq < D)) ok = false;
    if (seq < 0 || tok < 0) ok = false;
    const double last = double(N - 1) * double(seq) + double(T - 1) * double(tok) + double(D);
    if (last * double(es) > 4e18) ok = false;
    return ok ? (size_t)((N - 1) * seq + (T - 1) * tok + D) * es : 0;
}

// A tile, 4096 tokens at most, may start at any token and is counted in 31 bits.
constexpr int kMostTokens = 0x7fffffff - 8192;

// What the three recurrence calls share.  `x` is the strided input (the forward's x or
// the gradient's dh).
int glr_common(ttm::GlrArgs& a, int N, int T, int D, int dtype, int gate, const void* x,
               long long x_seq, long long x_tok, const void* g, long long g_seq, long long g_tok,
               Span& sx, Span& sg) {
    if (N < 1 || T < 0 || D < 1 || !dtype_ok(dtype)) return TTM_ERR_INVALID_ARG;
    if (gate != TTM_GATE_CHANNEL && gate != TTM_GATE_TOKEN) return TTM_ERR_INVALID_ARG;
    if (T > 0 && (!x || !g)) return TTM_ERR_INVALID_ARG;
    const size_t es = dtype == TTM_BF16 ? 2 : 4, gs = gate == TTM_GATE_TOKEN ? 4 : es;
    if (!aligned(x, es) || !aligned(g, gs)) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    sx = {x, view_bytes(N, T, D, x_seq, x_tok, es, ok)};
    sg = {g, view_bytes(N, T, gate == TTM_GATE_TOKEN ? 1 : D, g_seq, g_tok, gs, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    if ((long long)N * D > (1LL << 31) - 1 || T > kMostTokens) return TTM_ERR_UNSUPPORTED;
    a.N = N; a.T = T; a.D = D;
    a.bf16 = dtype == TTM_BF16;
    a.gate_token = gate == TTM_GATE_TOKEN;
    a.x = x; a.x_seq = x_seq; a.x_tok = x_tok;
    a.g = g; a.g_seq = g_seq; a.g_tok = g_tok;
    return TTM_OK;
}

int glr_run(ttm::GlrArgs& a, int backward, void* workspace, size_t workspace_bytes, void* stream) {
    const size_t need = ttm::glr_workspace_bytes(a, backward);
    if (need && (!workspace || workspace_bytes < need)) return TTM_ERR_INVALID_ARG;
    a.workspace = workspace;
    a.status = ttm::api_status_ptr();
    if (!a.status) return TTM_ERR_CUDA;
    a.wait_cycles = ttm::api_wait_cycles();
    a.debug_stall = (unsigned)ttm::api_take_stall();
    int launches = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = backward ? ttm::glr_bwd_launch(a, s, &launches)
                                   : ttm::glr_fwd_launch(a, s, &launches);
    if (e != cudaSuccess) return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

}  // namespace

extern "C" {

size_t ttm_glr_workspace_size(int N, int T, int D, int dtype, int gate, int backward) {
    ttm::GlrArgs a{};
    Span sx, sg;
    if (N < 1 || T < 0 || D < 1 || !dtype_ok(dtype) ||
        (gate != TTM_GATE_CHANNEL && gate != TTM_GATE_TOKEN) ||
        (long long)N * D > (1LL << 31) - 1 || T > kMostTokens)
        return 0;
    a.N = N; a.T = T; a.D = D;
    a.bf16 = dtype == TTM_BF16;
    a.gate_token = gate == TTM_GATE_TOKEN;
    return ttm::glr_workspace_bytes(a, backward != 0);
}

int ttm_glr_fwd(int N, int T, int D, int dtype, int gate, const void* x, long long x_seq,
                long long x_tok, const void* g, long long g_seq, long long g_tok, const float* h0,
                void* h, float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
    ttm::GlrArgs a{};
    Span sx, sg;
    const int r = glr_common(a, N, T, D, dtype, gate, x, x_seq, x_tok, g, g_seq, g_tok, sx, sg);
    if (r != TTM_OK) return r;
    if ((T > 0 && !h) || !h_last) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<4>({h0, h, h_last, workspace})) return TTM_ERR_INVALID_ARG;
    const size_t es = a.bf16 ? 2 : 4, nd = (size_t)N * D;
    const Span swk{workspace, workspace ? workspace_bytes : 0};
    const Span ins[] = {sx, sg, {h0, nd * 4}}, outs[] = {{h, nd * T * es}, {h_last, nd * 4}, swk};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.h0 = h0; a.h = h; a.h_last = h_last;
    return glr_run(a, 0, workspace, workspace_bytes, stream);
}

int ttm_glr_bwd(int N, int T, int D, int dtype, int gate, const void* g, long long g_seq,
                long long g_tok, const void* h, const float* h0, const void* dh, long long dh_seq,
                long long dh_tok, const float* dh_last, void* dx, void* dg, float* dh0,
                void* workspace, size_t workspace_bytes, void* stream) {
    ttm::GlrArgs a{};
    Span sx, sg;
    const int r =
        glr_common(a, N, T, D, dtype, gate, dh, dh_seq, dh_tok, g, g_seq, g_tok, sx, sg);
    if (r != TTM_OK) return r;
    if (T > 0 && (!h || !dx || !dg)) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<7>({h, h0, dh_last, dx, dg, dh0, workspace})) return TTM_ERR_INVALID_ARG;
    const size_t es = a.bf16 ? 2 : 4, nd = (size_t)N * D;
    const Span swk{workspace, workspace ? workspace_bytes : 0};
    const Span ins[] = {sx, sg, {h, nd * T * es}, {h0, nd * 4}, {dh_last, nd * 4}};
    const Span outs[] = {{dx, nd * T * es},
                         {dg, a.gate_token ? (size_t)N * T * 4 : nd * T * es},
                         {dh0, nd * 4},
                         swk};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.h = const_cast<void*>(h);
    a.h0 = h0; a.dh_last = dh_last;
    a.dx = dx; a.dg = dg; a.dh0 = dh0;
    return glr_run(a, 1, workspace, workspace_bytes, stream);
}

int ttm_glr_step(int N, int n, int D, int dtype, int gate, const void* x, long long x_seq,
                 long long x_tok, const void* g, long long g_seq, long long g_tok, float* state,
                 void* h, void* stream) {
    ttm::GlrArgs a{};
    Span sx, sg;
    if (n < 1) return TTM_ERR_INVALID_ARG;
    const int r = glr_common(a, N, n, D, dtype, gate, x, x_seq, x_tok, g, g_seq, g_tok, sx, sg);
    if (r != TTM_OK) return r;
    if (!state || !h || !all_aligned16<2>({state, h})) return TTM_ERR_INVALID_ARG;
    const size_t es = a.bf16 ? 2 : 4, nd = (size_t)N * D;
    const Span ins[] = {sx, sg}, outs[] = {{state, nd * 4}, {h, nd * n * es}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.h = h; a.h_last = state;
    if (ttm::glr_step_launch(a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return TTM_ERR_CUDA;
    ttm::api_note_launches(1);
    return TTM_OK;
}

int ttm_layer_norm_fwd(int N, int D, int dtype, const void* x, long long x_row, const float* w,
                       const float* b, float eps, void* y, float* mean, float* rstd,
                       void* stream) {
    if (N < 0 || D < 1 || !dtype_ok(dtype) || !(eps >= 0.f)) return TTM_ERR_INVALID_ARG;
    if (N > 0 && (!x || !y)) return TTM_ERR_INVALID_ARG;
    const size_t es = dtype == TTM_BF16 ? 2 : 4;
    if (!aligned(x, es) || !all_aligned16<5>({w, b, y, mean, rstd})) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    const Span sx{x, view_bytes(1, N, D, 0, x_row, es, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    const Span ins[] = {sx, {w, (size_t)D * 4}, {b, (size_t)D * 4}};
    const Span outs[] = {{y, (size_t)N * D * es}, {mean, (size_t)N * 4}, {rstd, (size_t)N * 4}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    if (N == 0) return TTM_OK;
    ttm::LayerNormArgs a{};
    a.N = N; a.D = D;
    a.bf16 = dtype == TTM_BF16;
    a.x = x; a.x_row = x_row; a.w = w; a.b = b; a.eps = eps;
    a.y = y; a.mean = mean; a.rstd = rstd;
    if (ttm::layer_norm_fwd_launch(a, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return TTM_ERR_CUDA;
    ttm::api_note_launches(1);
    return TTM_OK;
}

size_t ttm_layer_norm_bwd_workspace_size(int N, int D) {
    return N < 0 || D < 1 ? 0 : ttm::layer_norm_bwd_workspace_bytes(N, D);
}

int ttm_layer_norm_bwd(int N, int D, int dtype, const void* dy, long long dy_row, const void* x,
                       long long x_row, const float* w, const float* mean, const float* rstd,
                       void* dx, float* dw, float* db, void* workspace, size_t workspace_bytes,
                       void* stream) {
    if (N < 0 || D < 1 || !dtype_ok(dtype)) return TTM_ERR_INVALID_ARG;
    if (N > 0 && (!dy || !x || !mean || !rstd || !dx)) return TTM_ERR_INVALID_ARG;
    const size_t es = dtype == TTM_BF16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(dy, es)) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<7>({w, mean, rstd, dx, dw, db, workspace})) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    const Span sx{x, view_bytes(1, N, D, 0, x_row, es, ok)};
    const Span sdy{dy, view_bytes(1, N, D, 0, dy_row, es, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    const size_t need = ttm::layer_norm_bwd_workspace_bytes(N, D);
    if ((dw || db) && need && (!workspace || workspace_bytes < need)) return TTM_ERR_INVALID_ARG;
    const Span ins[] = {sx, sdy, {w, (size_t)D * 4}, {mean, (size_t)N * 4}, {rstd, (size_t)N * 4}};
    const Span outs[] = {{dx, (size_t)N * D * es},
                         {dw, (size_t)D * 4},
                         {db, (size_t)D * 4},
                         {workspace, workspace ? workspace_bytes : 0}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    ttm::LayerNormArgs a{};
    a.N = N; a.D = D;
    a.bf16 = dtype == TTM_BF16;
    a.x = x; a.x_row = x_row; a.w = w;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dy = dy; a.dy_row = dy_row;
    a.dx = dx; a.dw = dw; a.db = db;
    a.partial = static_cast<float*>(workspace);
    int launches = 0;
    if (ttm::layer_norm_bwd_launch(a, static_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
        return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

size_t ttm_orthogonalize_workspace_size(int batch, int m, int n) {
    return batch < 1 || m < 1 || n < 1 || m > TTM_ORTHO_MAX_DIM || n > TTM_ORTHO_MAX_DIM ||
                   batch > 65535
               ? 0
               : ttm::ortho_workspace_bytes(batch, m, n);
}

int ttm_orthogonalize(int batch, int m, int n, int dtype, const void* G, const float* coeffs,
                      int steps, float eps, void* out, void* workspace, size_t workspace_bytes,
                      void* stream) {
    if (batch < 1 || m < 1 || n < 1 || !dtype_ok(dtype) || !G || !out) return TTM_ERR_INVALID_ARG;
    if (steps < 0 || (steps > 0 && !coeffs) || !(eps > 0.f)) return TTM_ERR_INVALID_ARG;
    if (steps > ttm::kNsMaxSteps || m > TTM_ORTHO_MAX_DIM || n > TTM_ORTHO_MAX_DIM || batch > 65535)
        return TTM_ERR_UNSUPPORTED;
    if (!all_aligned16<3>({G, out, workspace})) return TTM_ERR_INVALID_ARG;
    const size_t es = dtype == TTM_BF16 ? 2 : 4, mn = (size_t)batch * m * n;
    const size_t need = ttm::ortho_workspace_bytes(batch, m, n);
    if (need && (!workspace || workspace_bytes < need)) return TTM_ERR_INVALID_ARG;
    const Span ins[] = {{G, mn * es}};
    const Span outs[] = {{out, mn * 2}, {workspace, workspace ? workspace_bytes : 0}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    ttm::OrthoArgs a{};
    a.batch = batch; a.m = m; a.n = n;
    a.bf16 = dtype == TTM_BF16;
    a.G = G; a.steps = steps; a.eps = eps; a.out = out; a.workspace = workspace;
    for (int i = 0; i < 3 * steps; ++i) {
        if (!std::isfinite(coeffs[i])) return TTM_ERR_INVALID_ARG;
        a.coeffs[i] = coeffs[i];
    }
    a.status = ttm::api_status_ptr();
    if (!a.status) return TTM_ERR_CUDA;
    a.wait_cycles = ttm::api_wait_cycles();
    a.debug_stall = ttm::api_take_stall();
    int launches = 0;
    if (ttm::ortho_launch(a, static_cast<cudaStream_t>(stream), &launches) != cudaSuccess)
        return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

}  // extern "C"
