// C ABI of the operators around the memory scan: host-side argument
// validation and launch.  Declarations and contract are in include/ttm.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

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

// What the three convolution calls share, but for the outputs.
int conv_common(ttm::ConvArgs& a, int N, int T, int C, int K, int dtype, int silu, const void* x, long long x_seq,
                long long x_tok, const float* w, const float* b, Span& sx) {
    if (N < 1 || T < 0 || C < 1 || K < 1 || !dtype_ok(dtype) || (silu != 0 && silu != 1)) return TTM_ERR_INVALID_ARG;
    if (!w || (T > 0 && !x)) return TTM_ERR_INVALID_ARG;
    const size_t es = dtype == TTM_BF16 ? 2 : 4;
    if (!aligned(x, es) || !aligned(w, 4) || !aligned(b, 4)) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    sx = {x, view_bytes(N, T, C, x_seq, x_tok, es, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    if ((long long)N * C > (1LL << 31) - 1 || T > kMostTokens || K > TTM_CONV_MAX_TAPS) return TTM_ERR_UNSUPPORTED;
    a.N = N; a.T = T; a.C = C; a.K = K;
    a.bf16 = dtype == TTM_BF16;
    a.silu = silu;
    a.x = x; a.x_seq = x_seq; a.x_tok = x_tok;
    a.w = w; a.b = b;
    return TTM_OK;
}

bool doc_ok(const ttm::ConvArgs& a, const int* doc, long long doc_seq, Span& sd) {
    // (only read: rows may overlap, as where one row serves every sequence)
    sd = {doc, 0};
    if (!doc) return true;
    if (!aligned(doc, 4) || (a.N > 1 && (doc_seq < 0 || double(a.N - 1) * double(doc_seq) > 1e18))) return false;
    sd.bytes = ((size_t)(a.N - 1) * (a.N > 1 ? doc_seq : 0) + a.T) * 4;
    return true;
}

// The distance to a next row says nothing where there is one row, but a tensor map takes it all the same.
long long row_step(int N, int D, long long step) { return N > 1 ? step : D; }

// Widths whose products count in 32 bits.
constexpr int kMostWidth = 1 << 24;

int ffn_common(ttm::FfnArgs& a, int N, int D, int F, int act, const void* x, long long x_row, const void* W_in,
               const void* W_out, Span& sx) {
    if (N < 0 || D < 8 || F < 8 || D % 8 || F % 8 || (act != TTM_ACT_SILU && act != TTM_ACT_GELU))
        return TTM_ERR_INVALID_ARG;
    if (!W_in || !W_out || (N > 0 && !x) || x_row % 8) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<3>({x, W_in, W_out})) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    sx = {x, view_bytes(1, N, D, 0, x_row, 2, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    if (D >= kMostWidth || F >= kMostWidth / 2 || N > kMostTokens) return TTM_ERR_UNSUPPORTED;
    a.N = N; a.D = D; a.F = F;
    a.gelu = act == TTM_ACT_GELU;
    a.x = x; a.x_row = row_step(N, D, x_row);
    a.W_in = W_in; a.W_out = W_out;
    return TTM_OK;
}

int ffn_run(ttm::FfnArgs& a, int backward, void* workspace, size_t workspace_bytes, void* stream) {
    const size_t need = ttm::ffn_workspace_bytes(a.N, a.D, a.F, backward);
    if (need && (!workspace || workspace_bytes < need)) return TTM_ERR_INVALID_ARG;
    a.workspace = workspace;
    a.status = ttm::api_status_ptr();
    if (!a.status) return TTM_ERR_CUDA;
    a.wait_cycles = ttm::api_wait_cycles();
    a.debug_stall = ttm::api_take_stall();
    int launches = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = backward ? ttm::ffn_bwd_launch(a, s, &launches) : ttm::ffn_fwd_launch(a, s, &launches);
    if (e != cudaSuccess) return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

struct Range {
    uintptr_t from, to;
    bool written;
};

template <typename F>
bool sorted_ranges_clash(size_t n, F range) {
    uintptr_t any = 0, written = 0;         // ends of the ranges so far
    for (size_t i = 0; i < n; ++i) {
        const Range x = range(i);
        if (x.from < written || (x.written && x.from < any)) return true;
        any = std::max(any, x.to);
        if (x.written) written = std::max(written, x.to);
    }
    return false;
}

// Whether a written range meets another one.  Sorted as one word each, the start (in 2 bytes, the least alignment) and the
// place: a list of a few hundred is a good part of a short call's time.
bool ranges_clash(const std::vector<Range>& r) {
    if (r.size() >= 65536) {
        std::vector<Range> by_start(r);
        std::sort(by_start.begin(), by_start.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
        return sorted_ranges_clash(by_start.size(), [&](size_t i) { return by_start[i]; });
    }
    std::vector<uint64_t> key(r.size());
    for (size_t i = 0; i < r.size(); ++i) key[i] = (uint64_t)(r[i].from >> 1) << 16 | i;
    if (!std::is_sorted(key.begin(), key.end())) std::sort(key.begin(), key.end());
    return sorted_ranges_clash(r.size(), [&](size_t i) { return r[key[i] & 0xffff]; });
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


int ttm_causal_conv_fwd(int N, int T, int C, int K, int dtype, int silu, const void* x, long long x_seq,
                        long long x_tok, const float* w, const float* b, const void* state0, const int* doc,
                        long long doc_seq, void* y, void* state, void* stream) {
    ttm::ConvArgs a{};
    Span sx, sd;
    const int r = conv_common(a, N, T, C, K, dtype, silu, x, x_seq, x_tok, w, b, sx);
    if (r != TTM_OK) return r;
    if (T > 0 && !y) return TTM_ERR_INVALID_ARG;
    if (!doc_ok(a, doc, doc_seq, sd) || !all_aligned16<3>({state0, y, state})) return TTM_ERR_INVALID_ARG;
    const size_t es = a.bf16 ? 2 : 4, nc = (size_t)N * C, st = nc * (K - 1) * es;
    const Span ins[] = {sx, sd, {w, (size_t)C * K * 4}, {b, (size_t)C * 4}, {state0, st}};
    const Span outs[] = {{y, nc * T * es}, {state, st}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.state0 = state0; a.doc = T > 0 ? doc : nullptr; a.doc_seq = doc_seq; a.y = y; a.state = state;
    int launches = 0;
    if (ttm::conv_fwd_launch(a, static_cast<cudaStream_t>(stream), &launches) != cudaSuccess) return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

size_t ttm_causal_conv_bwd_workspace_size(int C, int K) {
    if (C < 1 || K < 1 || K > TTM_CONV_MAX_TAPS) return 0;
    ttm::ConvArgs a{};
    a.C = C; a.K = K;
    return ttm::conv_bwd_workspace_bytes(a);
}

int ttm_causal_conv_bwd(int N, int T, int C, int K, int dtype, int silu, const void* dy, long long dy_seq,
                        long long dy_tok, const void* x, long long x_seq, long long x_tok, const float* w,
                        const float* b, const void* state0, const int* doc, long long doc_seq, const void* dstate,
                        void* dx, float* dw, float* db, void* dstate0, void* workspace, size_t workspace_bytes,
                        void* stream) {
    ttm::ConvArgs a{};
    Span sx, sd;
    const int r = conv_common(a, N, T, C, K, dtype, silu, x, x_seq, x_tok, w, b, sx);
    if (r != TTM_OK) return r;
    const size_t es = a.bf16 ? 2 : 4, nc = (size_t)N * C, st = nc * (K - 1) * es;
    if ((T > 0 && (!dy || !dx)) || !aligned(dy, es)) return TTM_ERR_INVALID_ARG;
    if (!doc_ok(a, doc, doc_seq, sd) || !all_aligned16<7>({state0, dstate, dx, dw, db, dstate0, workspace}))
        return TTM_ERR_INVALID_ARG;
    bool ok = true;
    const Span sdy{dy, view_bytes(N, T, C, dy_seq, dy_tok, es, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    const bool sums = dw || db;
    if (sums && (!workspace || workspace_bytes < ttm::conv_bwd_workspace_bytes(a))) return TTM_ERR_INVALID_ARG;
    const Span ins[] = {sx, sd, sdy, {w, (size_t)C * K * 4}, {b, (size_t)C * 4}, {state0, st}, {dstate, st}};
    const Span outs[] = {{dx, nc * T * es},
                         {dw, (size_t)C * K * 4},
                         {db, (size_t)C * 4},
                         {dstate0, st},
                         {workspace, workspace ? workspace_bytes : 0}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.state0 = state0; a.doc = T > 0 ? doc : nullptr; a.doc_seq = doc_seq;
    a.dy = dy; a.dy_seq = dy_seq; a.dy_tok = dy_tok;
    a.dstate = dstate; a.dx = dx; a.dw = dw; a.db = db; a.dstate0 = dstate0;
    a.partial = sums ? static_cast<float*>(workspace) : nullptr;
    int launches = 0;
    if (ttm::conv_bwd_launch(a, static_cast<cudaStream_t>(stream), &launches) != cudaSuccess) return TTM_ERR_CUDA;
    ttm::api_note_launches(launches);
    return TTM_OK;
}

int ttm_causal_conv_step(int N, int n, int C, int K, int dtype, int silu, const void* x, long long x_seq,
                         long long x_tok, const float* w, const float* b, void* state, void* y, void* stream) {
    ttm::ConvArgs a{};
    Span sx;
    if (n < 1) return TTM_ERR_INVALID_ARG;
    const int r = conv_common(a, N, n, C, K, dtype, silu, x, x_seq, x_tok, w, b, sx);
    if (r != TTM_OK) return r;
    if ((K > 1 && !state) || !y || !all_aligned16<2>({state, y})) return TTM_ERR_INVALID_ARG;
    const size_t es = a.bf16 ? 2 : 4, nc = (size_t)N * C;
    const Span ins[] = {sx, {w, (size_t)C * K * 4}, {b, (size_t)C * 4}};
    const Span outs[] = {{state, nc * (K - 1) * es}, {y, nc * n * es}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    a.state0 = a.state = state;
    a.y = y;
    if (ttm::conv_step_launch(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return TTM_ERR_CUDA;
    ttm::api_note_launches(1);
    return TTM_OK;
}

size_t ttm_gated_ffn_workspace_size(int N, int D, int F, int backward) {
    if (N < 1 || D < 8 || F < 8 || D % 8 || F % 8 || D >= kMostWidth || F >= kMostWidth / 2 || N > kMostTokens) return 0;
    return ttm::ffn_workspace_bytes(N, D, F, backward != 0);
}

int ttm_gated_ffn_fwd(int N, int D, int F, int act, const void* x, long long x_row, const void* W_in,
                      const void* W_out, const void* residual, long long residual_row, void* y, void* gu,
                      void* workspace, size_t workspace_bytes, void* stream) {
    ttm::FfnArgs a{};
    Span sx;
    const int r = ffn_common(a, N, D, F, act, x, x_row, W_in, W_out, sx);
    if (r != TTM_OK) return r;
    if ((N > 0 && !y) || !all_aligned16<4>({residual, y, gu, workspace})) return TTM_ERR_INVALID_ARG;
    bool ok = !residual || residual_row % 8 == 0;
    const Span sr{residual, residual ? view_bytes(1, N, D, 0, residual_row, 2, ok) : 0};
    if (!ok) return TTM_ERR_INVALID_ARG;
    const size_t df = (size_t)D * F, n = N;
    const Span ins[] = {sx, sr, {W_in, df * 4}, {W_out, df * 2}};
    const Span outs[] = {{y, n * D * 2}, {gu, n * F * 4}, {workspace, workspace ? workspace_bytes : 0}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    if (N == 0) return TTM_OK;
    a.residual = residual; a.residual_row = residual_row;
    a.y = y; a.gu = gu;
    return ffn_run(a, 0, workspace, workspace_bytes, stream);
}

int ttm_gated_ffn_bwd(int N, int D, int F, int act, const void* dy, long long dy_row, const void* x, long long x_row,
                      const void* gu, const void* W_in, const void* W_out, void* dx, void* dW_in, void* dW_out,
                      void* workspace, size_t workspace_bytes, void* stream) {
    ttm::FfnArgs a{};
    Span sx;
    const int r = ffn_common(a, N, D, F, act, x, x_row, W_in, W_out, sx);
    if (r != TTM_OK) return r;
    if ((N > 0 && (!dy || !gu)) || dy_row % 8) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<6>({dy, gu, dx, dW_in, dW_out, workspace})) return TTM_ERR_INVALID_ARG;
    bool ok = true;
    const Span sdy{dy, view_bytes(1, N, D, 0, dy_row, 2, ok)};
    if (!ok) return TTM_ERR_INVALID_ARG;
    const size_t df = (size_t)D * F, n = N;
    const Span ins[] = {sx, sdy, {gu, n * F * 4}, {W_in, df * 4}, {W_out, df * 2}};
    const Span outs[] = {{dx, n * D * 2}, {dW_in, df * 4}, {dW_out, df * 2}, {workspace, workspace ? workspace_bytes : 0}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    if (N == 0) {
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (dW_in && cudaMemsetAsync(dW_in, 0, df * 4, s) != cudaSuccess) return TTM_ERR_CUDA;
        if (dW_out && cudaMemsetAsync(dW_out, 0, df * 2, s) != cudaSuccess) return TTM_ERR_CUDA;
        return TTM_OK;
    }
    a.dy = dy; a.dy_row = row_step(N, D, dy_row);
    a.gu = const_cast<void*>(gu);
    a.dx = dx; a.dW_in = dW_in; a.dW_out = dW_out;
    return ffn_run(a, 1, workspace, workspace_bytes, stream);
}

int ttm_adamw_step(int count, const ttm_adamw_tensor* tensors, int bits, void* m, void* v, float* m_scale,
                   float* v_scale, int* step, double lr, const float* lr_at, double beta1, double beta2, double eps,
                   double weight_decay, const float* grad_scale, void* stream) {
    if (count < 0 || (count > 0 && !tensors) || (bits != 8 && bits != 32) || !step) return TTM_ERR_INVALID_ARG;
    if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0) || !((float)eps > 0.f) || !std::isfinite(eps) ||
        !std::isfinite(lr) || !std::isfinite(weight_decay))
        return TTM_ERR_INVALID_ARG;
    if ((bits == 8) != (m_scale != nullptr) || (bits == 8) != (v_scale != nullptr)) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<4>({m, v, m_scale, v_scale}) || !aligned(step, 4) || !aligned(lr_at, 4) || !aligned(grad_scale, 4))
        return TTM_ERR_INVALID_ARG;
    try {
        std::vector<ttm::AdamwEntry> list;
        std::vector<Range> ranges;
        list.reserve(count);
        ranges.reserve(3 * (size_t)count + 7);
        auto range = [&](const void* p, size_t bytes, bool written) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            if (p && bytes) ranges.push_back({at, at + bytes, written});
        };
        long long blocks = 0;
        for (int i = 0; i < count; ++i) {
            const ttm_adamw_tensor& t = tensors[i];
            if (t.n < 0 || !dtype_ok(t.param_dtype)) return TTM_ERR_INVALID_ARG;
            if (t.n > (1LL << 40)) return TTM_ERR_UNSUPPORTED;
            const long long first = blocks;
            blocks += (t.n + 255) / 256;
            if (!t.grad || t.n == 0) continue;
            const int pb = t.param_dtype == TTM_BF16, gb = t.grad_dtype == TTM_BF16;
            if (!t.param || !dtype_ok(t.grad_dtype) || !aligned(t.param, pb ? 2 : 4) || !aligned(t.grad, gb ? 2 : 4) ||
                !aligned(t.copy, 2))
                return TTM_ERR_INVALID_ARG;
            range(t.param, (size_t)t.n * (pb ? 2 : 4), true);
            range(t.grad, (size_t)t.n * (gb ? 2 : 4), false);
            range(t.copy, (size_t)t.n * 2, true);
            list.push_back({t.param, t.grad, t.copy, t.n, first, 0, pb, gb});
        }
        if (blocks && (!m || !v)) return TTM_ERR_INVALID_ARG;
        const size_t held = (size_t)blocks * 256 * (bits / 8);
        range(m, held, true);
        range(v, held, true);
        range(m_scale, (size_t)blocks * 4, true);
        range(v_scale, (size_t)blocks * 4, true);
        range(step, 8, true);
        range(lr_at, 4, false);
        range(grad_scale, 4, false);
        if (ranges_clash(ranges)) return TTM_ERR_INVALID_ARG;
        ttm::AdamwScalars a{};
        a.m = m; a.v = v; a.m_scale = m_scale; a.v_scale = v_scale; a.step = step;
        a.lr = (float)lr; a.lr_at = lr_at;
        a.b1 = (float)beta1; a.b2 = (float)beta2;
        a.c1 = (float)(1.0 - beta1); a.c2 = (float)(1.0 - beta2);
        a.log_b1 = (float)std::log(beta1); a.log_b2 = (float)std::log(beta2);
        // (the kernel's reciprocal takes a denominator below the smallest normal number as zero; a root above zero is 2^-75 at
        // least and takes no notice)
        a.eps = std::max((float)eps, FLT_MIN); a.decay = (float)weight_decay;
        a.grad_scale = grad_scale;
        int launches = 0;
        if (ttm::adamw_step_launch(list.data(), (int)list.size(), a, static_cast<cudaStream_t>(stream), &launches) !=
            cudaSuccess)
            return TTM_ERR_CUDA;
        ttm::api_note_launches(launches);
    } catch (const std::bad_alloc&) {
        return TTM_ERR_CUDA;
    }
    return TTM_OK;
}

int ttm_adamw_moments(long long blocks, const void* m, const void* v, const float* m_scale, const float* v_scale,
                      float* m_out, float* v_out, void* stream) {
    if (blocks < 0 || blocks > (1LL << 48)) return TTM_ERR_INVALID_ARG;
    if (blocks && (!m || !v || !m_scale || !v_scale || !m_out || !v_out)) return TTM_ERR_INVALID_ARG;
    if (!all_aligned16<6>({m, v, m_scale, v_scale, m_out, v_out})) return TTM_ERR_INVALID_ARG;
    const size_t n = (size_t)blocks * 256;
    const Span ins[] = {{m, n}, {v, n}, {m_scale, (size_t)blocks * 4}, {v_scale, (size_t)blocks * 4}};
    const Span outs[] = {{m_out, n * 4}, {v_out, n * 4}};
    if (!outputs_clear(ins, outs)) return TTM_ERR_INVALID_ARG;
    ttm::AdamwScalars a{};
    a.m = const_cast<void*>(m); a.v = const_cast<void*>(v);
    a.m_scale = const_cast<float*>(m_scale); a.v_scale = const_cast<float*>(v_scale);
    if (ttm::adamw_moments_launch(blocks, a, m_out, v_out, static_cast<cudaStream_t>(stream)) != cudaSuccess)
        return TTM_ERR_CUDA;
    ttm::api_note_launches(blocks > 0);
    return TTM_OK;
}

}  // extern "C"
