// Internal interface of the operators around the memory scan (gated linear
// recurrence, layer norm, orthogonalised update, short convolution, gated feed-forward block,
// AdamW): argument blocks that
// train_api.cu has validated, and the launchers of their translation units.
#pragma once

#include <cstddef>
#include <cuda_runtime.h>

namespace ttm {

// Gated linear recurrence (glr.cu): h_t = exp(g_t) h_{t-1} + x_t per sequence
// and channel.  Strides in elements; channels are contiguous.
struct GlrArgs {
    int N, T, D;
    int bf16;                       // type of x, h (and of g with a gate per channel)
    int gate_token;                 // 1: g is fp32, one value per token; 0: one per channel
    const void* x;                  // forward, step: the input; gradient: dh
    long long x_seq, x_tok;
    const void* g;
    long long g_seq, g_tok;
    const float* h0;                // [N][D] or NULL (0)
    void* h;                        // [N][T][D]: written (forward, step), read (gradient)
    float* h_last;                  // [N][D]: final state (forward); state in place (step)
    const float* dh_last;           // gradient: [N][D] or NULL
    void *dx, *dg;                  // gradient: [N][T][D]; dg [N][T] fp32 with a token gate
    float* dh0;                     // gradient: [N][D] or NULL
    void* workspace;
    int* status;
    long long wait_cycles;
    unsigned debug_stall;           // test hook: tile + 1 whose copies never complete; 0: none
};

size_t glr_workspace_bytes(const GlrArgs& a, int backward);
cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t s, int* launches);
cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t s, int* launches);
cudaError_t glr_step_launch(const GlrArgs& a, cudaStream_t s);

// Layer norm over the last axis (layer_norm.cu).
struct LayerNormArgs {
    int N, D;
    int bf16;
    const void* x;
    long long x_row;                // elements between rows
    const float *w, *b;             // [D] or NULL (1, 0)
    float eps;
    void* y;                        // forward: [N][D]
    float *mean, *rstd;             // [N]: written (forward, NULL to skip), read (gradient)
    const void* dy;
    long long dy_row;
    void* dx;                       // [N][D]
    float *dw, *db;                 // [D] or NULL
    float* partial;                 // gradient: workspace
};

size_t layer_norm_bwd_workspace_bytes(int N, int D);
cudaError_t layer_norm_fwd_launch(const LayerNormArgs& a, cudaStream_t s);
cudaError_t layer_norm_bwd_launch(const LayerNormArgs& a, cudaStream_t s, int* launches);

// Orthogonalised update (orthogonalize.cu).
constexpr int kNsMaxSteps = 32;
// One step with its operands as they are stored: X, A and B times a power of two each.
struct NsStep {
    float a;                        // A = a X X^T
    float b1, c2;                   // B = b1 A + c2 A A
    float keep, b;                  // X' = (keep + b diag B) X + b (B without its diagonal) X
};
struct OrthoArgs {
    int batch, m, n;
    int bf16;                       // type of G; 0: fp32
    const void* G;                  // [batch][m][n]
    int steps;
    float coeffs[3 * kNsMaxSteps];
    int late;                       // first step whose B takes its diagonal times all of X
    NsStep step[kNsMaxSteps];       // set by ortho_launch
    float eps;
    void* out;                      // [batch][m][n] bf16
    void* workspace;
    int* status;
    long long wait_cycles;
    int debug_stall;                // test hook: product or copy + 1 that is never announced; 0: none
};

size_t ortho_workspace_bytes(int batch, int m, int n);
cudaError_t ortho_launch(const OrthoArgs& a, cudaStream_t s, int* launches);

// Short causal convolution (causal_conv.cu), depthwise, with an optional SiLU.  Strides in elements;
// channels are contiguous.
struct ConvArgs {
    int N, T, C, K;
    int bf16;                       // type of x, y, dy, dx and the states
    int silu;
    const void* x;                  // [N][T][C]
    long long x_seq, x_tok;
    const float *w, *b;             // [C][K], [C] or NULL (0)
    const void* state0;             // [N][K-1][C] or NULL (0)
    const int* doc;                 // [N][T], doc_seq apart, or NULL
    long long doc_seq;
    void* y;                        // forward, step: [N][T][C]
    void* state;                    // forward, step: [N][K-1][C] or NULL; may be state0 in a step
    const void* dy;                 // gradient
    long long dy_seq, dy_tok;
    const void* dstate;             // [N][K-1][C] or NULL (0)
    void *dx, *dstate0;             // [N][T][C]; [N][K-1][C] or NULL
    float *dw, *db;                 // [C][K], [C] or NULL
    float* partial;                 // workspace, NULL when neither dw nor db is wanted
};

size_t conv_bwd_workspace_bytes(const ConvArgs& a);
cudaError_t conv_fwd_launch(const ConvArgs& a, cudaStream_t s, int* launches);
cudaError_t conv_step_launch(const ConvArgs& a, cudaStream_t s);
cudaError_t conv_bwd_launch(const ConvArgs& a, cudaStream_t s, int* launches);

// AdamW step over many tensors (adamw.cu).  The moments of tensor i lie from value 256 first on.
struct AdamwEntry {
    void* p;
    const void* g;
    void* copy;                     // bf16, or NULL
    long long n;
    long long first;                // block of 256 values
    int chunk;                      // chunks of the tensors before it in the same launch
    int p_bf16, g_bf16;
};
struct AdamwScalars {
    void *m, *v;
    float *m_scale, *v_scale;       // 8 bits, else NULL
    int* step;                      // steps done, blocks done
    float lr;
    const float* lr_at;             // or NULL
    float b1, b2, c1, c2;           // betas and one minus each
    float log_b1, log_b2;
    float eps, decay;
    const float* grad_scale;        // or NULL
};
cudaError_t adamw_step_launch(const AdamwEntry* tensors, int count, const AdamwScalars& a, cudaStream_t s,
                              int* launches);
cudaError_t adamw_moments_launch(long long blocks, const AdamwScalars& a, float* m, float* v, cudaStream_t s);

// Gated feed-forward block (gated_ffn.cu).  bf16; row strides in elements.
struct FfnArgs {
    int N, D, F;
    int gelu;                       // 0: SiLU
    const void* x;                  // [N][D]
    long long x_row;
    const void *W_in, *W_out;       // [D][2F], [F][D]
    const void* residual;           // [N][D] or NULL
    long long residual_row;
    void* y;                        // forward: [N][D]
    void* gu;                       // [N][2F]: written (forward, NULL to skip), read (gradient)
    const void* dy;                 // gradient: [N][D]
    long long dy_row;
    void *dx, *dW_in, *dW_out;      // gradient; each may be NULL
    void* workspace;
    int* status;
    long long wait_cycles;
    int debug_stall;                // test hook: stage + 1 that never fills; 0: none
};
size_t ffn_workspace_bytes(int N, int D, int F, int backward);
cudaError_t ffn_fwd_launch(const FfnArgs& a, cudaStream_t s, int* launches);
cudaError_t ffn_bwd_launch(const FfnArgs& a, cudaStream_t s, int* launches);

// Tensor map (a CUtensorMap) of a 3-D view: dims from the innermost on, byte strides of
// the outer two (multiples of 16, below 2^40, the second a multiple of the first), a box of at most
// 256 values a side whose inner extent is a multiple of 16 bytes.  Values outside the view load as zero.
// tma_map.cu; false when the driver refuses it.
enum class TmaType { f32, bf16, f16 };
bool make_tma_map(void* map, TmaType type, const void* ptr, const unsigned long long (&dims)[3],
                  const unsigned long long (&strides)[2], const unsigned (&box)[3], bool swizzle128);

// Process-wide state of the API layer (ttm_api.cu).
int* api_status_ptr();              // device status word of the current device; NULL on failure
long long api_wait_cycles();        // bounded-wait limit in SM cycles (0: default)
int api_take_stall();               // test hook: the setting + 1, used up; 0: none
void api_note_launches(int kernels);

}  // namespace ttm
