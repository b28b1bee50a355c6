// Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t, its gradient and its
// decode step.
//
// Gradient, with c_{T+1} = dL/dh_T's own adjoint dh_last:
//   G_t = dh_t + c_{t+1},  c_t = exp(g_t) G_t,
//   dx_t = G_t,  dg_t = c_t h_{t-1} (summed over the channels for a token gate),  dh0 = c_1.
#include <cuda_bf16.h>

#include "train_ops.h"

namespace ttm {
namespace {

template <typename E> __device__ __forceinline__ float to_f(E v) { return (float)v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_f(float v) { return (E)v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16(v); }

template <typename E, bool kToken>
__device__ __forceinline__ float gate(const GlrArgs& a, size_t n, size_t t, int d) {
    const size_t i = n * a.g_seq + t * a.g_tok;
    return expf(kToken ? static_cast<const float*>(a.g)[i] : to_f(static_cast<const E*>(a.g)[i + d]));
}

// One thread per (sequence, channel), token by token.
template <typename E, bool kToken>
__global__ void glr_fwd_kernel(GlrArgs a, const float* start) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (size_t)a.N * a.D) return;
    const size_t n = i / a.D;
    const int d = (int)(i % a.D);
    float h = start ? start[i] : 0.f;
    for (size_t t = 0; t < (size_t)a.T; ++t) {
        h = fmaf(gate<E, kToken>(a, n, t, d), h,
                 to_f(static_cast<const E*>(a.x)[n * a.x_seq + t * a.x_tok + d]));
        static_cast<E*>(a.h)[(n * a.T + t) * a.D + d] = from_f<E>(h);
    }
    a.h_last[i] = h;
}

// One block per sequence: threads stride over the channels, tokens from the
// last to the first; a token gate's gradient is reduced over the block.
template <typename E, bool kToken>
__global__ void glr_bwd_kernel(GlrArgs a, float* carry) {
    __shared__ float part[256];
    const size_t n = blockIdx.x;
    for (int d = threadIdx.x; d < a.D; d += blockDim.x)
        carry[n * a.D + d] = a.dh_last ? a.dh_last[n * a.D + d] : 0.f;
    for (size_t t = a.T; t-- > 0;) {
        float sum = 0.f;
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
            const size_t o = (n * a.T + t) * a.D + d;
            const float G = to_f(static_cast<const E*>(a.x)[n * a.x_seq + t * a.x_tok + d]) +
                            carry[n * a.D + d];
            const float c = gate<E, kToken>(a, n, t, d) * G;
            const float before = t ? to_f(static_cast<const E*>(a.h)[o - a.D])
                                   : (a.h0 ? a.h0[n * a.D + d] : 0.f);
            carry[n * a.D + d] = c;
            static_cast<E*>(a.dx)[o] = from_f<E>(G);
            if (kToken) sum += c * before;
            else static_cast<E*>(a.dg)[o] = from_f<E>(c * before);
        }
        if (kToken) {
            part[threadIdx.x] = sum;
            __syncthreads();
            for (int w = blockDim.x / 2; w > 0; w /= 2) {
                if (threadIdx.x < w) part[threadIdx.x] += part[threadIdx.x + w];
                __syncthreads();
            }
            if (threadIdx.x == 0) static_cast<float*>(a.dg)[n * a.T + t] = part[0];
        }
    }
    if (a.dh0)
        for (int d = threadIdx.x; d < a.D; d += blockDim.x) a.dh0[n * a.D + d] = carry[n * a.D + d];
}

template <typename E>
cudaError_t fwd(const GlrArgs& a, const float* start, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((size_t)a.N * a.D + 127) / 128);
    if (a.gate_token) glr_fwd_kernel<E, true><<<blocks, 128, 0, s>>>(a, start);
    else glr_fwd_kernel<E, false><<<blocks, 128, 0, s>>>(a, start);
    return cudaGetLastError();
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, int backward) {
    return backward ? (size_t)a.N * a.D * sizeof(float) : 0;
}

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    *launches = 1;
    return a.bf16 ? fwd<__nv_bfloat16>(a, a.h0, s) : fwd<float>(a, a.h0, s);
}

cudaError_t glr_step_launch(const GlrArgs& a, cudaStream_t s) {
    return a.bf16 ? fwd<__nv_bfloat16>(a, a.h_last, s) : fwd<float>(a, a.h_last, s);
}

cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    float* carry = static_cast<float*>(a.workspace);
    *launches = 1;
    if (a.bf16 && a.gate_token) glr_bwd_kernel<__nv_bfloat16, true><<<a.N, 256, 0, s>>>(a, carry);
    else if (a.bf16) glr_bwd_kernel<__nv_bfloat16, false><<<a.N, 256, 0, s>>>(a, carry);
    else if (a.gate_token) glr_bwd_kernel<float, true><<<a.N, 256, 0, s>>>(a, carry);
    else glr_bwd_kernel<float, false><<<a.N, 256, 0, s>>>(a, carry);
    return cudaGetLastError();
}

}  // namespace ttm
