// Layer norm over the last axis and its gradient.
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),
//   y = (x - mean) rstd w + b
//   with n = (x - mean) rstd and u = dy w:
//   dx = rstd (u - sum u / D - n sum(u n) / D),  dw = sum over rows of dy n,  db of dy
#include <cuda_bf16.h>

#include "train_ops.h"

namespace ttm {
namespace {

template <typename E> __device__ __forceinline__ float to_f(E v) { return (float)v; }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E from_f(float v) { return (E)v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16(v); }

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename E>
__global__ void ln_fwd_kernel(LayerNormArgs a) {
    const size_t row = (size_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= (size_t)a.N) return;
    const E* x = static_cast<const E*>(a.x) + row * a.x_row;
    float s = 0.f;
    for (int d = lane; d < a.D; d += 32) s += to_f(x[d]);
    const float mean = warp_sum(s) / a.D;
    s = 0.f;
    for (int d = lane; d < a.D; d += 32) s += (to_f(x[d]) - mean) * (to_f(x[d]) - mean);
    const float rstd = 1.f / sqrtf(warp_sum(s) / a.D + a.eps);
    for (int d = lane; d < a.D; d += 32) {
        const float n = (to_f(x[d]) - mean) * rstd;
        static_cast<E*>(a.y)[row * a.D + d] =
            from_f<E>((a.w ? n * a.w[d] : n) + (a.b ? a.b[d] : 0.f));
    }
    if (lane == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
}

template <typename E>
__global__ void ln_bwd_dx_kernel(LayerNormArgs a) {
    const size_t row = (size_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= (size_t)a.N) return;
    const E* x = static_cast<const E*>(a.x) + row * a.x_row;
    const E* dy = static_cast<const E*>(a.dy) + row * a.dy_row;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float su = 0.f, sn = 0.f;
    for (int d = lane; d < a.D; d += 32) {
        const float u = to_f(dy[d]) * (a.w ? a.w[d] : 1.f);
        su += u;
        sn += u * ((to_f(x[d]) - mean) * rstd);
    }
    su = warp_sum(su) / a.D;
    sn = warp_sum(sn) / a.D;
    for (int d = lane; d < a.D; d += 32) {
        const float u = to_f(dy[d]) * (a.w ? a.w[d] : 1.f);
        const float n = (to_f(x[d]) - mean) * rstd;
        static_cast<E*>(a.dx)[row * a.D + d] = from_f<E>(rstd * (u - su - n * sn));
    }
}

constexpr int kParts = 64;   // row ranges of the column sums

template <typename E>
__global__ void ln_bwd_dw_kernel(LayerNormArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    float sw = 0.f, sb = 0.f;
    for (size_t row = blockIdx.y; row < (size_t)a.N; row += kParts) {
        const float dy = to_f(static_cast<const E*>(a.dy)[row * a.dy_row + d]);
        const float x = to_f(static_cast<const E*>(a.x)[row * a.x_row + d]);
        sw += dy * ((x - a.mean[row]) * a.rstd[row]);
        sb += dy;
    }
    a.partial[((size_t)blockIdx.y * 2 + 0) * a.D + d] = sw;
    a.partial[((size_t)blockIdx.y * 2 + 1) * a.D + d] = sb;
}

__global__ void ln_bwd_join_kernel(LayerNormArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    float sw = 0.f, sb = 0.f;
    for (int p = 0; p < kParts; ++p) {
        sw += a.partial[((size_t)p * 2 + 0) * a.D + d];
        sb += a.partial[((size_t)p * 2 + 1) * a.D + d];
    }
    if (a.dw) a.dw[d] = sw;
    if (a.db) a.db[d] = sb;
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int, int D) { return (size_t)kParts * 2 * D * sizeof(float); }

cudaError_t layer_norm_fwd_launch(const LayerNormArgs& a, cudaStream_t s) {
    const unsigned blocks = (unsigned)(((size_t)a.N + 7) / 8);
    if (a.bf16) ln_fwd_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(a);
    else ln_fwd_kernel<float><<<blocks, 256, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t layer_norm_bwd_launch(const LayerNormArgs& a, cudaStream_t s, int* launches) {
    const unsigned blocks = (unsigned)(((size_t)a.N + 7) / 8);
    const dim3 cols((a.D + 127) / 128, kParts);
    *launches = 0;
    if (a.N > 0) {
        if (a.bf16) ln_bwd_dx_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(a);
        else ln_bwd_dx_kernel<float><<<blocks, 256, 0, s>>>(a);
        ++*launches;
    }
    if (a.dw || a.db) {
        if (a.bf16) ln_bwd_dw_kernel<__nv_bfloat16><<<cols, 128, 0, s>>>(a);
        else ln_bwd_dw_kernel<float><<<cols, 128, 0, s>>>(a);
        ln_bwd_join_kernel<<<cols.x, 128, 0, s>>>(a);
        *launches += 2;
    }
    return cudaGetLastError();
}

}  // namespace ttm
