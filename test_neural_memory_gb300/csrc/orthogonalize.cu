// Orthogonalised update: X_0 = G / max(|G|_F, eps), then per step
//   A = X X^T,  X <- a X + (b A + c A^2) X       (on the shorter side of G)
#include <cuda_bf16.h>

#include "train_ops.h"

namespace ttm {
namespace {

// X_0 in fp32, one block per matrix.
__global__ void ns_start_kernel(OrthoArgs a, float* X) {
    __shared__ float part[256];
    const size_t mn = (size_t)a.m * a.n, base = blockIdx.x * mn;
    auto G = [&](size_t i) {
        return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.G)[base + i])
                      : static_cast<const float*>(a.G)[base + i];
    };
    float s = 0.f;
    for (size_t i = threadIdx.x; i < mn; i += blockDim.x) s += G(i) * G(i);
    part[threadIdx.x] = s;
    __syncthreads();
    for (int w = 128; w > 0; w /= 2) {
        if (threadIdx.x < w) part[threadIdx.x] += part[threadIdx.x + w];
        __syncthreads();
    }
    const float r = 1.f / fmaxf(sqrtf(part[0]), a.eps);
    for (size_t i = threadIdx.x; i < mn; i += blockDim.x) X[base + i] = G(i) * r;
}

// out = alpha P Q + beta C with P [M][K], Q [K][N] given by strides; C and out [M][N].
__global__ void ns_product_kernel(int M, int N, int K, float alpha, const float* P, int p0, int p1,
                                  const float* Q, int q0, int q1, float beta, const float* C,
                                  float* out, size_t sP, size_t sQ, size_t sC,
                                  __nv_bfloat16* rounded) {
    __shared__ float p[16][17], q[16][17];
    const int r = blockIdx.y * 16 + threadIdx.y, c = blockIdx.x * 16 + threadIdx.x;
    P += blockIdx.z * sP;
    Q += blockIdx.z * sQ;
    float s = 0.f;
    for (int k = 0; k < K; k += 16) {
        p[threadIdx.y][threadIdx.x] =
            r < M && k + threadIdx.x < K ? P[(size_t)r * p0 + (size_t)(k + threadIdx.x) * p1] : 0.f;
        q[threadIdx.y][threadIdx.x] =
            c < N && k + threadIdx.y < K ? Q[(size_t)(k + threadIdx.y) * q0 + (size_t)c * q1] : 0.f;
        __syncthreads();
        for (int i = 0; i < 16; ++i) s += p[threadIdx.y][i] * q[i][threadIdx.x];
        __syncthreads();
    }
    if (r >= M || c >= N) return;
    const size_t o = blockIdx.z * sC + (size_t)r * N + c;
    const float v = alpha * s + (beta != 0.f ? beta * C[o] : 0.f);
    if (rounded) rounded[o] = __float2bfloat16(v);
    else out[o] = v;
}

__global__ void ns_round_kernel(size_t n, const float* X, __nv_bfloat16* out) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) out[i] = __float2bfloat16(X[i]);
}

}  // namespace

size_t ortho_workspace_bytes(int batch, int m, int n) {
    const size_t r = m < n ? m : n;
    return (size_t)batch * (2 * (size_t)m * n + 2 * r * r) * sizeof(float);
}

cudaError_t ortho_launch(const OrthoArgs& a, cudaStream_t s, int* launches) {
    const size_t mn = (size_t)a.m * a.n;
    const int r = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
    const bool wide = a.m <= a.n;
    const size_t rr = (size_t)r * r;
    float* X = static_cast<float*>(a.workspace);
    float *Y = X + a.batch * mn, *A = Y + a.batch * mn, *B = A + a.batch * rr;
    ns_start_kernel<<<a.batch, 256, 0, s>>>(a, X);
    *launches = 1;
    const dim3 t(16, 16);
    auto grid = [&](int M, int N) { return dim3((N + 15) / 16, (M + 15) / 16, a.batch); };
    for (int i = 0; i < a.steps; ++i) {
        const float* c = a.coeffs + 3 * i;
        __nv_bfloat16* last = i + 1 == a.steps ? static_cast<__nv_bfloat16*>(a.out) : nullptr;
        // A = X X^T (X^T X for a tall matrix); B = b A + c A^2; Y = a X + B X (X B)
        const int k0 = wide ? 1 : a.n, k1 = wide ? a.n : 1;
        ns_product_kernel<<<grid(r, r), t, 0, s>>>(r, r, l, 1.f, X, k1, k0, X, k0, k1, 0.f, nullptr,
                                                   A, mn, mn, rr, nullptr);
        ns_product_kernel<<<grid(r, r), t, 0, s>>>(r, r, r, c[2], A, r, 1, A, r, 1, c[1], A, B, rr,
                                                   rr, rr, nullptr);
        if (wide)
            ns_product_kernel<<<grid(a.m, a.n), t, 0, s>>>(a.m, a.n, r, 1.f, B, r, 1, X, a.n, 1, c[0],
                                                           X, Y, rr, mn, mn, last);
        else
            ns_product_kernel<<<grid(a.m, a.n), t, 0, s>>>(a.m, a.n, r, 1.f, X, a.n, 1, B, r, 1, c[0],
                                                           X, Y, mn, rr, mn, last);
        float* z = X; X = Y; Y = z;
        *launches += 3;
    }
    if (a.steps == 0) {
        ns_round_kernel<<<(unsigned)((a.batch * mn + 255) / 256), 256, 0, s>>>(
            a.batch * mn, X, static_cast<__nv_bfloat16*>(a.out));
        ++*launches;
    }
    return cudaGetLastError();
}

}  // namespace ttm
