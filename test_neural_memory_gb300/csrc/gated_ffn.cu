// Gated feed-forward block: g | u = x W_in, h = act(g) u, y = h W_out (+ residual), and its gradient.
// Plain tiles on the CUDA cores: 64 x 64 results a block, 4 x 4 a thread, 16 of K at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "train_ops.h"

namespace ttm {
namespace {

using bf16 = __nv_bfloat16;

// Element (row, k) of A at row * rs + k * ks.
struct Operand {
    const bf16* p;
    long long rs, ks;
};

__device__ __forceinline__ float act_of(float g, int gelu, float& slope) {
    if (gelu) {
        const float c = 0.5f * erfcf(-0.70710678f * g);
        slope = c + g * 0.39894228f * expf(-0.5f * g * g);
        return g * c;
    }
    const float s = 1.f / (1.f + expf(-g));
    slope = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
}

enum { kStore, kGated, kGatedBack };

struct Epilogue {
    bf16* out;                          // [M][N]
    const bf16* add;
    long long add_row;
    bf16 *h, *gu;                       // kGated: results [M][F], [M][2F]; kGatedBack: gu read, out = dgu
    int F, gelu;
};

template <int MODE>
__global__ void __launch_bounds__(256) gemm_kernel(Operand A, Operand B, int M, int N, int K, Epilogue e) {
    __shared__ float sa[16][65], sb[2][16][65];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int row0 = blockIdx.y * 64, col0 = blockIdx.x * 64;
    constexpr int kTwo = MODE == kGated ? 2 : 1;
    float acc[kTwo][4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int r = i >> 4, k = i & 15;
            sa[k][r] = row0 + r < M && k0 + k < K ? __bfloat162float(A.p[(row0 + r) * A.rs + (k0 + k) * A.ks]) : 0.f;
            for (int t = 0; t < kTwo; ++t)
                sb[t][k][r] = col0 + r < N && k0 + k < K
                                  ? __bfloat162float(B.p[(col0 + r + (long long)t * e.F) * B.rs + (k0 + k) * B.ks])
                                  : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j)
                    for (int t = 0; t < kTwo; ++t)
                        acc[t][i][j] = fmaf(sa[k][ty + 16 * i], sb[t][k][tx + 16 * j], acc[t][i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long r = row0 + ty + 16 * i;
            const int c = col0 + tx + 16 * j;
            if (r >= M || c >= N) continue;
            float slope;
            if (MODE == kStore) {
                float v = acc[0][i][j];
                if (e.add) v += __bfloat162float(e.add[r * e.add_row + c]);
                e.out[r * N + c] = __float2bfloat16_rn(v);
            } else if (MODE == kGated) {
                const float g = acc[0][i][j], u = acc[kTwo - 1][i][j];
                e.h[r * e.F + c] = __float2bfloat16_rn(act_of(g, e.gelu, slope) * u);
                if (e.gu) {
                    e.gu[r * 2 * e.F + c] = __float2bfloat16_rn(g);
                    e.gu[r * 2 * e.F + e.F + c] = __float2bfloat16_rn(u);
                }
            } else {
                const float dh = acc[0][i][j], g = __bfloat162float(e.gu[r * 2 * e.F + c]),
                            u = __bfloat162float(e.gu[r * 2 * e.F + e.F + c]), a = act_of(g, e.gelu, slope);
                e.h[r * e.F + c] = __float2bfloat16_rn(a * u);
                e.out[r * 2 * e.F + c] = __float2bfloat16_rn(dh * u * slope);
                e.out[r * 2 * e.F + e.F + c] = __float2bfloat16_rn(dh * a);
            }
        }
}

template <int MODE>
cudaError_t gemm(Operand A, Operand B, int M, int N, int K, const Epilogue& e, cudaStream_t s) {
    gemm_kernel<MODE><<<dim3((N + 63) / 64, (M + 63) / 64), 256, 0, s>>>(A, B, M, N, K, e);
    return cudaGetLastError();
}

}  // namespace

size_t ffn_workspace_bytes(int N, int D, int F, int backward) {
    return (size_t)N * F * 2 * (backward ? 3 : 1);
}

cudaError_t ffn_fwd_launch(const FfnArgs& a, cudaStream_t s, int* launches) {
    const bf16 *x = static_cast<const bf16*>(a.x), *wi = static_cast<const bf16*>(a.W_in),
               *wo = static_cast<const bf16*>(a.W_out);
    Epilogue e{};
    e.h = static_cast<bf16*>(a.workspace);
    e.gu = static_cast<bf16*>(a.gu);
    e.F = a.F;
    e.gelu = a.gelu;
    *launches = 2;
    const cudaError_t r = gemm<kGated>({x, a.x_row, 1}, {wi, 1, 2LL * a.F}, a.N, a.F, a.D, e, s);
    if (r != cudaSuccess) return r;
    e.out = static_cast<bf16*>(a.y);
    e.add = static_cast<const bf16*>(a.residual);
    e.add_row = a.residual_row;
    return gemm<kStore>({e.h, a.F, 1}, {wo, 1, a.D}, a.N, a.D, a.F, e, s);
}

cudaError_t ffn_bwd_launch(const FfnArgs& a, cudaStream_t s, int* launches) {
    const bf16 *x = static_cast<const bf16*>(a.x), *wi = static_cast<const bf16*>(a.W_in),
               *wo = static_cast<const bf16*>(a.W_out), *dy = static_cast<const bf16*>(a.dy);
    bf16* dgu = static_cast<bf16*>(a.workspace);
    bf16* h = dgu + (size_t)a.N * 2 * a.F;
    Epilogue e{};
    e.F = a.F;
    e.gelu = a.gelu;
    e.out = dgu;
    e.h = h;
    e.gu = static_cast<bf16*>(a.gu);
    *launches = 1;
    cudaError_t r = gemm<kGatedBack>({dy, a.dy_row, 1}, {wo, a.D, 1}, a.N, a.F, a.D, e, s);
    Epilogue o{};
    if (r == cudaSuccess && a.dx) {
        o.out = static_cast<bf16*>(a.dx);
        r = gemm<kStore>({dgu, 2LL * a.F, 1}, {wi, 2LL * a.F, 1}, a.N, a.D, 2 * a.F, o, s);
        ++*launches;
    }
    if (r == cudaSuccess && a.dW_in) {
        o.out = static_cast<bf16*>(a.dW_in);
        r = gemm<kStore>({x, 1, a.x_row}, {dgu, 1, 2LL * a.F}, a.D, 2 * a.F, a.N, o, s);
        ++*launches;
    }
    if (r == cudaSuccess && a.dW_out) {
        o.out = static_cast<bf16*>(a.dW_out);
        r = gemm<kStore>({h, 1, a.F}, {dy, 1, a.dy_row}, a.F, a.D, a.N, o, s);
        ++*launches;
    }
    return r;
}

}  // namespace ttm
