// Layer norm over the last axis and its gradient.
//
// Mathematics, per row of D values:
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  n = (x - mean) rstd,
//   y = n w + b;
// with u = dy w:
//   dx = rstd (u - sum u / D - n sum(u n) / D),
//   dw = sum over rows of dy n,  db = sum over rows of dy.
//
// What bounds it: HBM, two tensors forward and three in the gradient.  A row is read
// once and stays in registers: the variance is taken about the mean (no difference of
// large sums), and the gradient's dw and db are added up in registers over the rows that
// a thread group walks, so x and dy are read once for all three results.
//
// Layout: TPR threads share a row, each K packs of W values that are TPR packs apart
// (every access of a warp is contiguous), ROWS rows at a time so that enough loads are
// in flight and one reduction serves several rows.  TPR is 8 or 32 (shuffles) for
// short rows and the whole block of 256 (shuffles, then shared memory) for long ones.
// Rows longer than the registers hold are read again from the cache instead.
// W is the widest pack that the rows' alignment and D allow.
//
// The gradient's blocks leave their dw, db sums in the workspace and a second kernel adds
// them in a fixed order: no atomics, so equal inputs give equal bits.
#include <cuda_bf16.h>

#include <cstdint>

#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 152 * 4;     // gradient: blocks, and partial sums per column
constexpr int kLongThreads = 512;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float v) { o = __float2bfloat16(v); }

template <typename E, int W>
struct alignas(sizeof(E) * W) Pack {
    E v[W];
};

template <typename E, int W>
__device__ __forceinline__ Pack<E, W> load_pack(const E* p) {
    return *reinterpret_cast<const Pack<E, W>*>(p);
}

// W fp32 values; their address is a multiple of 4 W bytes, at most 16 taken at a time.
template <int W>
__device__ __forceinline__ void load_f(const float* p, float (&f)[W], float absent) {
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = absent;
    if (!p) return;
    constexpr int S = W < 4 ? W : 4;
#pragma unroll
    for (int i = 0; i < W; i += S) {
        const Pack<float, S> q = load_pack<float, S>(p + i);
#pragma unroll
        for (int j = 0; j < S; ++j) f[i + j] = q.v[j];
    }
}

// Sums over the TPR threads of a row; TPR = kThreads goes through `buf` (shared,
// [kWarps][C]), which the caller may use again after the next reduction's barrier.
template <int TPR, int C>
__device__ __forceinline__ void row_sums(float (&s)[C], float (*buf)[C]) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
            s[c] += __shfl_xor_sync(0xffffffffu, s[c], o);
    if (TPR > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) buf[warp][c] = s[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            s[c] = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) s[c] += buf[w][c];
        }
    }
}

template <typename E, int W, int TPR, int K, int ROWS>
__global__ void __launch_bounds__(kThreads) ln_fwd_kernel(LayerNormArgs a) {
    constexpr int kSets = kThreads / TPR;             // rows side by side in a block
    __shared__ float buf[2][kWarps][ROWS];
    const int lane = threadIdx.x % TPR, set = threadIdx.x / TPR;
    const int packs = a.D / W;
    const float inv = 1.f / a.D;
    const E* x = static_cast<const E*>(a.x);
    E* y = static_cast<E*>(a.y);
    for (long long r0 = (long long)blockIdx.x * kSets * ROWS; r0 < a.N;
         r0 += (long long)gridDim.x * kSets * ROWS) {
        Pack<E, W> in[ROWS][K];
        float s[ROWS], mean[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets + set;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (r < a.N && lane + k * TPR < packs)
                    in[i][k] = load_pack<E, W>(x + r * a.x_row + (lane + k * TPR) * W);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            s[i] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (r0 + i * kSets + set < a.N && lane + k * TPR < packs)
#pragma unroll
                    for (int v = 0; v < W; ++v) s[i] += to_f(in[i][k].v[v]);
        }
        row_sums<TPR>(s, buf[0]);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            mean[i] = s[i] * inv;
            s[i] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (r0 + i * kSets + set < a.N && lane + k * TPR < packs)
#pragma unroll
                    for (int v = 0; v < W; ++v) {
                        const float d = to_f(in[i][k].v[v]) - mean[i];
                        s[i] = fmaf(d, d, s[i]);
                    }
        }
        row_sums<TPR>(s, buf[1]);
        float rstd[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) rstd[i] = 1.f / sqrtf(fmaf(s[i], inv, a.eps));
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (lane + k * TPR) * W;
            if (lane + k * TPR >= packs) continue;
            float w[W], b[W];
            load_f<W>(a.w ? a.w + c : nullptr, w, 1.f);
            load_f<W>(a.b ? a.b + c : nullptr, b, 0.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + i * kSets + set;
                if (r >= a.N) continue;
                Pack<E, W> out;
#pragma unroll
                for (int v = 0; v < W; ++v)
                    put(out.v[v], fmaf((to_f(in[i][k].v[v]) - mean[i]) * rstd[i], w[v], b[v]));
                *reinterpret_cast<Pack<E, W>*>(y + r * a.D + c) = out;
            }
        }
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + i * kSets + set;
                if (r >= a.N) continue;
                if (a.mean) a.mean[r] = mean[i];
                if (a.rstd) a.rstd[r] = rstd[i];
            }
    }
}

template <typename E, int W, int TPR, int K, int ROWS>
__global__ void __launch_bounds__(kThreads) ln_bwd_kernel(LayerNormArgs a) {
    constexpr int kSets = kThreads / TPR;
    __shared__ float buf[2][kWarps][2 * ROWS];
    const int lane = threadIdx.x % TPR, set = threadIdx.x / TPR;
    const int packs = a.D / W;
    const float inv = 1.f / a.D;
    const E *x = static_cast<const E*>(a.x), *dy = static_cast<const E*>(a.dy);
    E* dx = static_cast<E*>(a.dx);
    float dw[K][W], db[K][W];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int v = 0; v < W; ++v) dw[k][v] = db[k][v] = 0.f;
    int turn = 0;
    for (long long r0 = (long long)blockIdx.x * kSets * ROWS; r0 < a.N;
         r0 += (long long)gridDim.x * kSets * ROWS, turn ^= 1) {
        Pack<E, W> px[ROWS][K], pd[ROWS][K];
        float mean[ROWS], rstd[ROWS], s[2 * ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets + set;
            const bool in = r < a.N;
            mean[i] = in ? a.mean[r] : 0.f;
            rstd[i] = in ? a.rstd[r] : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (lane + k * TPR) * W;
                if (in && lane + k * TPR < packs) {
                    px[i][k] = load_pack<E, W>(x + r * a.x_row + c);
                    pd[i][k] = load_pack<E, W>(dy + r * a.dy_row + c);
                } else {
#pragma unroll
                    for (int v = 0; v < W; ++v) {
                        put(px[i][k].v[v], 0.f);
                        put(pd[i][k].v[v], 0.f);
                    }
                }
            }
            s[2 * i] = s[2 * i + 1] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[W];
            load_f<W>(a.w && lane + k * TPR < packs ? a.w + (lane + k * TPR) * W : nullptr, w, 1.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const float g = to_f(pd[i][k].v[v]);
                    const float n = (to_f(px[i][k].v[v]) - mean[i]) * rstd[i];
                    const float u = g * w[v];
                    db[k][v] += g;                      // absent rows and columns have g = 0
                    dw[k][v] = fmaf(g, n, dw[k][v]);
                    s[2 * i] += u;
                    s[2 * i + 1] = fmaf(u, n, s[2 * i + 1]);
                }
        }
        row_sums<TPR>(s, buf[turn]);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (lane + k * TPR) * W;
            if (lane + k * TPR >= packs) continue;
            float w[W];
            load_f<W>(a.w ? a.w + c : nullptr, w, 1.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + i * kSets + set;
                if (r >= a.N) continue;
                const float su = s[2 * i] * inv, sn = s[2 * i + 1] * inv;
                Pack<E, W> out;
#pragma unroll
                for (int v = 0; v < W; ++v) {
                    const float n = (to_f(px[i][k].v[v]) - mean[i]) * rstd[i];
                    put(out.v[v], rstd[i] * (fmaf(to_f(pd[i][k].v[v]), w[v], -su) - n * sn));
                }
                *reinterpret_cast<Pack<E, W>*>(dx + r * a.D + c) = out;
            }
        }
    }
    if (!a.partial) return;
    // over the rows side by side in the block: sets of a warp by shuffles, warps through shared
    // memory (one warp or more per row: the sets are whole warps)
    float* part = a.partial + (size_t)blockIdx.x * 2 * a.D;
    if (TPR == kThreads) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < W; ++v) {
                const int c = (lane + k * TPR) * W + v;
                if (lane + k * TPR < packs) {
                    part[c] = dw[k][v];
                    part[a.D + c] = db[k][v];
                }
            }
    } else {
        extern __shared__ float sums[];                 // [kWarps][2][TPR K W]
        const int cols = TPR * K * W, warp = threadIdx.x >> 5;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < W; ++v) {
#pragma unroll
                for (int o = TPR; o < 32; o <<= 1) {
                    dw[k][v] += __shfl_xor_sync(0xffffffffu, dw[k][v], o);
                    db[k][v] += __shfl_xor_sync(0xffffffffu, db[k][v], o);
                }
                if ((threadIdx.x & 31) < TPR) {
                    const int c = (lane + k * TPR) * W + v;
                    sums[(warp * 2 + 0) * cols + c] = dw[k][v];
                    sums[(warp * 2 + 1) * cols + c] = db[k][v];
                }
            }
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) {
            const int which = c >= a.D, col = c - which * a.D;
            float t = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) t += sums[(w * 2 + which) * cols + col];
            part[c] = t;
        }
    }
}

// Rows longer than the registers: one block per row, values read again from the cache.
template <typename E>
__device__ __forceinline__ float block_sum(float s, float* buf) {
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < kLongThreads / 32; ++w) s += buf[w];
    return s;
}

template <typename E>
__global__ void __launch_bounds__(kLongThreads) ln_fwd_long_kernel(LayerNormArgs a) {
    __shared__ float buf[kLongThreads / 32];
    for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
        const E* x = static_cast<const E*>(a.x) + r * a.x_row;
        float s = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kLongThreads) s += to_f(x[d]);
        const float mean = block_sum<E>(s, buf) / a.D;
        s = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kLongThreads) {
            const float c = to_f(x[d]) - mean;
            s = fmaf(c, c, s);
        }
        const float rstd = 1.f / sqrtf(block_sum<E>(s, buf) / a.D + a.eps);
        for (int d = threadIdx.x; d < a.D; d += kLongThreads)
            put(static_cast<E*>(a.y)[r * a.D + d],
                fmaf((to_f(x[d]) - mean) * rstd, a.w ? a.w[d] : 1.f, a.b ? a.b[d] : 0.f));
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = rstd;
        }
    }
}

template <typename E>
__global__ void __launch_bounds__(kLongThreads) ln_bwd_long_kernel(LayerNormArgs a) {
    __shared__ float buf[kLongThreads / 32];
    float* part = a.partial ? a.partial + (size_t)blockIdx.x * 2 * a.D : nullptr;
    if (part)
        for (int d = threadIdx.x; d < 2 * a.D; d += kLongThreads) part[d] = 0.f;
    __syncthreads();
    for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
        const E* x = static_cast<const E*>(a.x) + r * a.x_row;
        const E* dy = static_cast<const E*>(a.dy) + r * a.dy_row;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float su = 0.f, sn = 0.f;
        for (int d = threadIdx.x; d < a.D; d += kLongThreads) {
            const float g = to_f(dy[d]), n = (to_f(x[d]) - mean) * rstd;
            const float u = g * (a.w ? a.w[d] : 1.f);
            su += u;
            sn = fmaf(u, n, sn);
            if (part) {                                  // this thread's own columns
                part[d] = fmaf(g, n, part[d]);
                part[a.D + d] += g;
            }
        }
        su = block_sum<E>(su, buf) / a.D;
        sn = block_sum<E>(sn, buf) / a.D;
        for (int d = threadIdx.x; d < a.D; d += kLongThreads) {
            const float n = (to_f(x[d]) - mean) * rstd;
            put(static_cast<E*>(a.dx)[r * a.D + d],
                rstd * (fmaf(to_f(dy[d]), a.w ? a.w[d] : 1.f, -su) - n * sn));
        }
    }
}

// dw, db from the blocks' partial sums: 32 columns a block, 16 threads down each.
__global__ void __launch_bounds__(512) ln_join_kernel(const float* part, int blocks, int D,
                                                      float* dw, float* db) {
    __shared__ float buf[16][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < 2 * D)
        for (int p = threadIdx.y; p < blocks; p += 16) s += part[(size_t)p * 2 * D + c];
    buf[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= 2 * D) return;
    s = 0.f;
#pragma unroll
    for (int y = 0; y < 16; ++y) s += buf[y][threadIdx.x];
    if (c < D) {
        if (dw) dw[c] = s;
    } else if (db) {
        db[c - D] = s;
    }
}

// ------------------------------------------------------------------------- host

template <typename E, int W, int TPR, int K>
cudaError_t run(const LayerNormArgs& a, bool back, int blocks_of_rows, cudaStream_t s) {
    constexpr int sets = kThreads / TPR;
    if (!back) {
        constexpr int rows = W * K * (int)sizeof(E) >= 64 ? 1 : (W * K * (int)sizeof(E) >= 32 ? 2 : 4);
        const long long need = ((long long)a.N + sets * rows - 1) / (sets * rows);
        ln_fwd_kernel<E, W, TPR, K, rows>
            <<<(unsigned)(need < 152 * 16 ? need : 152 * 16), kThreads, 0, s>>>(a);
    } else {
        constexpr int rows = W * K * (int)sizeof(E) >= 32 ? 1 : 2;
        const size_t shared = TPR == kThreads || !a.partial ? 0 : (size_t)kWarps * 2 * TPR * K * W * 4;
        auto kernel = ln_bwd_kernel<E, W, TPR, K, rows>;
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
        if (e != cudaSuccess) return e;
        kernel<<<blocks_of_rows, kThreads, shared, s>>>(a);
    }
    return cudaGetLastError();
}

// Widest pack the rows allow: 16 bytes, 4 bytes, one value.
template <typename E>
int pack_width(const LayerNormArgs& a, bool back) {
    auto fits = [&](int w) {
        const unsigned long long b = w * sizeof(E);
        if (a.D % w || reinterpret_cast<uintptr_t>(a.x) % b || (a.N > 1 && a.x_row * sizeof(E) % b))
            return false;
        return !back || (reinterpret_cast<uintptr_t>(a.dy) % b == 0 &&
                         (a.N <= 1 || a.dy_row * sizeof(E) % b == 0));
    };
    if (fits(16 / sizeof(E))) return 16 / sizeof(E);
    return sizeof(E) == 2 && fits(2) ? 2 : 1;
}

template <typename E, int W>
cudaError_t by_length(const LayerNormArgs& a, bool back, int blocks, cudaStream_t s) {
    const int packs = a.D / W;
    if (packs <= 8) return run<E, W, 8, 1>(a, back, blocks, s);
    if (packs <= 32) return run<E, W, 32, 1>(a, back, blocks, s);
    if (packs <= 64) return run<E, W, 32, 2>(a, back, blocks, s);
    if (packs <= 128) return run<E, W, 32, 4>(a, back, blocks, s);
    if (packs <= 256) return run<E, W, 256, 1>(a, back, blocks, s);
    if (packs <= 512) return run<E, W, 256, 2>(a, back, blocks, s);
    if (packs <= 1024) return run<E, W, 256, 4>(a, back, blocks, s);
    if (!back) ln_fwd_long_kernel<E><<<a.N < 152 * 4 ? a.N : 152 * 4, kLongThreads, 0, s>>>(a);
    else ln_bwd_long_kernel<E><<<blocks, kLongThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t by_width(const LayerNormArgs& a, bool back, int blocks, cudaStream_t s) {
    const int w = pack_width<E>(a, back);
    if (w == 1) return by_length<E, 1>(a, back, blocks, s);
    if constexpr (sizeof(E) == 2)
        if (w == 2) return by_length<E, 2>(a, back, blocks, s);
    return by_length<E, 16 / (int)sizeof(E)>(a, back, blocks, s);
}

// Blocks of the gradient: as many as run at a time, fewer for few rows (each leaves 2 D
// partial sums).  A function of N and D alone, which the workspace size is too.
int bwd_blocks(int N, int D) {
    const int sets = D <= 8 ? 32 : (D <= 128 ? 8 : 1);
    const long long need = ((long long)N + sets - 1) / sets;
    return (int)(need < 1 ? 1 : (need < kMaxBlocks ? need : kMaxBlocks));
}

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int N, int D) {
    return (size_t)bwd_blocks(N, D) * 2 * D * sizeof(float);
}

cudaError_t layer_norm_fwd_launch(const LayerNormArgs& a, cudaStream_t s) {
    return a.bf16 ? by_width<__nv_bfloat16>(a, false, 0, s) : by_width<float>(a, false, 0, s);
}

cudaError_t layer_norm_bwd_launch(const LayerNormArgs& in, cudaStream_t s, int* launches) {
    LayerNormArgs a = in;
    if (!a.dw && !a.db) a.partial = nullptr;
    const int blocks = bwd_blocks(a.N, a.D);
    *launches = 1;
    if (a.N == 0) {
        *launches = 0;
        for (float* p : {a.dw, a.db})
            if (p) {
                const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)a.D * sizeof(float), s);
                if (e != cudaSuccess) return e;
            }
        return cudaSuccess;
    }
    const cudaError_t e =
        a.bf16 ? by_width<__nv_bfloat16>(a, true, blocks, s) : by_width<float>(a, true, blocks, s);
    if (e != cudaSuccess || !a.partial) return e;
    ln_join_kernel<<<(2 * a.D + 31) / 32, dim3(32, 16), 0, s>>>(a.partial, blocks, a.D, a.dw, a.db);
    *launches = 2;
    return cudaGetLastError();
}

}  // namespace ttm
