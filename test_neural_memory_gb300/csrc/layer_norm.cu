// Layer norm over the last axis and its gradient.
//
// Mathematics, per row of D values:
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  n = (x - mean) rstd,
//   y = n w + b;
// with u = dy w:
//   dx = rstd (u - sum u / D - n sum(u n) / D),
//   dw = sum over rows of dy n,  db = sum over rows of dy.
// x - mean is taken first in both directions, then times rstd: x rstd - mean rstd would lose what a row
// far from zero has in n (5e-4 of it at a mean of 1e4 times the spread).
//
// What bounds it: HBM, two tensors forward and three in the gradient.  A row is read
// once and stays in registers: the variance is taken about the mean (no difference of
// large sums), and the gradient's dw and db are added up in registers over the rows that
// a thread group walks, so x and dy are read once for all three results.
//
// Layout: TPR threads share a row, each K packs of W values that are TPR packs apart
// (every access of a warp is contiguous), ROWS rows at a time so that enough loads are
// in flight and one reduction serves several rows.  TPR is the rows' packs up to a warp
// (shuffles), or the whole block of 256 (shuffles, then shared memory) for long rows; a warp
// takes rows of up to 1024 single values, in which a block of 256 would mostly wait at barriers
// (697568 x 169 bf16, gradient: 679 us with a row a block, 250 with a row a warp) once there are many.  Rows longer
// than the registers hold are read again from the cache instead.  W is the widest pack that the
// rows' alignment and D allow; rows of x and dy that do not start on 16 bytes are read in 16-byte
// words all the same and shifted into place (238817 x 768 bf16 from rows of 771, forward: 318 us
// value by value, 137 so).
//
// Measured, forward and gradient: bf16 131072 x 2048 200 and 285 us (5.4 and 5.6 TB/s of 6.8 that a
// copy reaches), 786432 x 64 39 and 61 us, 100000 x 512 40 and 62 us, 8000 x 8192 60 and 112 us (its
// sums of dw and db take the registers of one of the two blocks an SM); fp32 65536 x 2048 151 and 243 us,
// 100000 x 512 65 and 102 us.  The figures further down compare variants with x as dy, one read less.
//
// The gradient's blocks leave their dw, db sums in the workspace and a second kernel adds
// them in a fixed order: no atomics, so equal inputs give equal bits.
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "pairs.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLongThreads = 512;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float v) { o = __float2bfloat16(v); }

// W neighbouring values as they are stored: whole 32-bit words, or one bf16 value.  Taken as
// kN items of type T, pairs for W > 1.
template <typename E, int W>
struct Pack {
    using Word = std::conditional_t<sizeof(E) * W == 2, unsigned short, uint32_t>;
    using T = std::conditional_t<W == 1, float, f2>;
    static constexpr int kN = W == 1 ? 1 : W / 2, kWords = sizeof(E) * W / sizeof(Word);
    struct alignas(sizeof(E) * W) Data {
        Word w[kWords];
    } d;

    __device__ __forceinline__ void load(const E* p) { d = *reinterpret_cast<const Data*>(p); }
    __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<Data*>(p) = d; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) d.w[i] = 0;
    }
    // Forgets the unpacked values: they are cheaper to take again than to keep in registers.
    __device__ __forceinline__ void repack() {
        if constexpr (sizeof(Word) == 4) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) asm volatile("" : "+r"(d.w[i]));
        }
    }
    __device__ __forceinline__ T get(int i) const {
        if constexpr (W == 1) {
            if constexpr (sizeof(E) == 2) return __uint_as_float((uint32_t)d.w[0] << 16);
            else return __uint_as_float(d.w[0]);
        } else if constexpr (sizeof(E) == 2) {
            return pair_of_bf16(d.w[i]);
        } else {
            return pair(__uint_as_float(d.w[2 * i]), __uint_as_float(d.w[2 * i + 1]));
        }
    }
    __device__ __forceinline__ void set(int i, T v) {
        if constexpr (W == 1) {
            if constexpr (sizeof(E) == 2) d.w[0] = __bfloat16_as_ushort(__float2bfloat16(v));
            else d.w[0] = __float_as_uint(v);
        } else if constexpr (sizeof(E) == 2) {
            d.w[i] = bf16_of_pair(v);
        } else {
            float lo, hi;
            split(v, lo, hi);
            d.w[2 * i] = __float_as_uint(lo);
            d.w[2 * i + 1] = __float_as_uint(hi);
        }
    }
};

// A pack on its way from global memory; kShift: from a row that does not start on 16 bytes.  That one
// is read in the aligned 16-byte words that hold a value of it, two as a rule (the second one a
// neighbour's first, so from L1), and shifted into place when it is taken.
template <typename E, int W, bool kShift>
struct Coming {
    Pack<E, W> p;
    __device__ __forceinline__ void zero() { p.zero(); }
    __device__ __forceinline__ void load(const E* at, int) { p.load(at); }
    __device__ __forceinline__ Pack<E, W> take(int) const { return p; }
};
template <typename E, int W>
struct Coming<E, W, true> {
    uint4 u, v;
    __device__ __forceinline__ void zero() { u = v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const E* at, int shift) {   // shift: of `at` past 16 bytes
        const uint4* w = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(at) - shift);
        u = w[0];
        if (shift) v = w[1];
    }
    __device__ __forceinline__ Pack<E, W> take(int shift) const {
        static_assert(sizeof(Pack<E, W>) == 16, "16 bytes");
        uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        if (shift & 8)
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        if (shift & 4)
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        Pack<E, W> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.d.w[i] = sizeof(E) == 4 ? w[i] : __funnelshift_r(w[i], w[i + 1], (shift & 3) * 8);
        return r;
    }
};
template <typename E>
__device__ __forceinline__ int shift_of(const E* row) {
    return (int)(reinterpret_cast<uintptr_t>(row) & 15);
}

// W weights (fp32, or `absent` each), 16 bytes at a time.
template <int W, typename T, int N>
__device__ __forceinline__ void load_weights(const float* p, T (&f)[N], float absent) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = splat<T>(absent);
        return;
    }
    if constexpr (W == 1) {
        f[0] = p[0];
    } else if constexpr (W == 2) {
        const float2 q = *reinterpret_cast<const float2*>(p);
        f[0] = pair(q.x, q.y);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float4 q = *reinterpret_cast<const float4*>(p + 2 * i);
            f[i] = pair(q.x, q.y);
            f[i + 1] = pair(q.z, q.w);
        }
    }
}

// Sums over the TPR threads of a row; TPR = kThreads goes through `buf` (shared), which
// the caller may use again after the next reduction's barrier.
template <int TPR, int C>
__device__ __forceinline__ void row_sums(float (&s)[C], float (*buf)[kWarps]) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int o = (TPR < 32 ? TPR : 32) / 2; o; o >>= 1)
            s[c] += __shfl_xor_sync(0xffffffffu, s[c], o);
    if (TPR > 32) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int c = 0; c < C; ++c) buf[c][threadIdx.x >> 5] = s[c];
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float4 a = *reinterpret_cast<const float4*>(&buf[c][0]);
            const float4 b = *reinterpret_cast<const float4*>(&buf[c][4]);
            s[c] = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
        }
    }
}

// s / d from inv = 1 / d and its remainder: the mean of equal values is that value, which s inv misses for
// some lengths (7, 60, 1000, 3001).  A division takes 25 % longer where a thread has little of a row.
__device__ __forceinline__ float divide(float s, float d, float inv) {
    const float q = s * inv, left = fmaf(-q, d, s);
    return left == left ? fmaf(left, inv, q) : q;       // an infinite sum stays one
}

template <typename E, int W, bool kShift, int TPR, int K, int ROWS>
__global__ void __launch_bounds__(kThreads) ln_fwd_kernel(const __grid_constant__ LayerNormArgs a) {
    using P = Pack<E, W>;
    using T = typename P::T;
    constexpr int kSets = kThreads / TPR, N = P::kN;  // rows side by side in a block
    __shared__ __align__(16) float buf[2][ROWS][kWarps];
    const int lane = threadIdx.x % TPR, set = threadIdx.x / TPR;
    const int packs = a.D / W;
    const float inv = 1.f / a.D;
    const E* x = static_cast<const E*>(a.x);
    const long long r0 = (long long)blockIdx.x * kSets * ROWS + set;   // rows r0 + i kSets
    Coming<E, W, kShift> coming[ROWS][K];
    P in[ROWS][K];
    float s[ROWS], mean[ROWS], rstd[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const E* row = x + (r0 + i * kSets) * a.x_row;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            coming[i][k].zero();
            if (r0 + i * kSets < a.N && lane + k * TPR < packs)
                coming[i][k].load(row + (lane + k * TPR) * W, shift_of(row));
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        T t = splat<T>(0.f);
        const int shift = shift_of(x + (r0 + i * kSets) * a.x_row);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            in[i][k] = coming[i][k].take(shift);
#pragma unroll
            for (int j = 0; j < N; ++j) t = add(t, in[i][k].get(j));
            in[i][k].repack();
        }
        s[i] = total(t);
    }
    row_sums<TPR>(s, buf[0]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        mean[i] = divide(s[i], (float)a.D, inv);
        T t = splat<T>(0.f);
        const T m = splat<T>(-mean[i]);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (lane + k * TPR < packs)
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const T d = add(in[i][k].get(j), m);
                    t = fma(d, d, t);
                }
            in[i][k].repack();
        }
        s[i] = total(t);
    }
    row_sums<TPR>(s, buf[1]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) rstd[i] = 1.f / sqrtf(fmaf(s[i], inv, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (lane + k * TPR) * W;
        if (lane + k * TPR >= packs) continue;
        T w[N], b[N];
        load_weights<W>(a.w ? a.w + c : nullptr, w, 1.f);
        load_weights<W>(a.b ? a.b + c : nullptr, b, 0.f);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets;
            if (r >= a.N) continue;
            const T m = splat<T>(-mean[i]), q = splat<T>(rstd[i]);
            P out;
#pragma unroll
            for (int j = 0; j < N; ++j)
                out.set(j, fma(mul(add(in[i][k].get(j), m), q), w[j], b[j]));
            out.store(static_cast<E*>(a.y) + r * a.D + c);
        }
    }
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets;
            if (r >= a.N) continue;
            if (a.mean) a.mean[r] = mean[i];
            if (a.rstd) a.rstd[r] = rstd[i];
        }
}

template <typename E, int W, bool kShift, int TPR, int K, int ROWS, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) ln_bwd_kernel(const __grid_constant__ LayerNormArgs a) {
    using P = Pack<E, W>;
    using T = typename P::T;
    constexpr int kSets = kThreads / TPR, N = P::kN;
    __shared__ __align__(16) float buf[2][2 * ROWS][kWarps];
    const int lane = threadIdx.x % TPR, set = threadIdx.x / TPR;
    const int packs = a.D / W;
    const float inv = 1.f / a.D;
    const E *x = static_cast<const E*>(a.x), *dy = static_cast<const E*>(a.dy);
    T dw[K][N], db[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) dw[k][j] = db[k][j] = splat<T>(0.f);
    // the next rows are asked for before the reduction of these
    Coming<E, W, kShift> nx[ROWS][K], nd[ROWS][K];
    float nmean[ROWS], nrstd[ROWS];
    auto fetch = [&](long long r0) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets + set;
            const bool in = r < a.N;
            const E *xr = x + r * a.x_row, *dr = dy + r * a.dy_row;
            nmean[i] = in ? a.mean[r] : 0.f;
            nrstd[i] = in ? a.rstd[r] : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (lane + k * TPR) * W;
                nx[i][k].zero();
                nd[i][k].zero();
                if (in && lane + k * TPR < packs) {
                    nx[i][k].load(xr + c, shift_of(xr));
                    nd[i][k].load(dr + c, shift_of(dr));
                }
            }
        }
    };
    constexpr bool kAhead = K * W <= 32;                // or the registers are full
    int turn = 0;
    const long long stride = (long long)gridDim.x * kSets * ROWS;
    if (kAhead) fetch((long long)blockIdx.x * kSets * ROWS);
    for (long long r0 = (long long)blockIdx.x * kSets * ROWS; r0 < a.N; r0 += stride, turn ^= 1) {
        if (!kAhead) fetch(r0);
        P px[ROWS][K], pd[ROWS][K];
        float mean[ROWS], rstd[ROWS], s[2 * ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const long long r = r0 + i * kSets + set;
            const int sx = shift_of(x + r * a.x_row), sd = shift_of(dy + r * a.dy_row);
            mean[i] = nmean[i];
            rstd[i] = nrstd[i];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                px[i][k] = nx[i][k].take(sx);
                pd[i][k] = nd[i][k].take(sd);
            }
        }
        if (kAhead) fetch(r0 + stride);
        T su[ROWS], sn[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) su[i] = sn[i] = splat<T>(0.f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            T w[N];
            load_weights<W>(a.w && lane + k * TPR < packs ? a.w + (lane + k * TPR) * W : nullptr, w, 1.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const T q = splat<T>(rstd[i]), m = splat<T>(-mean[i]);
#pragma unroll
                for (int j = 0; j < N; ++j) {           // absent rows and columns have dy = 0
                    const T g = pd[i][k].get(j), d = add(px[i][k].get(j), m), u = mul(g, w[j]);
                    db[k][j] = add(db[k][j], g);
                    dw[k][j] = fma(mul(g, q), d, dw[k][j]);
                    su[i] = add(su[i], u);
                    sn[i] = fma(u, d, sn[i]);           // sum(u n) / rstd
                }
                px[i][k].repack();
                pd[i][k].repack();
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            s[2 * i] = total(su[i]);
            s[2 * i + 1] = total(sn[i]);
        }
        row_sums<TPR>(s, buf[turn]);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (lane + k * TPR) * W;
            if (lane + k * TPR >= packs) continue;
            T w[N];
            load_weights<W>(a.w ? a.w + c : nullptr, w, 1.f);
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const long long r = r0 + i * kSets + set;
                if (r >= a.N) continue;
                // rstd (u - su - n sn)
                const T q = splat<T>(rstd[i]), m = splat<T>(-mean[i]), c0 = splat<T>(-s[2 * i] * inv);
                const T c1 = splat<T>(-s[2 * i + 1] * rstd[i] * inv * rstd[i]);
                P out;
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const T d = add(px[i][k].get(j), m);
                    out.set(j, mul(q, fma(d, c1, fma(pd[i][k].get(j), w[j], c0))));
                }
                out.store(static_cast<E*>(a.dx) + r * a.D + c);
            }
        }
    }
    if (!a.partial) return;
    // over the rows side by side in the block: sets of a warp by shuffles, warps through shared
    // memory (one warp or more per row: the sets are whole warps)
    float* part = a.partial + (size_t)blockIdx.x * 2 * a.D;
    extern __shared__ float sums[];                     // TPR < kThreads: [kWarps][2][TPR K W]
    const int cols = TPR * K * W, warp = threadIdx.x >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float v[2][2];                              // [dw, db][first, second of the item]
            if constexpr (W == 1) {
                v[0][0] = dw[k][j];
                v[1][0] = db[k][j];
            } else {
                split(dw[k][j], v[0][0], v[0][1]);
                split(db[k][j], v[1][0], v[1][1]);
            }
#pragma unroll
            for (int e = 0; e < (W == 1 ? 1 : 2); ++e) {
                const int c = (lane + k * TPR) * W + 2 * j + e;
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    if (TPR == kThreads) {
                        if (lane + k * TPR < packs) part[z * a.D + c] = v[z][e];
                    } else {
#pragma unroll
                        for (int o = TPR; o < 32; o <<= 1)
                            v[z][e] += __shfl_xor_sync(0xffffffffu, v[z][e], o);
                        if ((threadIdx.x & 31) < TPR) sums[(warp * 2 + z) * cols + c] = v[z][e];
                    }
                }
            }
        }
    if (TPR == kThreads) return;
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.D; c += kThreads) {
        const int which = c >= a.D, col = c - which * a.D;
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += sums[(w * 2 + which) * cols + col];
        part[c] = t;
    }
}

// Rows longer than the registers: one block per row, values read again from the cache.  Columns count in
// 64 bits: 2 D passes 31 of them, and the last stride past D 32.
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
        for (long long d = threadIdx.x; d < a.D; d += kLongThreads) s += to_f(x[d]);
        const float mean = block_sum<E>(s, buf) / a.D;
        s = 0.f;
        for (long long d = threadIdx.x; d < a.D; d += kLongThreads) {
            const float c = to_f(x[d]) - mean;
            s = fmaf(c, c, s);
        }
        const float rstd = 1.f / sqrtf(block_sum<E>(s, buf) / a.D + a.eps);
        for (long long d = threadIdx.x; d < a.D; d += kLongThreads)
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
        for (long long d = threadIdx.x; d < 2ll * a.D; d += kLongThreads) part[d] = 0.f;
    __syncthreads();
    for (long long r = blockIdx.x; r < a.N; r += gridDim.x) {
        const E* x = static_cast<const E*>(a.x) + r * a.x_row;
        const E* dy = static_cast<const E*>(a.dy) + r * a.dy_row;
        const float mean = a.mean[r], rstd = a.rstd[r];
        float su = 0.f, sn = 0.f;
        for (long long d = threadIdx.x; d < a.D; d += kLongThreads) {
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
        for (long long d = threadIdx.x; d < a.D; d += kLongThreads) {
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
    const long long c = blockIdx.x * 32ll + threadIdx.x;
    float s = 0.f;
    if (c < 2ll * D)
        for (int p = threadIdx.y; p < blocks; p += 16) s += part[p * 2ll * D + c];
    buf[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= 2ll * D) return;
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

// Gradient: two blocks an SM with two rows each in flight and two more on the way.  At 131072 x
// 2048 bf16: 284 us; 300 us with one block of four rows, 314 with three of one row, 420 with
// four (their registers spill).
constexpr int kResident = 2;
constexpr int kMaxBlocks = 152 * kResident;

// Whether the gradient shifts rows into place: fp32 rows read value by value, which need half the
// registers on the way, are faster between these lengths (100000 x 512: 94 us against 122, 16000 x
// 4096: 132 and 209; but 1000000 x 24: 137 and 93).
template <typename E>
constexpr bool shift_pays(int D) {
    return sizeof(E) == 2 || D <= 32 || D > 4096;
}

template <typename E, int W, bool kShift, int TPR, int K>
cudaError_t run(const LayerNormArgs& a, bool back, int blocks, cudaStream_t s) {
    constexpr int sets = kThreads / TPR, word = W * (int)sizeof(E) < 4 ? 4 : W * (int)sizeof(E);
    constexpr int bytes = K * word;                     // of registers for a row
    if (!back) {
        constexpr int rows = bytes >= 64 ? 1 : (bytes >= 32 ? 2 : 4);   // 64 bytes in flight a thread
        const long long need = ((long long)a.N + sets * rows - 1) / (sets * rows);
        ln_fwd_kernel<E, W, kShift, TPR, K, rows><<<(unsigned)need, kThreads, 0, s>>>(a);
    } else if constexpr (kShift ? shift_pays<E>(TPR * K * W) : W > 2 || TPR > 32 || K * W < 32) {
        constexpr int rows = bytes > (kShift ? 16 : 32) || K * W > 8 ? 1 : 2;
        constexpr int resident = K * W <= (kShift ? 8 : 16) ? kResident : 1;
        // The limit is what a call with dw or db needs, also for one without: calls of two host threads
        // set the same
        constexpr int most = TPR == kThreads ? 0 : kWarps * 2 * TPR * K * W * 4;
        const size_t shared = a.partial ? most : 0;
        auto kernel = ln_bwd_kernel<E, W, kShift, TPR, K, rows, resident>;
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        kernel<<<blocks, kThreads, shared, s>>>(a);
    }
    return cudaGetLastError();
}

// Widest pack the rows allow: 16 bytes (0: shifted into place, where only the outputs' rows start on
// 16 bytes), 4 bytes, one value.
template <typename E>
int pack_width(const LayerNormArgs& a, bool back) {
    auto fits = [&](int w) {
        const unsigned long long b = w * sizeof(E);
        if (a.D % w || reinterpret_cast<uintptr_t>(a.x) % b || (a.N > 1 && a.x_row * sizeof(E) % b))
            return false;
        return !back || (reinterpret_cast<uintptr_t>(a.dy) % b == 0 &&
                         (a.N <= 1 || a.dy_row * sizeof(E) % b == 0));
    };
    if (a.D % (16 / sizeof(E)) == 0 && fits(16 / sizeof(E))) return 16 / sizeof(E);
    if (a.D % (16 / sizeof(E)) == 0 && (!back || shift_pays<E>(a.D))) return 0;
    return sizeof(E) == 2 && fits(2) ? 2 : 1;
}

// Rows of more than 128 values or pairs, a warp each: with enough of them, or a block a row has more
// loads in flight (1537 x 500 bf16 in odd rows: 4.0 and 7.9 us by blocks, 5.7 and 9.6 by warps; 12000: 13.9
// and 21.6, 9.8 and 18.1).  In the gradient a warp's registers do not reach for 32 values a thread
// (48000 x 900: 91 us, 78 by blocks).
constexpr int kManyRows = 4096;
template <typename E, int W, bool kShift = false>
cudaError_t by_length(const LayerNormArgs& a, bool back, int blocks, cudaStream_t s) {
    const int packs = a.D / W;
    if (packs <= 4) return run<E, W, kShift, 4, 1>(a, back, blocks, s);
    if (packs <= 8) return run<E, W, kShift, 8, 1>(a, back, blocks, s);
    if (packs <= 16) return run<E, W, kShift, 16, 1>(a, back, blocks, s);
    if (packs <= 32) return run<E, W, kShift, 32, 1>(a, back, blocks, s);
    if (packs <= 64) return run<E, W, kShift, 32, 2>(a, back, blocks, s);
    if constexpr (W > 2)
        if (packs <= 96) return run<E, W, kShift, 32, 3>(a, back, blocks, s);
    if (packs <= 128) return run<E, W, kShift, 32, 4>(a, back, blocks, s);
    if constexpr (W <= 2) {
        if (a.N >= kManyRows) {
            if (packs <= 256) return run<E, W, kShift, 32, 8>(a, back, blocks, s);
            if (packs <= 512 && !(back && W == 2)) return run<E, W, kShift, 32, 16>(a, back, blocks, s);
            if constexpr (W == 1)
                if (packs <= 1024 && !back) return run<E, W, kShift, 32, 32>(a, back, blocks, s);
        }
        if (packs <= 256) return run<E, W, kShift, 256, 1>(a, back, blocks, s);
        if (packs <= 512) return run<E, W, kShift, 256, 2>(a, back, blocks, s);
        if (packs <= 1024) return run<E, W, kShift, 256, 4>(a, back, blocks, s);
        if (packs <= 2048) return run<E, W, kShift, 256, 8>(a, back, blocks, s);
        if (packs <= 4096) return run<E, W, kShift, 256, 16>(a, back, blocks, s);
    } else {
        if (packs <= 256) return run<E, W, kShift, 256, 1>(a, back, blocks, s);
        if (packs <= 512) return run<E, W, kShift, 256, 2>(a, back, blocks, s);
        if (packs <= 1024) return run<E, W, kShift, 256, 4>(a, back, blocks, s);
        if constexpr (W == 4 || !kShift)
            if (packs <= 2048) return run<E, W, kShift, 256, 8>(a, back, blocks, s);
    }
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
    if (w == 0) return by_length<E, 16 / (int)sizeof(E), true>(a, back, blocks, s);
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
    ln_join_kernel<<<(unsigned)((2ll * a.D + 31) / 32), dim3(32, 16), 0, s>>>(a.partial, blocks, a.D, a.dw, a.db);
    *launches = 2;
    return cudaGetLastError();
}

}  // namespace ttm
