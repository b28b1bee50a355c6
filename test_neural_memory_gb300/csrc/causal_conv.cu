// Short causal convolution, depthwise, with an optional SiLU, per sequence and channel:
//   pre_t = b + sum_i w[i] x_{t-K+1+i},   y_t = pre_t or pre_t / (1 + exp(-pre_t)),
// rows before the first from a state (the last K - 1 inputs) or zero, taps whose row is of another
// document than the token left out; its gradient
//   d_t = dy_t act'(pre_t),  dx_s = sum_i w[i] d_{s+K-1-i},  dw[i] = sum_t d_t x_{t-K+1+i},  db = sum_t d_t;
// and its form for a few tokens on a resident state.
//
// Bound by HBM: two tensors forward, three in the gradient, K products and one exponential a value.  So
// every value is read once (but for the K - 1 rows between strips) and the window stays in registers: a
// thread takes V neighbouring channels, as wide as the rows' alignment allows, and walks a strip of
// tokens, the loads of kBatch rows ahead of their use.  Measured (K = 4, bf16, SiLU): forward 131072 x 6144 540 us, 6.0 TB/s,
// 89 % of a copy; gradient 8 x 8192 x 2304 174 us, 5.2 TB/s, its 26 instructions a value and three blocks of registers
// an SM as much the bound as the memory; a step of 64 x 6144 4.6 to 5.0 us, of which the GPU's part is a launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "conv_plan.h"
#include "overlap.cuh"
#include "pairs.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kBatch = kConvBatch, kFwdThreads = kConvThreads, kBwdThreads = kConvThreads;
// Blocks of the gradient an SM, by registers (8 x 8192 x 2304 bf16 in pairs of values: 212 us with 4, 278 with 3).
template <int V, int KW> constexpr int kBwdBlocks = V <= 2 && KW <= 4 ? 4 : 3;

// V values of a row as they are stored, and as fp32: pairs of values (two results an instruction), or one.
template <int BYTES> struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };
template <typename T, int V> using Raw = typename Word<sizeof(T) * V>::type;
template <int V> struct Lanes { static constexpr int n = V / 2; using type = f2; };
template <> struct Lanes<1> { static constexpr int n = 1; using type = float; };
template <int V> using Val = typename Lanes<V>::type;
template <int V> constexpr int kVals = Lanes<V>::n;

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load(const T* p) {
    return *reinterpret_cast<const Raw<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& raw, Val<V> (&f)[kVals<V>]) {
    if constexpr (sizeof(T) == 4) {
        const float* s = reinterpret_cast<const float*>(&raw);
        if constexpr (V == 1) {
            f[0] = s[0];
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) f[i] = pair(s[2 * i], s[2 * i + 1]);
        }
    } else if constexpr (V == 1) {
        f[0] = __uint_as_float((uint32_t)raw << 16);
    } else {
        const uint32_t* s = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) f[i] = pair_of_bf16(s[i]);
    }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const Val<V> (&f)[kVals<V>]) {
    Raw<T, V> raw;
    if constexpr (sizeof(T) == 4) {
        float* d = reinterpret_cast<float*>(&raw);
        if constexpr (V == 1) {
            d[0] = f[0];
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) split(f[i], d[2 * i], d[2 * i + 1]);
        }
    } else if constexpr (V == 1) {
        raw = __bfloat16_as_ushort(__float2bfloat16_rn(f[0]));
    } else {
        uint32_t* d = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) d[i] = bf16_of_pair(f[i]);
    }
    *reinterpret_cast<Raw<T, V>*>(p) = raw;
}
// A value of 4, 8 or 16 bytes into shared memory, asynchronously.
template <typename R, typename T>
__device__ __forceinline__ void copy_async(R* to, const T* from) {
    if constexpr (sizeof(R) >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                     "n"(sizeof(R))
                     : "memory");
}
template <int V>
__device__ __forceinline__ Val<V> gather(const float* p, long long step) {     // the values of neighbouring channels
    if constexpr (V == 1) return p[0];
    else return pair(p[0], p[step]);
}
// The K taps of V channels from c on, tap i in slot i + KW - K.  kAll: four taps on 16 bytes.
template <int V, int KW, bool kAll>
__device__ __forceinline__ void load_taps(Val<V> (&w)[KW][kVals<V>], const float* p, int c, int K) {
    constexpr int step = V / kVals<V>;
#pragma unroll
    for (int v = 0; v < kVals<V>; ++v) {
        if constexpr (kAll) {
            const float4 a = reinterpret_cast<const float4*>(p)[c + step * v];
            if constexpr (V == 1) {
                w[0][v] = a.x; w[1][v] = a.y; w[2][v] = a.z; w[3][v] = a.w;
            } else {
                const float4 b = reinterpret_cast<const float4*>(p)[c + step * v + 1];
                w[0][v] = pair(a.x, b.x); w[1][v] = pair(a.y, b.y); w[2][v] = pair(a.z, b.z); w[3][v] = pair(a.w, b.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < KW; ++i)
                w[i][v] = i >= KW - K ? gather<V>(p + (long long)(c + step * v) * K + i - (KW - K), K) : splat<Val<V>>(0.f);
        }
    }
}
template <typename E> __device__ __forceinline__ E zero() { return splat<E>(0.f); }

// 1 / (1 + exp(-x)); the fast one for bf16 results.
template <typename T>
__device__ __forceinline__ float sigmoid(float x) {
    if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-x));
    else return fast_logistic(x);
}
template <typename T>
__device__ __forceinline__ f2 sigmoid(f2 x) {
    float a, b;
    split(x, a, b);
    return pair(sigmoid<T>(a), sigmoid<T>(b));
}

// What a thread walks: rows of one sequence, its V channels.
template <typename T>
struct Rows {
    const T* x;                         // row 0, first channel
    long long tok;
    const T* state;                     // [K-1][C] of this sequence, first channel, or NULL
    int C, K;
    template <int V>
    __device__ __forceinline__ Raw<T, V> at(int t) const {           // rows before 0 from the state
        if (t >= 0) return load<T, V>(x + (long long)t * tok);
        const int s = t + K - 1;
        if (state && s >= 0) return load<T, V>(state + (long long)s * C);
        return Raw<T, V>{};
    }
};

// KW: the window, K at most (kAll: K itself); tap i of K sits in slot i + KW - K, slots before it take no part.
// kOne: every row of the window is of the token's document.
template <int V, int KW, bool kAll, bool kOne>
__device__ __forceinline__ void taps(Val<V> (&out)[kVals<V>], const Val<V> (&w)[KW][kVals<V>],
                                     const Val<V> (&win)[KW][kVals<V>], const int (&id)[KW], int before) {
#pragma unroll
    for (int i = 0; i < KW; ++i) {
        if ((!kAll && i < before) || (!kOne && id[i] != id[KW - 1])) continue;
#pragma unroll
        for (int v = 0; v < kVals<V>; ++v) out[v] = fma(w[i][v], win[i][v], out[v]);
    }
}

// A strip of tokens a thread; the thread of a sequence's last strip writes the state.  `strips` = 1
// lets the state be updated in place.
template <typename T, int V, int KW, bool kAll, bool DOC>
__global__ void __launch_bounds__(kFwdThreads) conv_fwd_kernel(const __grid_constant__ ConvArgs a, unsigned groups,
                                                                unsigned strips, int strip) {
    constexpr int NV = kVals<V>;
    const unsigned long long id = (unsigned long long)blockIdx.x * kFwdThreads + threadIdx.x;
    unsigned group, part, n;
    if (id >> 32) {
        const unsigned long long rest = id / groups;
        group = (unsigned)(id - rest * groups);
        n = (unsigned)(rest / strips);
        part = (unsigned)(rest - (unsigned long long)n * strips);
    } else {
        const unsigned rest = (unsigned)id / groups;
        group = (unsigned)id - rest * groups;
        n = rest / strips;
        part = rest - n * strips;
    }
    after_all_before();
    if (n >= (unsigned)a.N) return;
    const int c = (int)group * V, K = a.K, C = a.C, before = kAll ? 0 : KW - K;
    const int t0 = (int)part * strip, t1 = conv_strip_end(a.T, t0, strip);
    const Rows<T> rows{static_cast<const T*>(a.x) + n * a.x_seq + c, a.x_tok,
                       a.state0 ? static_cast<const T*>(a.state0) + (long long)n * (K - 1) * C + c : nullptr, C, K};
    const int* doc = DOC ? a.doc + n * a.doc_seq : nullptr;
    Raw<T, V> next[kBatch];
    int next_id[kBatch];
    const T* from = rows.x + (long long)t0 * rows.tok;
    auto fetch = [&](int t) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (t + j < t1) {
                next[j] = load<T, V>(from);
                if (DOC) next_id[j] = doc[t + j];
            }
            from += rows.tok;
        }
    };
    fetch(t0);
    Val<V> w[KW][NV], bias[NV], win[KW][NV];            // win: slots up to KW - 2 the rows before the token
    int ids[KW];
#pragma unroll
    for (int i = 1; i < KW; ++i) {
        const int t = t0 - KW + i;
        Raw<T, V> raw{};
        if (i > before) raw = rows.template at<V>(t);
        unpack<T, V>(raw, win[i]);
        if (DOC) ids[i] = doc[max(t, 0)];
    }
    load_taps<V, KW, kAll>(w, a.w, c, K);
#pragma unroll
    for (int v = 0; v < NV; ++v) bias[v] = a.b ? gather<V>(a.b + c + v * (V / NV), 1) : zero<Val<V>>();
    T* y = static_cast<T*>(a.y) + ((long long)n * a.T + t0) * C + c;
    auto token = [&](auto one, const Raw<T, V>& raw, int raw_id) {
#pragma unroll
        for (int i = 0; i + 1 < KW; ++i) {
#pragma unroll
            for (int v = 0; v < NV; ++v) win[i][v] = win[i + 1][v];
            if (DOC) ids[i] = ids[i + 1];
        }
        unpack<T, V>(raw, win[KW - 1]);
        if (DOC) ids[KW - 1] = raw_id;
        Val<V> out[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) out[v] = bias[v];
        taps<V, KW, kAll, decltype(one)::value>(out, w, win, ids, before);
        if (a.silu) {
#pragma unroll
            for (int v = 0; v < NV; ++v) out[v] = mul(out[v], sigmoid<T>(out[v]));
        }
        store<T, V>(y, out);
        y += C;
    };
    int t = t0;
    for (; t + kBatch <= t1; t += kBatch) {             // whole batches: the window stays in place
        Raw<T, V> raw[kBatch];
        int raw_id[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            raw[j] = next[j];
            raw_id[j] = DOC ? next_id[j] : 0;
        }
        fetch(t + kBatch);
        bool one = true;                // the window and the batch are of one document
        if (DOC) {
#pragma unroll
            for (int i = 1; i + 1 < KW; ++i) one &= ids[i] == ids[KW - 1];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) one &= raw_id[j] == ids[KW - 1];
        }
        if (one) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) token(std::true_type{}, raw[j], raw_id[j]);
        } else if constexpr (DOC) {
#pragma unroll 1
            for (int j = 0; j < kBatch; ++j) {          // (one copy of the code for the few batches with a border)
                Raw<T, V> r = raw[0];
                int id = raw_id[0];
#pragma unroll
                for (int i = 1; i < kBatch; ++i)
                    if (j == i) { r = raw[i]; id = raw_id[i]; }
                token(std::false_type{}, r, id);
            }
        }
    }
#pragma unroll
    for (int j = 0; j + 1 < kBatch; ++j)
        if (t + j < t1) token(std::integral_constant<bool, !DOC>{}, next[j], DOC ? next_id[j] : 0);
    if (a.state && part + 1 == strips) {
        T* s = static_cast<T*>(a.state) + (long long)n * (K - 1) * C + c;
#pragma unroll
        for (int i = 1; i < KW; ++i) {
            if (i <= before) continue;
            Val<V> f[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) f[v] = !DOC || ids[i] == ids[KW - 1] ? win[i][v] : zero<Val<V>>();
            store<T, V>(s + (long long)(i - before - 1) * C, f);
        }
    }
}

// T = 0: the state passes on as it came.
template <typename T>
__global__ void conv_pass_kernel(const T* from, T* to, long long n) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : T(0.f);
}

// A thread walks strips of V channels, KW - 1 tokens past each strip's end, and row t - KW + 1 leaves once d_t
// is known (the d of those tokens are computed twice, their share of dw only by the strip that they are in).  A
// block is bx threads of neighbouring channels by as many strips as it has threads left.  dw and db are added up
// in registers over a thread's strips, over the block's threads in shared memory in their order, and leave as
// one part of the block's row of the grid, joined by conv_join_kernel in the rows' order: equal inputs give
// equal bits.
template <typename T, int V, int KW, bool kAll, bool DOC>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks<V, KW>)
    conv_bwd_kernel(const __grid_constant__ ConvArgs a, int groups, int strips, int strip) {
    constexpr int NV = kVals<V>;
    using E = Val<V>;
    constexpr bool kRing = sizeof(Raw<T, V>) >= 4;      // (asynchronous copies take 4 bytes at least)
    constexpr int kDeep = 4;                            // batches of rows on their way, or in the ring
    __shared__ Raw<T, V> ring[kRing ? kDeep * kBatch * 2 : 1][kBwdThreads];
    __shared__ float sums[kBwdThreads * V];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int K = a.K, C = a.C, before = kAll ? 0 : KW - K;
    const unsigned group = blockIdx.x * blockDim.x + threadIdx.x;     // (the last block's may pass 2^31)
    const bool live = group < (unsigned)groups;
    const int c = live ? (int)group * V : 0;
    after_all_before();
    E w[KW][NV], bias[NV], dw[KW][NV], db[NV];
    load_taps<V, KW, kAll>(w, a.w, c, K);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        bias[v] = a.b ? gather<V>(a.b + c + v * (V / NV), 1) : zero<E>();
        db[v] = zero<E>();
#pragma unroll
        for (int i = 0; i < KW; ++i) dw[i][v] = zero<E>();
    }
    const long long total = live ? (long long)a.N * strips : 0;
    for (long long s = (long long)blockIdx.y * blockDim.y + threadIdx.y; s < total;
         s += (long long)gridDim.y * blockDim.y) {
        const long long n = s / strips;
        const int t0 = (int)(s % strips) * strip, t1 = conv_strip_end(a.T, t0, strip), end = min(a.T, t1 + KW - 1);
        const Rows<T> rows{static_cast<const T*>(a.x) + n * a.x_seq + c, a.x_tok,
                           a.state0 ? static_cast<const T*>(a.state0) + n * (K - 1) * C + c : nullptr, C, K};
        const int* doc = DOC ? a.doc + n * a.doc_seq : nullptr;
        const int id_last = DOC ? doc[a.T - 1] : 0;
        T* dx = static_cast<T*>(a.dx) + n * a.T * (long long)C + c;
        T* ds0 = a.dstate0 ? static_cast<T*>(a.dstate0) + n * (K - 1) * C + c : nullptr;
        const T* ds = a.dstate ? static_cast<const T*>(a.dstate) + n * (K - 1) * C + c : nullptr;
        const int first_row = t0 == 0 && ds0 ? -(K - 1) : t0;
        Raw<T, V> next[kBatch], dnext[kBatch];
        int next_id[kBatch];
        const T *from = rows.x + (long long)t0 * rows.tok, *dfrom = static_cast<const T*>(a.dy) + n * a.dy_seq + (long long)t0 * a.dy_tok + c;
        int slot = 0;
        // Rows t .. t + kBatch - 1 on their way: into this thread's places of the ring, or registers.
        auto fetch = [&](int t) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (t + j < end) {
                    if constexpr (kRing) {
                        copy_async(&ring[(slot * kBatch + j) * 2][tid], from);
                        copy_async(&ring[(slot * kBatch + j) * 2 + 1][tid], dfrom);
                    } else {
                        next[j] = load<T, V>(from);
                        dnext[j] = load<T, V>(dfrom);
                        if (DOC) next_id[j] = doc[t + j];
                    }
                }
                from += rows.tok;
                dfrom += a.dy_tok;
            }
            if constexpr (kRing) asm volatile("cp.async.commit_group;" ::: "memory");
            slot = slot + 1 == kDeep ? 0 : slot + 1;
        };
        fetch(t0);
        if constexpr (kRing) {
#pragma unroll
            for (int i = 1; i < kDeep; ++i) fetch(t0 + i * kBatch);
        }
        E win[KW][NV], d[KW][NV];       // rows t - KW + 1 .. t and their d
        int ids[KW];
#pragma unroll
        for (int i = 0; i < KW; ++i) {
            const int t = t0 - KW + i;
            Raw<T, V> raw{};
            if (i > before) raw = rows.template at<V>(t);
            unpack<T, V>(raw, win[i]);
            if (DOC) ids[i] = doc[max(t, 0)];
#pragma unroll
            for (int v = 0; v < NV; ++v) d[i][v] = zero<E>();
        }
        // One token: kInner where it is of the strip, its row to leave too, neither is next to an end, and all of the
        // window is of one document.
        auto token = [&](auto inner, int now, const Raw<T, V>& raw, const Raw<T, V>& draw, int raw_id) {
            constexpr bool kInner = decltype(inner)::value;
            const int row = now - (KW - 1);
#pragma unroll
            for (int i = 0; i + 1 < KW; ++i) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    win[i][v] = win[i + 1][v];
                    d[i][v] = d[i + 1][v];
                }
                if (DOC) ids[i] = ids[i + 1];
            }
            if (kInner || now < end) {
                unpack<T, V>(raw, win[KW - 1]);
                unpack<T, V>(draw, d[KW - 1]);
                if (DOC) ids[KW - 1] = raw_id;
                if (a.silu) {
                    E pre[NV];
#pragma unroll
                    for (int v = 0; v < NV; ++v) pre[v] = bias[v];
                    taps<V, KW, kAll, kInner || !DOC>(pre, w, win, ids, before);
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        const E g = sigmoid<T>(pre[v]);
                        // 1 + pre (1 - g)
                        const E up = fma(pre[v], fma(g, splat<E>(-1.f), splat<E>(1.f)), splat<E>(1.f));
                        d[KW - 1][v] = mul(d[KW - 1][v], mul(g, up));
                    }
                }
                if (kInner || now < t1) {
#pragma unroll
                    for (int i = 0; i < KW; ++i) {
                        if ((!kAll && i < before) || (DOC && !kInner && ids[i] != ids[KW - 1])) continue;
#pragma unroll
                        for (int v = 0; v < NV; ++v) dw[i][v] = fma(d[KW - 1][v], win[i][v], dw[i][v]);
                    }
#pragma unroll
                    for (int v = 0; v < NV; ++v) db[v] = add(db[v], d[KW - 1][v]);
                }
            } else {                    // past the sequence, or past what the strip's rows need
#pragma unroll
                for (int v = 0; v < NV; ++v) d[KW - 1][v] = zero<E>();
                if (DOC) ids[KW - 1] = id_last;
            }
            if (kInner || (row >= first_row && row < t1)) {
                // row + m met row in its tap K - 1 - m, slot KW - 1 - m
                E out[NV];
#pragma unroll
                for (int v = 0; v < NV; ++v) out[v] = zero<E>();
#pragma unroll
                for (int m = 0; m < KW; ++m) {
                    if ((!kAll && m >= K) || (DOC && !kInner && ids[m] != ids[0])) continue;
#pragma unroll
                    for (int v = 0; v < NV; ++v) out[v] = fma(w[KW - 1 - m][v], d[m][v], out[v]);
                }
                if constexpr (!kInner) {
                    const int tail = row - (a.T - (K - 1));
                    if (ds && tail >= 0 && (!DOC || ids[0] == id_last)) {
                        E f[NV];
                        unpack<T, V>(load<T, V>(ds + (long long)tail * C), f);
#pragma unroll
                        for (int v = 0; v < NV; ++v) out[v] = add(out[v], f[v]);
                    }
                }
                store<T, V>(kInner || row >= 0 ? dx + (long long)row * C : ds0 + (long long)(row + K - 1) * C, out);
            }
        };
        // rows up to t1 - KW leave within the strip: before T - K + 1, where dstate begins
        for (int t = t0; t < t1 + KW - 1; t += kBatch) {
            Raw<T, V> raw[kBatch], draw[kBatch];
            int raw_id[kBatch];
            if constexpr (kRing) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    raw[j] = ring[(slot * kBatch + j) * 2][tid];
                    draw[j] = ring[(slot * kBatch + j) * 2 + 1][tid];
                    raw_id[j] = DOC && t + j < end ? doc[t + j] : 0;
                }
                fetch(t + kDeep * kBatch);
            } else {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    raw[j] = next[j];
                    draw[j] = dnext[j];
                    raw_id[j] = DOC ? next_id[j] : 0;
                }
                fetch(t + kBatch);
            }
            bool inner = t - (KW - 1) >= t0 && t + kBatch <= t1;
            if (DOC) {
#pragma unroll
                for (int i = 1; i + 1 < KW; ++i) inner &= ids[i] == ids[KW - 1];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) inner &= raw_id[j] == ids[KW - 1];
            }
            if (inner) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) token(std::true_type{}, t + j, raw[j], draw[j], raw_id[j]);
            } else {
#pragma unroll 1
                for (int j = 0; j < kBatch; ++j) {      // (one copy of the code for the few tokens at the ends)
                    Raw<T, V> r = raw[0], q = draw[0];
                    int id = raw_id[0];
#pragma unroll
                    for (int i = 1; i < kBatch; ++i)
                        if (j == i) { r = raw[i]; q = draw[i]; id = raw_id[i]; }
                    token(std::false_type{}, t + j, r, q, id);
                }
            }
        }
        if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    if (!a.partial) return;
    const int bx = blockDim.x;
    float* to = a.partial + (size_t)blockIdx.y * (K + 1) * C;
#pragma unroll
    for (int q = 0; q <= KW; ++q) {     // tap slots, then db
        if (q < before) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const E x = q < KW ? dw[q < KW ? q : 0][v] : db[v];
            if constexpr (V == 1) sums[tid] = x;
            else split(x, sums[tid * V + 2 * v], sums[tid * V + 2 * v + 1]);
        }
        __syncthreads();
        for (int i = tid; i < bx * V; i += kBwdThreads) {
            float total = 0.f;
            for (int y = 0; y < (int)blockDim.y; ++y) total += sums[y * bx * V + i];
            const unsigned channel = blockIdx.x * bx * V + i;
            if (channel < (unsigned)C) to[(size_t)(q - before) * C + channel] = total;
        }
        __syncthreads();
    }
}

// dw [C][K] and db [C] from the parts [rows][K + 1][C].  32 channels by 8 shares of the rows a block.
__global__ void __launch_bounds__(256) conv_join_kernel(const float* parts, int rows, int C, int K, float* dw,
                                                         float* db) {
    __shared__ float sums[8][32];
    after_all_before();
    const unsigned c = blockIdx.x * 32 + threadIdx.x, q = blockIdx.y;
    const bool live = c < (unsigned)C;
    float total = 0.f;
    if (live)
        for (int r = threadIdx.y; r < rows; r += 8) total += parts[((size_t)r * (K + 1) + q) * C + c];
    sums[threadIdx.y][threadIdx.x] = total;
    __syncthreads();
    if (threadIdx.y != 0 || !live) return;
#pragma unroll
    for (int y = 1; y < 8; ++y) total += sums[y][threadIdx.x];
    if (q < (unsigned)K) { if (dw) dw[(size_t)c * K + q] = total; }
    else if (db) db[c] = total;
}

// ----------------------------------------------------------------------------- host

// Bytes that V neighbouring values may span: what every row of every tensor starts on.
int widest(const ConvArgs& a, bool back) {
    const int es = a.bf16 ? 2 : 4;
    uint64_t bits = (uint64_t)a.C * es | 16;
    auto at = [&](const void* p) { bits |= reinterpret_cast<uintptr_t>(p); };
    auto step = [&](long long elements, bool used) { if (used) bits |= (uint64_t)elements * es; };
    at(a.x);
    step(a.x_tok, a.T > 1);
    step(a.x_seq, a.N > 1);
    if (back) {
        at(a.dy);
        step(a.dy_tok, a.T > 1);
        step(a.dy_seq, a.N > 1);
    }
    return (int)(bits & (~bits + 1));   // every other pointer is 16-byte aligned, its rows C values apart
}

template <typename T, int V, int KW, bool kAll>
cudaError_t fwd(const ConvArgs& a, bool one_strip, cudaStream_t s) {
    const int groups = a.C / V;
    const ConvFwdPlan p = conv_fwd_plan(a.N, a.T, groups, one_strip);
    if (p.blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_overlapped(a.doc ? conv_fwd_kernel<T, V, KW, kAll, true> : conv_fwd_kernel<T, V, KW, kAll, false>,
                             dim3((unsigned)p.blocks), dim3(kFwdThreads), s, a, (unsigned)groups, (unsigned)p.strips, p.strip);
}

template <typename T, int V, int KW, bool kAll>
cudaError_t bwd(const ConvArgs& a, cudaStream_t s) {
    const int groups = a.C / V;
    const ConvBwdPlan p = conv_bwd_plan(a.N, a.T, a.C, groups, kBwdBlocks<V, KW>);
    const dim3 grid(p.across, p.rows), block(p.bx, p.by);
    const cudaError_t e = launch_overlapped(a.doc ? conv_bwd_kernel<T, V, KW, kAll, true> : conv_bwd_kernel<T, V, KW, kAll, false>,
                                            grid, block, s, a, groups, p.strips, p.strip);
    if (e != cudaSuccess || !a.partial) return e;
    return launch_overlapped(conv_join_kernel, dim3(((unsigned)a.C + 31) / 32, a.K + 1), dim3(32, 8), s, (const float*)a.partial, p.rows,
                             a.C, a.K, a.dw, a.db);
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The window: 4 taps exactly (the usual case), up to 4, up to 8.
#define CONV_BY_TAPS(F, T, V, V8, ...)                              \
    do {                                                            \
        if (a.K == 4 && on16(a.w)) return F<T, V, 4, true>(a, ##__VA_ARGS__); \
        if (a.K <= 4) return F<T, V, 4, false>(a, ##__VA_ARGS__);   \
        return F<T, V8, 8, false>(a, ##__VA_ARGS__);                \
    } while (0)

// As many channels a thread as the rows' alignment and the registers allow.
cudaError_t fwd_any(const ConvArgs& a, bool one_strip, cudaStream_t s) {
    const int bytes = widest(a, false);
    if (a.bf16) {
        if (bytes >= 16) CONV_BY_TAPS(fwd, __nv_bfloat16, 8, 4, one_strip, s);
        if (bytes >= 8) CONV_BY_TAPS(fwd, __nv_bfloat16, 4, 4, one_strip, s);
        if (bytes >= 4) CONV_BY_TAPS(fwd, __nv_bfloat16, 2, 2, one_strip, s);
        CONV_BY_TAPS(fwd, __nv_bfloat16, 1, 1, one_strip, s);
    }
    if (bytes >= 16) CONV_BY_TAPS(fwd, float, 4, 4, one_strip, s);
    if (bytes >= 8) CONV_BY_TAPS(fwd, float, 2, 2, one_strip, s);
    CONV_BY_TAPS(fwd, float, 1, 1, one_strip, s);
}

cudaError_t bwd_any(const ConvArgs& a, cudaStream_t s) {
    const int bytes = widest(a, true);
    if (a.bf16) {
        if (bytes >= 8) CONV_BY_TAPS(bwd, __nv_bfloat16, 4, 2, s);
        if (bytes >= 4) CONV_BY_TAPS(bwd, __nv_bfloat16, 2, 2, s);
        CONV_BY_TAPS(bwd, __nv_bfloat16, 1, 1, s);
    }
    if (bytes >= 8) CONV_BY_TAPS(bwd, float, 2, 2, s);
    CONV_BY_TAPS(bwd, float, 1, 1, s);
}
#undef CONV_BY_TAPS

cudaError_t pass_state(const ConvArgs& a, const void* from, void* to, cudaStream_t s, int* launches) {
    const long long n = (long long)a.N * (a.K - 1) * a.C;
    *launches = to && n > 0;
    if (!*launches) return cudaSuccess;
    const unsigned blocks = (unsigned)((n + 255) / 256);
    if (a.bf16)
        conv_pass_kernel<<<blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(from), static_cast<__nv_bfloat16*>(to), n);
    else
        conv_pass_kernel<<<blocks, 256, 0, s>>>(static_cast<const float*>(from), static_cast<float*>(to), n);
    return cudaGetLastError();
}

}  // namespace

size_t conv_bwd_workspace_bytes(const ConvArgs& a) {
    return (size_t)conv_most_rows(a.C) * (a.K + 1) * a.C * 4;
}

cudaError_t conv_fwd_launch(const ConvArgs& a, cudaStream_t s, int* launches) {
    *launches = 1;
    return a.T > 0 ? fwd_any(a, false, s) : pass_state(a, a.state0, a.state, s, launches);
}

cudaError_t conv_step_launch(const ConvArgs& a, cudaStream_t s) { return fwd_any(a, true, s); }

cudaError_t conv_bwd_launch(const ConvArgs& a, cudaStream_t s, int* launches) {
    *launches = a.partial ? 2 : 1;
    if (a.T > 0) return bwd_any(a, s);
    // no tokens: the state passed on, the sums are empty
    cudaError_t e = pass_state(a, a.dstate, a.dstate0, s, launches);
    if (e == cudaSuccess && a.dw) e = cudaMemsetAsync(a.dw, 0, (size_t)a.C * a.K * 4, s);
    if (e == cudaSuccess && a.db) e = cudaMemsetAsync(a.db, 0, (size_t)a.C * 4, s);
    return e;
}

}  // namespace ttm
