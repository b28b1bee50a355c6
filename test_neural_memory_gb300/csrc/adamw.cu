// AdamW step over many tensors in one launch:
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
//   p <- p (1 - lr decay) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps),
// g scaled by a number on the device, p in fp32 or bf16, fp32 weights with a bf16 copy on request, m and v in
// fp32 or in 8 bits.
//
// 8 bits.  m and sqrt(v) are e4m3 values times a power of two per 256 of them, the smallest that leaves none over
// 448.  Rounding to nearest would stand still: a step changes v by (1 - b2) (g^2 - v), a thousandth of it, and
// half a step of e4m3 is a sixteenth.  So a value goes up or down as its distance to the two neighbours and a
// dither say, a fixed hash of the value's place and the step: the moments move by the right amount on average, and
// equal calls give equal bits.  One exception: beside an m that is not coded as zero a root is not either, but as the
// smallest size.  Values of 2^-15 of their block's largest would else see m / (almost nothing) in the next step: with
// gradients of sizes exp(3 normal) the largest of 250 steps of 16384 values was 1e4 to 1e5 times the rate, and is 2.4 times.
// The moments' own arithmetic rounds after every operation (no fused multiply-add): whether a value is past the dither
// then does not depend on how a compiler contracts it.
//
// Bound by HBM: 28 bytes a value with fp32 moments and gradients, 14 in 8 bits with bf16 gradients.  A warp
// takes blocks of 256 values, 8 a lane in two runs of 4, so that every access of a warp is one piece of
// memory; tensors that do not start on 16 bytes, and their last blocks, go value by value.  The table of
// tensors travels as a kernel argument (a copy to the device would be a call of its own, and not the
// captured graph's), and a block finds its first tensor by bisection.  Measured: 92 M values of 12 layers, bf16 gradients and
// copies, 396 us, 98 % of a copy's rate; 8 bits 55 M values cold 211 us, 3.9 TB/s, bound by 96 instructions a value (hash,
// two roundings, scales), and 91 us for reading the moments out.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "overlap.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kSms = 152, kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlock = 256;             // values that share a scale
constexpr int kChunk = kWarps * kBlock; // values a block of threads takes at a time

template <int CAP>
struct Table {
    AdamwEntry e[CAP];
    int count, chunks;
    int last;                           // the launch that ends the step
};

struct Consts {
    float lr, keep, b1, b2, c1, c2, lr1, root2, eps, scale;   // lr1: lr / (1 - b1^t); root2: 1 / sqrt(1 - b2^t)
    uint32_t key;                       // of the dither
};

// lowbias32 of C. Wellons' search for integer hashes ("Prospecting for Hash Functions", 2018).
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ (x >> 16);
}

// The power of two, as an exponent, that a block's largest size (its bits) is divided by.
__device__ __forceinline__ int scale_of(uint32_t most) {
    const int e = (int)(most >> 23) - 127 - 8 + ((most & 0x7fffffu) > 0x600000u);
    return max(e, -126);
}
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The e4m3 code of a size y (bits u) from 2^-6 to 448: its lower neighbour on the grid, or the upper one where the missing part
// of a step and `frac`, in 2^-16 of one and shifted by 4, make a step: added below the three bits that stay, it
// carries by itself.
constexpr uint32_t kSmallest = 0x3c800000u;             // 2^-6
__device__ __forceinline__ uint32_t to_code(uint32_t u, uint32_t frac4) { return (u + frac4 - (120u << 23)) >> 20; }
__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&c)[4]) {
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
// Below 2^-6, where steps are 2^-9 (the sum is rounded to 24 bits before the floor).
__device__ __forceinline__ uint32_t to_small_code(float y, uint32_t frac4) {
    return (uint32_t)__fadd_rn(y * 512.f, (float)frac4 * (1.f / 1048576.f));
}

__device__ __forceinline__ float4 decode4(uint32_t code) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(code & 0xffffu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(code >> 16), __NV_E4M3);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float decode1(unsigned char code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
}
// Sizes compare as their bits do.
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInf = 0x7f800000u;

__device__ __forceinline__ Consts constants(const AdamwScalars& a) {
    Consts k;
    const int t = *reinterpret_cast<const volatile int*>(a.step) + 1;
    k.lr = a.lr_at ? *a.lr_at : a.lr;
    k.keep = fmaf(-k.lr, a.decay, 1.f);
    k.b1 = a.b1; k.b2 = a.b2; k.c1 = a.c1; k.c2 = a.c2;
    k.lr1 = k.lr / -expm1f((float)t * a.log_b1);
    k.root2 = 1.f / sqrtf(-expm1f((float)t * a.log_b2));
    k.eps = a.eps;
    k.scale = a.grad_scale ? *a.grad_scale : 1.f;
    k.key = (uint32_t)t * 0x9e3779b9u;
    return k;
}

// m, v and p of one value.
__device__ __forceinline__ void moments(const Consts& k, float g, float& m, float& v) {
    g = __fmul_rn(g, k.scale);
    m = __fadd_rn(__fmul_rn(m, k.b1), __fmul_rn(g, k.c1));
    v = __fadd_rn(__fmul_rn(v, k.b2), __fmul_rn(__fmul_rn(g, g), k.c2));
}
__device__ __forceinline__ float update(const Consts& k, float p, float m, float root) {
    float r;                            // 1 unit off
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(root, k.root2, k.eps)));
    return fmaf(-(k.lr1 * m), r, p * k.keep);
}

// One block of up to 256 values by a warp.  VEC: 256 of them, in runs of 4 a lane; otherwise lane l takes the
// values l, l + 32, ..
template <bool EIGHT, bool VEC>
__device__ __forceinline__ void step_block(const AdamwEntry& e, const AdamwScalars& a, const Consts& k, long long block,
                                           int lane) {
    const long long i0 = block * kBlock;                            // of the tensor
    const long long s0 = (e.first + block) * kBlock;                // of the moments
    const int n = (int)min((long long)kBlock, e.n - i0);
    auto index = [&](int j) { return VEC ? (j >> 2) * 128 + lane * 4 + (j & 3) : lane + 32 * j; };
    float p[8], g[8], m[8], v[8];
    if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * 128 + lane * 4;
            if (e.p_bf16) {
                const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(e.p) + i0 + i);
                p[4 * h] = __uint_as_float(u.x << 16); p[4 * h + 1] = __uint_as_float(u.x & 0xffff0000u);
                p[4 * h + 2] = __uint_as_float(u.y << 16); p[4 * h + 3] = __uint_as_float(u.y & 0xffff0000u);
            } else {
                *reinterpret_cast<float4*>(p + 4 * h) = *reinterpret_cast<const float4*>(static_cast<const float*>(e.p) + i0 + i);
            }
            if (e.g_bf16) {
                const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(e.g) + i0 + i);
                g[4 * h] = __uint_as_float(u.x << 16); g[4 * h + 1] = __uint_as_float(u.x & 0xffff0000u);
                g[4 * h + 2] = __uint_as_float(u.y << 16); g[4 * h + 3] = __uint_as_float(u.y & 0xffff0000u);
            } else {
                *reinterpret_cast<float4*>(g + 4 * h) = *reinterpret_cast<const float4*>(static_cast<const float*>(e.g) + i0 + i);
            }
            if constexpr (EIGHT) {
                *reinterpret_cast<float4*>(m + 4 * h) = decode4(*reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(a.m) + s0 + i));
                *reinterpret_cast<float4*>(v + 4 * h) = decode4(*reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(a.v) + s0 + i));
            } else {
                *reinterpret_cast<float4*>(m + 4 * h) = *reinterpret_cast<const float4*>(static_cast<const float*>(a.m) + s0 + i);
                *reinterpret_cast<float4*>(v + 4 * h) = *reinterpret_cast<const float4*>(static_cast<const float*>(a.v) + s0 + i);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = lane + 32 * j;
            p[j] = g[j] = m[j] = v[j] = 0.f;
            if (i >= n) continue;
            p[j] = e.p_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.p)[i0 + i]) : static_cast<const float*>(e.p)[i0 + i];
            g[j] = e.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.g)[i0 + i]) : static_cast<const float*>(e.g)[i0 + i];
            if constexpr (EIGHT) {
                m[j] = decode1(static_cast<const unsigned char*>(a.m)[s0 + i]);
                v[j] = decode1(static_cast<const unsigned char*>(a.v)[s0 + i]);
            } else {
                m[j] = static_cast<const float*>(a.m)[s0 + i];
                v[j] = static_cast<const float*>(a.v)[s0 + i];
            }
        }
    }
    float ms = 0.f, vs = 0.f;
    if constexpr (EIGHT) {
        ms = a.m_scale[e.first + block];
        vs = a.v_scale[e.first + block];
    }
    uint32_t most_m = 0, most_r = 0, mc[2], vc[2];  // largest sizes; codes, four to a word
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (EIGHT) {
            m[j] = __fmul_rn(m[j], ms);
            v[j] = __fmul_rn(v[j], vs);
            v[j] = __fmul_rn(v[j], v[j]);
        }
        moments(k, g[j], m[j], v[j]);
        const float root = sqrtf(v[j]);
        p[j] = update(k, p[j], m[j], root);
        if constexpr (EIGHT) {
            v[j] = root;
            if (VEC || index(j) < n) {
                most_m = max(most_m, size_bits(m[j]));
                most_r = max(most_r, size_bits(root));
            }
        }
    }
    if constexpr (VEC) {                // the weights leave first: the codes take registers
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * 128 + lane * 4;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(p[4 * h], p[4 * h + 1]);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(p[4 * h + 2], p[4 * h + 3]);
            const uint2 half = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            if (e.p_bf16) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(e.p) + i0 + i) = half;
            else *reinterpret_cast<float4*>(static_cast<float*>(e.p) + i0 + i) = *reinterpret_cast<float4*>(p + 4 * h);
            if (e.copy) *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(e.copy) + i0 + i) = half;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = lane + 32 * j;
            if (i >= n) continue;
            if (e.p_bf16) static_cast<__nv_bfloat16*>(e.p)[i0 + i] = __float2bfloat16_rn(p[j]);
            else static_cast<float*>(e.p)[i0 + i] = p[j];
            if (e.copy) static_cast<__nv_bfloat16*>(e.copy)[i0 + i] = __float2bfloat16_rn(p[j]);
        }
    }
    if constexpr (EIGHT) {
        most_m = __reduce_max_sync(0xffffffffu, most_m);
        most_r = __reduce_max_sync(0xffffffffu, most_r);
        const bool odd = max(most_m, most_r) >= kInf;   // a value that is not finite: the scale goes by the others
        if (odd) {
            most_m = most_r = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!VEC && index(j) >= n) continue;
                if (size_bits(m[j]) < kInf) most_m = max(most_m, size_bits(m[j]));
                if (size_bits(v[j]) < kInf) most_r = max(most_r, size_bits(v[j]));
            }
            most_m = __reduce_max_sync(0xffffffffu, most_m);
            most_r = __reduce_max_sync(0xffffffffu, most_r);
        }
        const int em = scale_of(most_m), er = scale_of(most_r);
        const float im = power(-em), ir = power(-er);
        // a block's places differ in their low 8 bits
        const uint32_t key = (uint32_t)s0 + k.key + (uint32_t)((unsigned long long)s0 >> 32) * 0x85ebca6bu;
        uint32_t least = kInf;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t cm[4], cr[4];                      // (garbage above the low byte for what is below 2^-6)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 4 * q + i;
                const uint32_t h = hash32(key + index(j)), um = __float_as_uint(fabsf(m[j]) * im), ur = __float_as_uint(v[j] * ir);
                cm[i] = to_code(um, h << 4 & 0xffff0u) | (__float_as_uint(m[j]) >> 24 & 0x80u);
                cr[i] = to_code(ur, h >> 12 & 0xffff0u);
                least = min(least, min(um, ur));
            }
            mc[q] = low_bytes(cm);
            vc[q] = low_bytes(cr);
        }
        if (least < kSmallest || odd) {                 // rare: values 2^-14 of their block's largest, zeros, no numbers
            auto put = [](uint32_t& word, int at, uint32_t code) { word = (word & ~(0xffu << 8 * at)) | code << 8 * at; };
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h = hash32(key + index(j));
                const float ym = fabsf(m[j]) * im, yr = v[j] * ir;
                if (__float_as_uint(ym) < kSmallest)
                    put(mc[j / 4], j & 3, to_small_code(ym, h << 4 & 0xffff0u) | (__float_as_uint(m[j]) >> 24 & 0x80u));
                if (__float_as_uint(yr) < kSmallest)    // (beside an m that is not zero: the smallest size at least)
                    put(vc[j / 4], j & 3, max(to_small_code(yr, h >> 12 & 0xffff0u), (uint32_t)((mc[j / 4] >> 8 * (j & 3) & 0x7fu) != 0)));
                if (size_bits(m[j]) >= kInf) put(mc[j / 4], j & 3, 0x7f);        // e4m3 has no infinity
                if (size_bits(v[j]) >= kInf) put(vc[j / 4], j & 3, 0x7f);
            }
        }
        if (lane == 0) {
            a.m_scale[e.first + block] = power(em);
            a.v_scale[e.first + block] = power(er);
        }
    }
    if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = h * 128 + lane * 4;
            if constexpr (EIGHT) {
                *reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(a.m) + s0 + i) = mc[h];
                *reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(a.v) + s0 + i) = vc[h];
            } else {
                *reinterpret_cast<float4*>(static_cast<float*>(a.m) + s0 + i) = *reinterpret_cast<float4*>(m + 4 * h);
                *reinterpret_cast<float4*>(static_cast<float*>(a.v) + s0 + i) = *reinterpret_cast<float4*>(v + 4 * h);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int i = lane + 32 * j;
            if (i >= n) continue;
            if constexpr (EIGHT) {
                static_cast<unsigned char*>(a.m)[s0 + i] = (unsigned char)(mc[j / 4] >> 8 * (j & 3));
                static_cast<unsigned char*>(a.v)[s0 + i] = (unsigned char)(vc[j / 4] >> 8 * (j & 3));
            } else {
                static_cast<float*>(a.m)[s0 + i] = m[j];
                static_cast<float*>(a.v)[s0 + i] = v[j];
            }
        }
    }
}

// Blocks an SM: 8 bits have 96 instructions to a value and want every warp; 32 bits are at HBM's rate either way
// and go 3 % faster with fewer rows of memory open at a time (92 M values 396 us, 407 with four).
template <bool EIGHT> constexpr int kBlocksPerSm = EIGHT ? 4 : 3;

template <bool EIGHT, int CAP>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm<EIGHT>) adamw_kernel(const __grid_constant__ Table<CAP> t,
                                                          const __grid_constant__ AdamwScalars a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    after_all_before();
    const Consts k = constants(a);
    int lo = 0, hi = t.count - 1;       // the last tensor that starts at or before the first chunk
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].chunk <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    for (int chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
        while (lo + 1 < t.count && t.e[lo + 1].chunk <= chunk) ++lo;
        const AdamwEntry& e = t.e[lo];
        const long long block = (long long)(chunk - e.chunk) * kWarps + warp;
        if (block * kBlock >= e.n) continue;
        const uint64_t at = reinterpret_cast<uintptr_t>(e.p) << e.p_bf16 | reinterpret_cast<uintptr_t>(e.g) << e.g_bf16 |
                            reinterpret_cast<uintptr_t>(e.copy) << 1;    // 4 bf16 values are 8 bytes
        if (at % 16 == 0 && (block + 1) * kBlock <= e.n) step_block<EIGHT, true>(e, a, k, block, lane);
        else step_block<EIGHT, false>(e, a, k, block, lane);
    }
    // The last block to finish counts the step: every block has read the count by then.
    if (t.last) {
        __syncthreads();
        if (threadIdx.x == 0 && atomicAdd(a.step + 1, 1) == (int)gridDim.x - 1) {
            a.step[1] = 0;
            a.step[0] += 1;
        }
    }
}

// m and v in fp32 from 8 bits: a warp a block of 256 values.
__global__ void __launch_bounds__(kThreads) adamw_moments_kernel(long long blocks, const __grid_constant__ AdamwScalars a,
                                                                  float* m, float* v) {
    const int lane = threadIdx.x & 31;
    after_all_before();
    for (long long b = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); b < blocks; b += (long long)gridDim.x * kWarps) {
        const float ms = a.m_scale[b], vs = a.v_scale[b];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = b * kBlock + h * 128 + lane * 4;
            float4 x = decode4(*reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(a.m) + i));
            float4 r = decode4(*reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(a.v) + i));
            x.x *= ms; x.y *= ms; x.z *= ms; x.w *= ms;
            r.x *= vs; r.y *= vs; r.z *= vs; r.w *= vs;
            *reinterpret_cast<float4*>(m + i) = x;
            *reinterpret_cast<float4*>(v + i) = make_float4(r.x * r.x, r.y * r.y, r.z * r.z, r.w * r.w);
        }
    }
}

template <bool EIGHT, int CAP>
cudaError_t launch(const AdamwEntry* tensors, int count, int chunks, int last, const AdamwScalars& a, cudaStream_t s) {
    Table<CAP> t;
    for (int i = 0; i < count; ++i) t.e[i] = tensors[i];
    t.count = count;
    t.chunks = chunks;
    t.last = last;
    const int most = kSms * kBlocksPerSm<EIGHT>, grid = chunks < 1 ? 1 : chunks < most ? chunks : most;
    return launch_overlapped(adamw_kernel<EIGHT, CAP>, dim3(grid), dim3(kThreads), s, t, a);
}

// Kernel arguments take 32764 bytes at most: kMost tensors.  A call writes its whole table, so short lists go with a shorter
// one: 30 tensors of 100 values 5.1 us with kFew and 5.8 with kMost, 96 tensors 9.4 us with kSome and 10.0 with kMost.
constexpr int kMost = 500, kSome = 128, kFew = 32;

template <bool EIGHT>
cudaError_t run(const AdamwEntry* tensors, int count, const AdamwScalars& a, cudaStream_t s, int* launches) {
    static_assert(sizeof(Table<kMost>) + sizeof(AdamwScalars) <= 32764, "kernel arguments");
    AdamwEntry part[kMost];
    int at = 0;
    *launches = 0;
    do {
        int n = 0;
        long long chunks = 0;
        while (at < count && n < kMost) {
            const long long more = (tensors[at].n + kChunk - 1) / kChunk;
            if (chunks + more > INT_MAX) break;
            part[n] = tensors[at++];
            part[n++].chunk = (int)chunks;
            chunks += more;
        }
        const cudaError_t e = n <= kFew    ? launch<EIGHT, kFew>(part, n, (int)chunks, at == count, a, s)
                              : n <= kSome ? launch<EIGHT, kSome>(part, n, (int)chunks, at == count, a, s)
                                           : launch<EIGHT, kMost>(part, n, (int)chunks, at == count, a, s);
        if (e != cudaSuccess) return e;
        ++*launches;
    } while (at < count);
    return cudaSuccess;
}

}  // namespace

cudaError_t adamw_step_launch(const AdamwEntry* tensors, int count, const AdamwScalars& a, cudaStream_t s,
                              int* launches) {
    return a.m_scale ? run<true>(tensors, count, a, s, launches) : run<false>(tensors, count, a, s, launches);
}

cudaError_t adamw_moments_launch(long long blocks, const AdamwScalars& a, float* m, float* v, cudaStream_t s) {
    if (blocks == 0) return cudaSuccess;
    const long long need = (blocks + kWarps - 1) / kWarps;
    const int grid = need < kSms * 8 ? (int)need : kSms * 8;
    return launch_overlapped(adamw_moments_kernel, dim3(grid), dim3(kThreads), s, blocks, a, m, v);
}

}  // namespace ttm
