// Arithmetic on pairs of fp32 values in one 64-bit register (two results an instruction on
// sm_100 and later), and its scalar twin, so that a kernel is written once for both.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace ttm {

struct f2 {
    unsigned long long v;
};

__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(f2 a, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ f2 add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }

template <typename T> __device__ __forceinline__ T splat(float v);
template <> __device__ __forceinline__ float splat<float>(float v) { return v; }
template <> __device__ __forceinline__ f2 splat<f2>(float v) { return pair(v, v); }

__device__ __forceinline__ float total(float a) { return a; }
__device__ __forceinline__ float total(f2 a) {
    float lo, hi;
    split(a, lo, hi);
    return lo + hi;
}

// Two bf16 values (low half first) as a pair and back.
__device__ __forceinline__ f2 pair_of_bf16(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_of_pair(f2 a) {
    float lo, hi;
    split(a, lo, hi);
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ f2 sub(f2 a, f2 b) { return fma(b, splat<f2>(-1.f), a); }

// 1 / (1 + exp(-x)) by the base-2 and reciprocal units: (4 + 0.7 |x|) 2^-23 of itself off at most, 0 where it is
// below the smallest normal number.
__device__ __forceinline__ float fast_logistic(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
    return r;
}

__device__ __forceinline__ f2 fast_logistic(f2 x) {
    float a, b;
    split(x, a, b);
    return pair(fast_logistic(a), fast_logistic(b));
}

}  // namespace ttm
