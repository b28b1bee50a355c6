// Orthogonalised update: X_0 = G / max(|G|_F, eps), then per step
//   A = X X^T,  X <- a X + (b A + c A^2) X
// on the shorter side of G (X^T X from the right for a tall G), r the shorter side, l the
// longer.
//
// Numbers.  The products take fp16 operands and add in fp32.  bf16 operands are not
// enough: the steps multiply small singular values by up to a = 3.4 each, and their
// rounding with them (1 % off for a normal matrix, 6 % for one of low rank plus noise).  With
// fp16 operands, X itself kept to fp32's accuracy (in registers, or as the sum of two fp16
// values, hi + lo, in every step) and the diagonal of B, its largest entries once X is near
// orthogonal, in fp32 beside the product, the result is 1.7e-3 to 2.1e-3 off (2.8e-3 at 16 x 24), of
// which rounding it to bf16 is 1.7e-3; with B's diagonal in fp16 it would be up to
// 2.6e-3.  lo is kept to the end because a matrix of few directions has nothing that puts a
// rounding of X right: with lo dropped from the last three of five states one of rank 1
// was 1.4e-2 off.  For the same reason the diagonal multiplies all of X in the last steps alone, and
// before them hi, as the rest of B does: B (X - hi) is next to nothing for a matrix of few directions, its
// diagonal's share by itself is not, and grows with the steps to come (rank 1: 2.6e-2 off at 16 x 24,
// 4e-3 at 128 x 128).  Near the end that growth is small (kLateGrowth) and a matrix of full rank gains
// (512 x 512: 1.86e-3 off, 2.06e-3 with hi in every step).  Operands are stored times 2^10, so
// that entries of 1e-4 stay clear of fp16's subnormal range, and by other powers of two where the
// coefficients let the singular values leave the neighbourhood of one (operand_scales): a fixed 2^10 gave
// infinities for an entry of bA + cA^2 beyond 64.
//
// Three ways, by size.  128 x 128 at most, or 64 x 1024: one block, or a cluster, keeps a matrix on chip through all
// steps (ns_small_kernel: 192 x 128 x 128 in 28 us on the device).  A longer long side: the steps run on A alone, and
// G is read three times in all (ns_gram_kernel and those after it: 158 x 39 x 3516 in 131 us, 630 as products of every
// step).  A longer short side: three products a step (ns_gemm_kernel).  A and
// B = b A + c A^2 are symmetric, so only their tiles on and below the diagonal are
// computed and each is written twice, once transposed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "../../include/ttm.h"
#include "tc_ptx.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

using namespace tc;

constexpr float kScale = 1024.f, kUnscale = 1.f / 1024.f;
constexpr long long kWaitCycles = 4000000000LL;   // default limit, ~2 s at 2 GHz

// Instruction descriptor of tcgen05.mma .kind::f16 with fp16 A / B and an fp32 accumulator.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
           (uint32_t(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
__device__ __forceinline__ uint32_t bf162_bits(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 1 / max(norm, eps); NaN stays NaN.  A sum of squares is 0 or above 1e-45, so a norm 0 or above 1e-23;
// below 1e-30 eps counts as that, or 1 / eps times 2^10 were infinite and a zero matrix NaN.
__device__ __forceinline__ float inverse_norm(float sum_of_squares, float eps) {
    const float norm = sqrtf(sum_of_squares);
    return norm <= eps ? 1.f / fmaxf(eps, 1e-30f) : 1.f / norm;
}

__device__ __forceinline__ float4 load4(const OrthoArgs& a, size_t i) {
    if (!a.bf16) return *reinterpret_cast<const float4*>(static_cast<const float*>(a.G) + i);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.G) + i);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const OrthoArgs& a, size_t i) {
    return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.G)[i])
                  : static_cast<const float*>(a.G)[i];
}

// Bounded wait.  A wait that runs out sets the block's abort flag (every role then
// stops) and the device status word.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort, int* status,
                                       long long limit) {
    const long long t0 = clock64();
    while (!mbar_try_wait_sleep(bar, parity, 20000)) {
        if (*(volatile int*)abort) return false;
        if (clock64() - t0 > limit) {
            *(volatile int*)abort = 1;
            atomicExch(status, TTM_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, int* abort, int* status,
                                         long long limit) {
    return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, status, limit);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort, int* status,
                                          long long limit) {
    return __all_sync(0xffffffffu, wait_one(bar, parity, abort, status, limit));
}
// After an abort: give copies and products in flight a last bounded chance to land, however short the
// waits themselves are.
constexpr long long kDrainCycles = 20000000LL;    // ~10 ms
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, long long limit) {
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > max(limit, kDrainCycles)) return;
}

// ------------------------------------------------------------------- clusters (PTX)

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void peer_store2(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// ------------------------------------------------- one block, or one cluster, a matrix

// X, 128 x 128 zero-padded, as fp16 operands in two halves of 64 columns (rows of 128 bytes,
// 128-byte swizzle), its fp32 values in registers: thread (row, half) holds 64 of them.
// A, then B in its place, likewise.  Per step three products into the same 128 columns of
// tensor memory, each followed by its epilogue; two blocks share an SM, so that one's
// products run beside the other's epilogue.
//
// kCluster: a short side of up to 64 whose long one, of up to 1024, is split over the blocks of a cluster, 128
// columns each.
// A is then a sum over the blocks: each leaves its share in shared memory (fp32), adds a
// range of rows over all blocks in their order and hands the result to all of them;
// everything else stays a block's own.  (2 x 709 x 37: 27 us, 88 as products from global
// memory.)
constexpr int kSide = 128, kSmallThreads = 256, kMaxCluster = 8;
constexpr uint32_t kHalfBytes = kSide * 128;            // 64 columns of an operand
constexpr uint32_t kOperandBytes = 2 * kHalfBytes;

struct SmallShared {
    uint64_t done;
    uint32_t tmem;
    int abort;
    float part[kSmallThreads / 32];
    float sum;
    float diag[kSide];
};

__device__ __forceinline__ uint4* operand_at(unsigned char* base, int row, int chunk) {
    return reinterpret_cast<uint4*>(base + (chunk >> 3) * kHalfBytes + row * 128 +
                                    (((chunk & 7) ^ (row & 7)) << 4));
}

template <bool kCluster>
__global__ void __launch_bounds__(kSmallThreads, kCluster ? 1 : 2)
    ns_small_kernel(const __grid_constant__ OrthoArgs a) {
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char *sx = base, *sa = base + kOperandBytes;
    unsigned char* shares = base + 2 * kOperandBytes;   // kCluster: this block's share of A
    SmallShared& S = *reinterpret_cast<SmallShared*>(shares + (kCluster ? kSide * kSide * 4 : 0));
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const bool wide = a.m <= a.n;
    const int rank = kCluster ? (int)cluster_rank() : 0, ranks = kCluster ? (int)cluster_size() : 1;
    const int c0 = rank * kSide;                        // of the long side: this block's columns
    const int r = wide ? a.m : a.n, l = min((wide ? a.n : a.m) - c0, kSide);
    const int rp = r <= 64 ? 64 : 128, lp = l <= 64 ? 64 : 128;
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const size_t mat = (size_t)(blockIdx.x / ranks) * a.m * a.n;

    if (warp == 0) tmem_alloc(&S.tmem, 128);
    if (tid == 0) {
        mbar_init(&S.done, 1);
        fence_mbar_init();
        S.abort = 0;
    }

    // X_0: row of the short side, columns of the long one.  A wide G is read along its rows
    // into shared memory (fp32 rows of 512 bytes over both operands, 16-byte groups
    // permuted by row) and taken from there by row; a tall one's columns are already what
    // neighbouring lanes want.
    float X[64];
    if (wide) {
        auto at = [&](int i, int j) {
            return reinterpret_cast<float*>(base + i * 512 + (((j >> 2) ^ (i & 7)) << 4) + (j & 3) * 4);
        };
        if (a.n % 4 == 0) {
            const int per = l / 4;
#pragma unroll 4
            for (int i = tid; i < a.m * per; i += kSmallThreads)
                *reinterpret_cast<float4*>(at(i / per, i % per * 4)) =
                    load4(a, mat + (size_t)(i / per) * a.n + c0 + i % per * 4);
        } else {
#pragma unroll 4
            for (int i = tid; i < a.m * l; i += kSmallThreads)
                *at(i / l, i % l) = load1(a, mat + (size_t)(i / l) * a.n + c0 + i % l);
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
            const float4 q = *reinterpret_cast<const float4*>(at(row, half * 64 + c));
            const float f[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) X[c + e] = row < r && half * 64 + c + e < l ? f[e] : 0.f;
        }
        __syncthreads();                                // before the operands take its place
    } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) {
            const int col = half * 64 + c;
            X[c] = row < r && col < l ? load1(a, mat + (size_t)(c0 + col) * a.n + row) : 0.f;
        }
    }
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < 64; ++c) s = fmaf(X[c], X[c], s);
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) S.part[warp] = s;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    s = 0.f;
    for (int w = 0; w < kSmallThreads / 32; ++w) s += S.part[w];
    if (kCluster) {                                     // the norm is that of all blocks' columns
        if (tid == 0) S.sum = s;
        cluster_sync();
        s = 0.f;
        for (int i = 0; i < ranks; ++i) s += peer_load(peer_addr(&S.sum, i));
    }
    const float inv = inverse_norm(s, a.eps) * kScale;
#pragma unroll
    for (int c = 0; c < 64; ++c) X[c] *= inv;

    const uint32_t xb = smem_u32(sx), ab = smem_u32(sa);
    const uint32_t acc = tmem_addr(tmem, (warp & 3) * 32, half * 64);
    uint32_t phase = 0;
    bool lost = false;                                  // a wait of this warp ran out (S.abort is set)
    bool gone = false;                                  // one of this block did: no products any more
    // Every epilogue ends here: operands written, accumulators read, next product issued, unless a
    // wait of any warp has run out.  One verdict for the block, as all its warps meet at the barriers
    // that follow.
    auto ready = [&]() {
        fence_proxy_async_smem();
        tc_fence_before();
        const bool any = __syncthreads_or(lost);
        tc_fence_after();
        return !any;
    };
    auto wait_product = [&]() {
        if (!wait_warp(&S.done, phase, &S.abort, a.status, a.wait_cycles)) lost = true;
        phase ^= 1;
        tc_fence_after();
    };
    auto announce = [&](int product) {                  // or not, for a test of the waits
        if (product + 1 != a.debug_stall || rank + 1 != ranks) mma_commit(&S.done);
    };
    for (int step = 0; step < a.steps; ++step) {
        const NsStep& c = a.step[step];
        if (!gone) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                *operand_at(sx, row, half * 8 + q) =
                    make_uint4(half2_bits(X[8 * q], X[8 * q + 1]), half2_bits(X[8 * q + 2], X[8 * q + 3]),
                               half2_bits(X[8 * q + 4], X[8 * q + 5]), half2_bits(X[8 * q + 6], X[8 * q + 7]));
            gone = !ready();
        }
        if (gone && !kCluster) break;
        if (warp == 0 && !gone) {                       // A = X X^T
            if (elect_one()) {
                const uint32_t id = idesc_f16(128, rp, 0, 0);
                const uint64_t d0 = sdesc(xb, 16, 1024, 2);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t d = d0 + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4);
                    if (k * 16 < lp) mma_bf16(tmem, d, d, id, k > 0);
                }
                announce(3 * step);
            }
            __syncwarp();
        }
        if (!gone) wait_product();
        const bool mine = half * 64 < rp;               // columns of A and B that exist
        if (kCluster) {
            // rows of 512 bytes, 16-byte groups permuted by row
            auto group = [&](int i, int g) { return shares + i * 512 + ((g ^ (i & 7)) << 4); };
            if (mine) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[16];
                    tmem_ld16(acc + 16 * q, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        *reinterpret_cast<float4*>(group(row, half * 16 + 4 * q + h)) =
                            make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
                }
            }
            tc_fence_before();
            cluster_sync();                             // every block's share is written
            tc_fence_after();
            // Whether a wait of any block has run out: all see the same flags, which do not change
            // before the next product, so all leave in the same step, and none while another one
            // still reads its shared memory (they meet once more at the end).
            const float flag = lane < ranks ? peer_load(peer_addr(&S.abort, lane)) : 0.f;
            const int rows = (rp + ranks - 1) / ranks, groups = rp / 4;
#pragma unroll 2
            for (int i = tid; i < rows * groups; i += kSmallThreads) {
                const int y = rank * rows + i / groups, g = i % groups;
                if (y >= rp) break;
                float4 t = make_float4(0.f, 0.f, 0.f, 0.f), q[kMaxCluster];
#pragma unroll
                for (int k = 0; k < kMaxCluster; ++k)
                    if (k < ranks) q[k] = peer_load4(peer_addr(group(y, g), k));
#pragma unroll
                for (int k = 0; k < kMaxCluster; ++k)
                    if (k < ranks) { t.x += q[k].x; t.y += q[k].y; t.z += q[k].z; t.w += q[k].w; }
                const uint32_t lo = half2_bits(t.x * c.a, t.y * c.a);
                const uint32_t hi = half2_bits(t.z * c.a, t.w * c.a);
                const unsigned char* at = reinterpret_cast<unsigned char*>(operand_at(sa, y, g >> 1)) + (g & 1) * 8;
                for (int k = 0; k < ranks; ++k) peer_store2(peer_addr(at, k), lo, hi);
            }
            if (__any_sync(0xffffffffu, __float_as_int(flag) != 0)) break;
            asm volatile("fence.proxy.async;" ::: "memory");
            cluster_sync();                             // A is whole in every block
        } else if (mine) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float* f = v + 8 * h;
                    *operand_at(sa, row, half * 8 + 2 * q + h) =
                        make_uint4(half2_bits(f[0] * c.a, f[1] * c.a), half2_bits(f[2] * c.a, f[3] * c.a),
                                   half2_bits(f[4] * c.a, f[5] * c.a), half2_bits(f[6] * c.a, f[7] * c.a));
                }
            }
        }
        if (!ready()) break;                            // kCluster: not since all looked at the flags
        if (warp == 0) {                                // A A (A is symmetric)
            if (elect_one()) {
                const uint32_t id = idesc_f16(128, rp, 0, 0);
                const uint64_t d0 = sdesc(ab, 16, 1024, 2);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint64_t d = d0 + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4);
                    if (k * 16 < rp) mma_bf16(tmem, d, d, id, k > 0);
                }
                announce(3 * step + 1);
            }
            __syncwarp();
        }
        wait_product();
        float diag = 0.f;                               // of B, this row's
        if (mine) {                                     // B = b A + c A A over A, without its diagonal
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4* at = operand_at(sa, row, half * 8 + 2 * q + h);
                    uint32_t w[4] = {at->x, at->y, at->z, at->w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 old = half2_floats(w[i]);
                        v[8 * h + 2 * i] = fmaf(c.c2, v[8 * h + 2 * i], c.b1 * old.x);
                        v[8 * h + 2 * i + 1] = fmaf(c.c2, v[8 * h + 2 * i + 1], c.b1 * old.y);
                    }
                    if (half * 8 + 2 * q + h == row >> 3) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i == (row & 7)) {
                                diag = v[8 * h + i];
                                v[8 * h + i] = 0.f;
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = half2_bits(v[8 * h + 2 * i], v[8 * h + 2 * i + 1]);
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
        if (mine && row < rp && (row >> 6) == half) S.diag[row] = diag;
        if (!ready()) {                                 // kCluster: tells the others in the next step
            gone = true;
            continue;
        }
        const float beside = row < rp ? S.diag[row] * c.b : 0.f;
        const float keep = step < a.late ? 1.f : c.keep + beside;
        if (warp == 0) {                                // B X, X as [k][n]
            if (elect_one()) {
                const uint32_t id = idesc_f16(128, lp, 0, 1);
                const uint64_t d0 = sdesc(ab, 16, 1024, 2), e0 = sdesc(xb, kHalfBytes, 1024, 2);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k * 16 < rp)
                        mma_bf16(tmem, d0 + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                                 e0 + (k * 2048 >> 4), id, k > 0);
                announce(3 * step + 2);
            }
            __syncwarp();
        }
        if (step < a.late) {                            // the diagonal times hi, the rest of a step a X
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                const float2 h = half2_floats(half2_bits(X[i], X[i + 1]));
                X[i] = fmaf(c.keep, X[i], beside * h.x);
                X[i + 1] = fmaf(c.keep, X[i + 1], beside * h.y);
            }
        }
        wait_product();
        if (half * 64 < lp) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    X[16 * q + i] = fmaf(keep, X[16 * q + i], v[i] * c.b);
            }
        }
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + mat;
    if (wide && a.n % 8 == 0) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int col = half * 64 + 8 * q;
            const float* f = X + 8 * q;
            if (row < r && col < l)
                *reinterpret_cast<uint4*>(out + (size_t)row * a.n + c0 + col) =
                    make_uint4(bf162_bits(f[0] * kUnscale, f[1] * kUnscale),
                               bf162_bits(f[2] * kUnscale, f[3] * kUnscale),
                               bf162_bits(f[4] * kUnscale, f[5] * kUnscale),
                               bf162_bits(f[6] * kUnscale, f[7] * kUnscale));
        }
    } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) {
            const int col = half * 64 + c;
            if (row < r && col < l)
                out[wide ? (size_t)row * a.n + c0 + col : (size_t)(c0 + col) * a.n + row] =
                    __float2bfloat16(X[c] * kUnscale);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (S.abort && tid == 0) drain(&S.done, phase ^ 1, a.wait_cycles);   // the product issued last
    __syncthreads();
    if (kCluster) cluster_sync();                       // no access to a block that has left
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 128);
}

// The kernels of a call are launched so that one may start while the blocks of the one before
// finish: its set-up runs beside them, and it waits here before it reads what they wrote.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ norm and X_0

constexpr int kNormBlocks = 1024;      // partial sums of a matrix

__device__ __forceinline__ float block_sum(float s) {
    __shared__ float buf[8];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
    for (int w = 0; w < 8; ++w) s += buf[w];
    return s;
}

__global__ void __launch_bounds__(256) ns_norm_kernel(const __grid_constant__ OrthoArgs a, float* part) {
    const size_t mn = (size_t)a.m * a.n, base = blockIdx.y * mn;
    float s = 0.f;
    if (mn % 4 == 0) {
#pragma unroll 4
        for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4; i < mn; i += (size_t)gridDim.x * 1024) {
            const float4 g = load4(a, base + i);
            s += g.x * g.x + g.y * g.y + (g.z * g.z + g.w * g.w);
        }
    } else {
        for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < mn; i += (size_t)gridDim.x * 256)
            s = fmaf(load1(a, base + i), load1(a, base + i), s);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// X_0 as hi + lo, rows `pitch` values apart.
__global__ void __launch_bounds__(256) ns_start_kernel(const __grid_constant__ OrthoArgs a, const float* part,
                                                       int parts, int pitch, __half* hi, __half* lo) {
    float s = 0.f;
    for (int i = threadIdx.x; i < parts; i += 256) s += part[blockIdx.y * parts + i];
    s = block_sum(s);
    const float inv = inverse_norm(s, a.eps) * kScale;
    const int V = a.n % 4 == 0 ? 4 : 1, per = a.n / V;
    const size_t total = (size_t)a.m * per, mat = (size_t)blockIdx.y * a.m;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
        const size_t row = mat + i / per, src = row * a.n + (i % per) * V, dst = row * pitch + (i % per) * V;
        if (V == 4) {
            float4 g = load4(a, src);
            g.x *= inv; g.y *= inv; g.z *= inv; g.w *= inv;
            const uint2 h = make_uint2(half2_bits(g.x, g.y), half2_bits(g.z, g.w));
            const float2 h0 = half2_floats(h.x), h1 = half2_floats(h.y);
            *reinterpret_cast<uint2*>(hi + dst) = h;
            *reinterpret_cast<uint2*>(lo + dst) =
                make_uint2(half2_bits(g.x - h0.x, g.y - h0.y), half2_bits(g.z - h1.x, g.w - h1.y));
        } else {
            const float g = load1(a, src) * inv;
            hi[dst] = __float2half_rn(g);
            lo[dst] = __float2half_rn(g - __half2float(hi[dst]));
        }
    }
}

// No steps asked for: the normalised matrix itself.
__global__ void __launch_bounds__(256) ns_round_kernel(int m, int n, int pitch, const __half* hi,
                                                       const __half* lo, __nv_bfloat16* out) {
    const size_t total = (size_t)m * n, mat = (size_t)blockIdx.y * m;
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
        const size_t src = (mat + i / n) * pitch + i % n;
        out[mat * n + i] = __float2bfloat16((__half2float(hi[src]) + __half2float(lo[src])) * kUnscale);
    }
}

// ------------------------------------------------------- two blocks on one tile (PTX)

__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Tensor copy into this block's shared memory, counted on a barrier of either block.
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const void* tmap, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` in both blocks once the products issued so far are complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)), "h"((uint16_t)3)
        : "memory");
}
// ------------------------------------------------- a short side of at most 128, in A alone
//
// A step multiplies X by a polynomial of A = X X^T: X <- P X, P = a I + b A + c A^2, after which
// A <- P A P, and all of these commute.  So X_n = Q X_0 with Q the product of the steps' P, and the
// steps need A alone: G is read for |G|_F, for A_0 and for Q X_0, three times in all and not
// twice a step.  What that costs is accuracy: a rounding of A_0 is not put right by the next step's
// A.  Every operand here is therefore a sum hi + lo of two fp16 values, and a product takes hi hi +
// hi lo + lo hi: 1e-4 off for a matrix of low rank plus noise, 1e-5 for a normal one, before
// the result is rounded to bf16 (1.66e-3).  Next to rank one that is 6e-4 (short side 50) to 2e-3 (128),
// 1.8e-3 to 2.6e-3 in all: the tensor cores cut their sums off at 24 bits, and Q's large part, 485 times
// what has no direction of X in it, cancels.  Roundings grow as small singular values do, so coefficients that grow these by
// more than 1024 in all take the other path (tame).
//
//   ns_gram_kernel:  A_0 by parts of the long side, 128 of it at a time (fp32 sums)
//   ns_sum_kernel:   the parts' sums, in the parts' order, where they are many
//   ns_poly_kernel:  Q from A_0, a block a matrix: a chain of three products and their epilogues a
//                    step, 33 us for five steps (24 for RP = 64) whatever the long side
//   ns_apply_kernel: Q X_0, 128 of the long side at a time
// 158 x 39 x 3516 fp32: norm 18, A_0 44, Q 24, Q X_0 54 us, where reading G takes 13: the tiles' conversion to
// hi and lo, and stores of 64 bytes a warp, bound the two that read it.
//
// RP: the short side, padded to 64 or 128.  4 RP threads, so that each takes 32 of a tile's elements:
// those of the next tile are on their way while the products of this one run and its results
// leave.  Operands are RP rows of 64 columns (128 bytes, 128-byte swizzle) next to one another, tiles of
// a tall G 128 rows; with RP = 64 a product of 128 rows reads 64 more than there are, whose results
// nobody takes and which lie in the same block's shared memory (kPad).
constexpr float kQScale = 32.f;
template <int RP> constexpr int kGramThreads = 4 * RP;
template <int RP> constexpr uint32_t kTileBytes = RP * 256;           // hi, and lo behind it
template <int RP> constexpr uint32_t kQBytes = RP * RP * 2;           // likewise
template <int RP> constexpr uint32_t kPad = RP == 64 ? 16384 : 0;
template <int RP> constexpr int kGramSmem = 1024 + 2 * kTileBytes<RP> + kPad<RP> + 64;
template <int RP> constexpr int kPolySmem = 1024 + 6 * kQBytes<RP> + kPad<RP> + 64;
template <int RP> constexpr int kApplySmem = 1024 + 2 * kTileBytes<RP> + 2 * kQBytes<RP> + kPad<RP> + 64;

struct GramShared {
    uint64_t done;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(GramShared) <= 64, "the room left for it");

struct GramPlan {
    int rp;
    int chunks;                     // of 128 of the long side
    int gram_parts, gram_each;      // parts of a matrix in ns_gram_kernel, chunks of a part
    int apply_parts, apply_each;
    int norm_parts;
    float *norm, *sums;             // sums: [matrix][part][column / 4][row][4]
    unsigned char* q;               // Q as an operand, hi and lo, [matrix]
};

// hi and lo of eight values.
__device__ __forceinline__ void split8(const float* f, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = half2_bits(f[2 * i], f[2 * i + 1]);
        const float2 x = half2_floats(h[i]);
        l[i] = half2_bits(f[2 * i] - x.x, f[2 * i + 1] - x.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// An operand in shared memory: hi, its lo, bytes between 64 columns; mn: its rows are K.
struct Operand {
    uint32_t hi, lo, half;
    bool mn;
};

// acc (+)= (hi + lo)(hi + lo) but for lo lo, over `steps` blocks of 16 of K.
__device__ __forceinline__ void mma_split(uint32_t acc, const Operand& x, const Operand& y, int N, int steps,
                                          bool add) {
    const uint32_t id = idesc_f16(128, N, x.mn, y.mn);
    const uint64_t x0 = sdesc(x.hi, x.mn ? x.half : 16, 1024, 2), y0 = sdesc(y.hi, y.mn ? y.half : 16, 1024, 2);
    const uint32_t xl = (x.lo - x.hi) >> 4, yl = (y.lo - y.hi) >> 4;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (k >= steps) break;
        const uint32_t inside = (k & 3) * 32, down = k * 2048;
        const uint64_t xh = x0 + ((x.mn ? down : (k >> 2) * x.half + inside) >> 4);
        const uint64_t yh = y0 + ((y.mn ? down : (k >> 2) * y.half + inside) >> 4);
        mma_bf16(acc, xh, yh, id, add || k > 0);
        mma_bf16(acc, xh, yh + yl, id, true);
        mma_bf16(acc, xh + xl, yh, id, true);
    }
}

// A tile of G, rows x cols from element `at` on: on its way in registers, then an operand hi and lo,
// zero up to multiples of 16.
template <int RP>
struct Tile {
    float4 g[8];
    int rows, cols, col, first, step;
    bool four;                                          // four neighbours at a time, else two rows' pairs

    __device__ __forceinline__ void fetch(const OrthoArgs& a, size_t at, int rows_, int cols_) {
        rows = rows_;
        cols = cols_;
        four = a.n % 4 == 0;
        const int v = four ? 4 : 2, c16 = (cols + 15) & ~15;
        int log = 2;                                    // threads side by side over the columns
        while ((v << log) < c16) ++log;
        col = (threadIdx.x & ((1 << log) - 1)) * v;
        first = threadIdx.x >> log;
        step = kGramThreads<RP> >> log;
        at += col;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            g[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (four) {
                const int row = first + i * step;
                if (row < rows && col < cols) g[i] = load4(a, at + (size_t)row * a.n);
            } else {
                const int r0 = first + 2 * i * step, r1 = r0 + step;
                const size_t e0 = at + (size_t)r0 * a.n, e1 = at + (size_t)r1 * a.n;
                if (r0 < rows && col < cols) g[i].x = load1(a, e0);
                if (r0 < rows && col + 1 < cols) g[i].y = load1(a, e0 + 1);
                if (r1 < rows && col < cols) g[i].z = load1(a, e1);
                if (r1 < rows && col + 1 < cols) g[i].w = load1(a, e1 + 1);
            }
        }
    }
    __device__ __forceinline__ void put(unsigned char* hi, uint32_t half, float scale) const {
        const int r16 = (rows + 15) & ~15;
        if (col >= ((cols + 15) & ~15)) return;
        auto at = [&](int row) {
            return hi + (col >> 6) * half + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4) + (col & 7) * 2;
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 x = make_float4(g[i].x * scale, g[i].y * scale, g[i].z * scale, g[i].w * scale);
            const uint2 h = make_uint2(half2_bits(x.x, x.y), half2_bits(x.z, x.w));
            const float2 f0 = half2_floats(h.x), f1 = half2_floats(h.y);
            const uint2 l = make_uint2(half2_bits(x.x - f0.x, x.y - f0.y), half2_bits(x.z - f1.x, x.w - f1.y));
            if (four) {
                const int row = first + i * step;
                if (row >= r16) continue;
                *reinterpret_cast<uint2*>(at(row)) = h;
                *reinterpret_cast<uint2*>(at(row) + kTileBytes<RP>) = l;
            } else {
                const int r0 = first + 2 * i * step, r1 = r0 + step;
                if (r0 < r16) {
                    *reinterpret_cast<uint32_t*>(at(r0)) = h.x;
                    *reinterpret_cast<uint32_t*>(at(r0) + kTileBytes<RP>) = l.x;
                }
                if (r1 < r16) {
                    *reinterpret_cast<uint32_t*>(at(r1)) = h.y;
                    *reinterpret_cast<uint32_t*>(at(r1) + kTileBytes<RP>) = l.y;
                }
            }
        }
    }
};

// 2^10 / max(|G|_F, eps), the same in every warp.
__device__ __forceinline__ float start_scale(const OrthoArgs& a, const GramPlan& p, size_t mat) {
    float s = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x & 31; i < p.norm_parts; i += 32) s += p.norm[mat * p.norm_parts + i];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return inverse_norm(s, a.eps) * kScale;
}

// Operands in shared memory, accumulators read: the next product may be issued.
__device__ __forceinline__ void operands_ready() {
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// Waits for the products issued last; the same verdict in every warp, as all meet at the barriers that
// follow.
__device__ __forceinline__ bool products_done(GramShared& S, uint32_t& phase, const OrthoArgs& a) {
    const bool ok = wait_warp(&S.done, phase, &S.abort, a.status, a.wait_cycles);
    if (__syncthreads_or(!ok)) return false;
    phase ^= 1;
    tc_fence_after();
    return true;
}

__device__ __forceinline__ uint32_t set_up(GramShared& S, int warp, int columns) {
    if (warp == 0) tmem_alloc(&S.tmem, columns);
    if (threadIdx.x == 0) {
        mbar_init(&S.done, 1);
        fence_mbar_init();
        S.abort = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return S.tmem;
}
__device__ __forceinline__ void tear_down(GramShared& S, int warp, int columns, uint32_t phase, const OrthoArgs& a) {
    tc_fence_before();
    __syncthreads();
    if (S.abort && threadIdx.x == 0) drain(&S.done, phase, a.wait_cycles);
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(S.tmem, columns);
}

template <int RP>
__global__ void __launch_bounds__(kGramThreads<RP>, RP == 64 ? 4 : 2)
    ns_gram_kernel(const __grid_constant__ OrthoArgs a, const __grid_constant__ GramPlan p) {
    extern __shared__ unsigned char raw[];
    unsigned char* tile = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    GramShared& S = *reinterpret_cast<GramShared*>(tile + 2 * kTileBytes<RP> + kPad<RP>);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool wide = a.m <= a.n;
    const int r = wide ? a.m : a.n, l = wide ? a.n : a.m;
    const size_t mat = blockIdx.x / p.gram_parts;
    const int part = blockIdx.x % p.gram_parts;
    const uint32_t tmem = set_up(S, warp, 128);
    after_previous();
    const int c0 = part * p.gram_each, c1 = min(p.chunks, c0 + p.gram_each);
    const uint32_t x = smem_u32(tile), half = wide ? RP * 128 : kHalfBytes;
    const Operand X{x, x + kTileBytes<RP>, half, !wide};
    Tile<RP> t;
    auto fetch = [&](int c) {
        const int at = c * kSide, len = min(kSide, l - at);
        t.fetch(a, mat * a.m * a.n + (wide ? (size_t)at : (size_t)at * a.n), wide ? r : len, wide ? len : r);
    };
    fetch(c0);
    const float scale = start_scale(a, p, mat);
    uint32_t phase = 0;
    bool ok = true;
    for (int c = c0; c < c1; ++c) {
        if (c > c0 && !(ok = products_done(S, phase, a))) break;
        t.put(tile, half, scale);
        const int len = wide ? t.cols : t.rows;
        operands_ready();
        if (warp == 0) {
            if (elect_one()) {
                mma_split(tmem, X, X, RP, (len + 15) / 16, c > c0);
                mma_commit(&S.done);
            }
            __syncwarp();
        }
        if (c + 1 < c1) fetch(c + 1);
    }
    if (ok) ok = products_done(S, phase, a);
    const int row = (warp & 3) * 32 + lane, q0 = (warp >> 2) * 8;   // 32 columns a thread
    if (ok && row < RP) {
        float* to = p.sums + (size_t)blockIdx.x * RP * RP + row * 4;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float v[16];
            tmem_ld16(tmem_addr(tmem, (warp & 3) * 32, q0 * 4 + 16 * q), v);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 4; ++h)
                *reinterpret_cast<float4*>(to + (size_t)(q0 + 4 * q + h) * 4 * RP) =
                    make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        }
    }
    tear_down(S, warp, 128, phase, a);
}

// The sums of a matrix's parts into its first one: 64 words of 16 bytes a block, four threads a word, each a
// quarter of the parts (128 parts of 128 x 128: 27 us with a thread a word).
__global__ void __launch_bounds__(256) ns_sum_kernel(const __grid_constant__ GramPlan p) {
    __shared__ float4 quarter[4][64];
    after_previous();
    const size_t n = (size_t)p.rp * p.rp / 4;
    const int word = threadIdx.x & 63, mine = threadIdx.x >> 6, each = (p.gram_parts + 3) / 4;
    float4* at = reinterpret_cast<float4*>(p.sums) + blockIdx.y * p.gram_parts * n + blockIdx.x * 64 + word;
    const int k1 = min(p.gram_parts, (mine + 1) * each);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = mine * each; k < k1; ++k) {
        const float4 v = at[k * n];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    quarter[mine][word] = s;
    __syncthreads();                                    // the first part has been read
    if (mine) return;
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        const float4 v = quarter[i][word];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    at[0] = s;
}
constexpr int kFewParts = 4;        // ns_poly_kernel adds as many itself

template <int RP>
__global__ void __launch_bounds__(kGramThreads<RP>, RP == 64 ? 2 : 1)
    ns_poly_kernel(const __grid_constant__ OrthoArgs a, const __grid_constant__ GramPlan p) {
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    constexpr uint32_t ob = kQBytes<RP>, half = RP * 128;
    unsigned char *sa = base, *sp = base + 2 * ob, *sq = base + 4 * ob;
    GramShared& S = *reinterpret_cast<GramShared*>(base + 6 * ob + kPad<RP>);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int r = a.m <= a.n ? a.m : a.n, row = (warp & 3) * 32 + lane, c0 = (warp >> 2) * 32;
    const bool mine = row < RP;                         // 32 columns from c0 on
    const size_t mat = blockIdx.x;
    const uint32_t tmem = set_up(S, warp, 2 * RP), acc = tmem_addr(tmem, (warp & 3) * 32, c0);
    after_previous();

    auto put = [&](unsigned char* to, int q, const float* f) {   // columns c0 + 8 q ..
        uint4 hi, lo;
        split8(f, hi, lo);
        unsigned char* at = to + ((c0 + 8 * q) >> 6) * half + row * 128 + (((((c0 >> 3) + q) & 7) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = hi;
        *reinterpret_cast<uint4*>(at + ob) = lo;
    };
    // A_0 from the parts, in their order; zero past the short side
    float A[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) A[c] = 0.f;
    if (row < r) {
        const int parts = p.gram_parts > kFewParts ? 1 : p.gram_parts;
        const float* from = p.sums + mat * p.gram_parts * RP * RP + (size_t)c0 * RP + row * 4;
        for (int k = 0; k < parts; ++k, from += RP * RP) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(from + q * 4 * RP);
                A[4 * q] += v.x; A[4 * q + 1] += v.y; A[4 * q + 2] += v.z; A[4 * q + 3] += v.w;
            }
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) A[c] = c0 + c < r ? A[c] * (kUnscale * kUnscale) : 0.f;
    }
    auto put_A = [&]() {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = A[8 * q + i] * kScale;
            put(sa, q, f);
        }
    };
    if (mine) put_A();
    uint32_t phase = 0;
    const int steps = (r + 15) / 16;
    // x y.  All are symmetric but for their roundings; with y's transpose in its place those of one step came
    // back on the side where the next one multiplies them by up to 3.4 (rank 1 at 128 x 2000: 3.4e-3 off).
    auto product = [&](uint32_t column, const unsigned char* x, const unsigned char* y) {
        const uint32_t u = smem_u32(x), v = smem_u32(y);
        mma_split(tmem_addr(tmem, 0, column), Operand{u, u + ob, half, false}, Operand{v, v + ob, half, true}, RP,
                  steps, false);
    };
    auto announce = [&](int product) {                  // or not, for a test of the waits
        if (product + 1 != a.debug_stall) mma_commit(&S.done);
    };
    bool ok = true;
    for (int k = 0; k < a.steps; ++k) {
        const float ca = a.coeffs[3 * k], cb = a.coeffs[3 * k + 1], cc = a.coeffs[3 * k + 2];
        const bool last = k + 1 == a.steps;
        operands_ready();
        if (warp == 0) {
            if (elect_one()) {
                product(0, sa, sa);
                announce(3 * k);
            }
            __syncwarp();
        }
        if (!(ok = products_done(S, phase, a))) break;
        if (mine) {                                     // P; the first is Q too
            const float c2 = cc * (kUnscale * kUnscale);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float v[16], f[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int col = c0 + 16 * q + i;
                    v[i] = fmaf(c2, v[i], cb * A[16 * q + i]) + (col == row && row < r ? ca : 0.f);
                }
                if (k == 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = v[i] * kQScale;
                    put(sq, 2 * q, f);
                    put(sq, 2 * q + 1, f + 8);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = v[i] * kScale;
                put(sp, 2 * q, f);
                put(sp, 2 * q + 1, f + 8);
            }
        }
        if (last && k == 0) break;
        operands_ready();
        if (warp == 0) {
            if (elect_one()) {
                if (!last) product(0, sp, sa);
                if (k > 0) product(RP, sp, sq);
                announce(3 * k + 1);
            }
            __syncwarp();
        }
        if (!(ok = products_done(S, phase, a))) break;
        if (mine && !last) {                            // P A over A
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float v[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= kUnscale;
                put(sa, 2 * q, v);
                put(sa, 2 * q + 1, v + 8);
            }
        }
        if (!last) {
            operands_ready();
            if (warp == 0) {
                if (elect_one()) {
                    product(0, sa, sp);
                    announce(3 * k + 2);
                }
                __syncwarp();
            }
        }
        if (mine && k > 0) {                            // P Q over Q, beside the product above
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float v[16];
                tmem_ld16(acc + RP + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= kUnscale;
                put(sq, 2 * q, v);
                put(sq, 2 * q + 1, v + 8);
            }
        }
        if (last) break;
        if (!(ok = products_done(S, phase, a))) break;
        if (mine) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float v[16];
                tmem_ld16(acc + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) A[16 * q + i] = v[i] * (kUnscale * kUnscale);
            }
            put_A();
        }
    }
    __syncthreads();
    if (ok) {
        uint4* to = reinterpret_cast<uint4*>(p.q + mat * 2 * ob);
        for (uint32_t i = threadIdx.x; i < 2 * ob / 16; i += kGramThreads<RP>)
            to[i] = reinterpret_cast<const uint4*>(sq)[i];
    }
    tear_down(S, warp, 2 * RP, phase, a);
}

// A wide G's tile is the first operand, with the long side as its rows, a tall one's the second, with
// the long side as the accumulators' columns: either way neighbouring lanes write neighbouring
// elements.
template <int RP>
__global__ void __launch_bounds__(kGramThreads<RP>, RP == 64 ? 3 : 1)
    ns_apply_kernel(const __grid_constant__ OrthoArgs a, const __grid_constant__ GramPlan p) {
    extern __shared__ unsigned char raw[];
    unsigned char* tile = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    constexpr uint32_t ob = kQBytes<RP>;
    unsigned char* sq = tile + 2 * kTileBytes<RP>;
    GramShared& S = *reinterpret_cast<GramShared*>(sq + 2 * ob + kPad<RP>);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool wide = a.m <= a.n;
    const int r = wide ? a.m : a.n, l = wide ? a.n : a.m;
    const size_t mat = blockIdx.x / p.apply_parts, mn = (size_t)a.m * a.n;
    const int part = blockIdx.x % p.apply_parts;
    const int N = wide ? RP : kSide;                    // columns of an accumulator, of two in turn
    const uint32_t tmem = set_up(S, warp, 2 * N);
    after_previous();
    const int c0 = part * p.apply_each, c1 = min(p.chunks, c0 + p.apply_each);
    Tile<RP> t;
    auto fetch = [&](int c) {
        const int at = c * kSide, len = min(kSide, l - at);
        t.fetch(a, mat * mn + (wide ? (size_t)at : (size_t)at * a.n), wide ? r : len, wide ? len : r);
    };
    fetch(c0);
    const float scale = start_scale(a, p, mat);
    const uint4* from = reinterpret_cast<const uint4*>(p.q + mat * 2 * ob);
    for (uint32_t i = threadIdx.x; i < 2 * ob / 16; i += kGramThreads<RP>) reinterpret_cast<uint4*>(sq)[i] = from[i];
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + mat * mn;
    const uint32_t x = smem_u32(tile), q = smem_u32(sq), half = wide ? RP * 128 : kHalfBytes;
    const Operand X{x, x + kTileBytes<RP>, half, wide}, Q{q, q + ob, RP * 128, false};
    const int row = (warp & 3) * 32 + lane, each = N / (kGramThreads<RP> / 128), col0 = (warp >> 2) * each;
    uint32_t phase = 0;
    auto issue = [&](int c) {
        t.put(tile, half, scale);
        operands_ready();
        if (warp == 0) {
            if (elect_one()) {
                const uint32_t acc = tmem_addr(tmem, 0, (c & 1) * N);
                if (wide) mma_split(acc, X, Q, N, (r + 15) / 16, false);
                else mma_split(acc, Q, X, N, (r + 15) / 16, false);
                mma_commit(&S.done);
            }
            __syncwarp();
        }
        if (c + 1 < c1) fetch(c + 1);
    };
    issue(c0);
    for (int c = c0; c < c1; ++c) {
        if (!products_done(S, phase, a)) break;
        if (c + 1 < c1) issue(c + 1);
        const int at = c * kSide, len = min(kSide, l - at);
        const int rows = wide ? len : r, cols = wide ? r : len;   // of the accumulators
        if ((warp & 3) * 32 >= rows) continue;
        __nv_bfloat16* o = out + (wide ? (size_t)at : (size_t)at * a.n) + row + (size_t)col0 * a.n;
        for (int i0 = 0; i0 < each && col0 + i0 < cols; i0 += 16, o += (size_t)16 * a.n) {
            float v[16];
            tmem_ld16(tmem_addr(tmem, (warp & 3) * 32, (c & 1) * N + col0 + i0), v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (row < rows && col0 + i0 + i < cols)
                    o[(size_t)i * a.n] = __float2bfloat16(v[i] * (kUnscale / kQScale));
        }
    }
    tear_down(S, warp, 2 * N, phase, a);
}

template <int CG>
__device__ __forceinline__ void alloc_columns(uint32_t* dst, uint32_t n) {
    if (CG == 1) {
        tmem_alloc(dst, n);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(n)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void free_columns(uint32_t t, uint32_t n) {
    if (CG == 1) tmem_dealloc(t, n);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(n) : "memory");
}

// ------------------------------------------------------------------------ products

// One of the three products of a step, tiles of 128 CG x BN, K in blocks of 64.  With CG = 2
// two blocks (a cluster) share a tile: each copies in its 128 rows of A and half of the BN
// rows of B, one issues products over both (M = 256), each keeps its rows' accumulators.
// That halves what a block reads of B, and the copies are what bounds a tile: they reach about 50
// bytes a cycle and SM, so that a block of K takes 490 cycles for the 24 KB of a tile of 256 x 128 and
// 650 for the 32 KB of 256 x 256, whose products take 256 and 512.  At 2048 x 8240 A takes 36 us
// (129 blocks of K in one round of tiles), B 16 and the update 58 (37 without its
// epilogue, whose 134 MB pass through the same L2): 550 us for five steps with norm and start, 1.02
// PFLOP/s with the symmetric products counted half.
//   kGram:   out = alpha acc                (A; on and below the diagonal, mirrored; or, with few
//            tiles and a long K, fp32 sums over parts of K, which ns_join_kernel adds)
//   kSquare: out = alpha acc + beta in      (B from A A and A; likewise)
//   kUpdate: X'  = alpha acc + beta X       (X and X' as hi + lo; the last one to bf16)
// Roles (320 threads, one block an SM): warp 0 copies operand tiles in (kStages deep), warp 1
// issues the products into one of two accumulators, two teams of four warps (2-5, 6-9) take
// them through the epilogue, 32 rows a warp, 64 columns at a time: every other chunk of a
// tile each, or, where K is short and a block has several tiles, every other tile (the
// epilogue's latency is what those would wait for: 612 matrices of 491 x 200 took 1440 us
// without, 1260 with; the 2048 x 8240 projection, K of 2048 and more, 560 against
// 590).  The values to add and the results go through shared
// memory, so that accesses to global memory are full rows of 128 bytes.
enum { kGram, kSquare, kUpdate };
constexpr int kBM = 128, kBK = 64, kEpiWarps = 8, kGemmThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kChunkBytes = 32 * 128;              // 32 rows of 64 fp16 values
constexpr uint32_t kEpiBytes = kEpiWarps * 2 * kChunkBytes;   // (hi, lo) for each warp

// As many stages as fit beside the epilogue's buffers in 227 KB, at most 6.
__host__ __device__ constexpr int stages_of(int CG, int BN) {
    const int n = (int)((232448 - 1024 - 3072 - kEpiBytes) / ((kBM + BN / CG) * 128));
    return n < 6 ? n : 6;
}
__host__ __device__ constexpr uint32_t stage_bytes(int CG, int BN) { return (kBM + BN / CG) * 128; }

struct GemmParams {
    int M, N, K, batch;
    int tiles_m, tiles_n, per_matrix, tiles;
    int whole;                      // kUpdate, BN = 256: tiles before the halved ones
    int splits, split_blocks;       // kGram: parts of K, blocks of K in a part
    float* parts;                   // splits > 1: [splits][batch][M][part_pitch]
    int part_pitch;
    float alpha, beta;
    float* diag;                    // B's diagonal, [batch][short side]: kSquare writes it, kUpdate
                                    // adds it to beta, by row (or by_column): beta + diag times hi,
                                    // beta + diag_lo / diag_scale of it times lo
    float diag_scale, diag_lo;      // diag_lo: diag_scale, or 0
    int by_column, diag_n;
    const __half* in_hi;            // values to add, [batch][M][pitch]
    __half* out_hi;                 // results, likewise
    __half* lo;                     // kUpdate: lo of X, and of X' in its place
    int pitch;                      // of all three, a multiple of 8
    __nv_bfloat16* last;            // kUpdate, last step: the result instead, [batch][M][N]
    int* status;
    long long limit;
    int debug_stall;                // stage (modulo their number) + 1 that never fills; 0: none
};

struct GemmShared {
    float cols[kEpiWarps][64];
    uint64_t full[6], empty[6], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int abort;
};

struct TileAt {
    int row, col, mat, width;       // width: BN, or half of it
    int k0, k1, split;              // its blocks of K
};

// Tile t: all tiles (columns outermost, so that tiles at work share columns of X), or for the
// symmetric results those with an element on or below the diagonal, row by row.  Where the last
// round of tiles 256 wide would leave more than half of the blocks idle, its tiles are halved.
template <int EPI, int TM, int BN> constexpr bool kHalves = EPI == kUpdate && TM == 256 && BN == 256;

template <int EPI, int TM, int BN>
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
    TileAt at;
    const int kblocks = (p.K + kBK - 1) / kBK;
    at.split = 0;
    at.k0 = 0;
    at.k1 = kblocks;
    if (EPI == kGram && p.splits > 1) {
        at.split = t % p.splits;
        t /= p.splits;
        at.k0 = at.split * p.split_blocks;
        at.k1 = min(kblocks, at.k0 + p.split_blocks);
    }
    const bool halved = kHalves<EPI, TM, BN> && t >= p.whole;
    const int part = halved ? (t - p.whole) & 1 : 0;
    if (halved) t = p.whole + ((t - p.whole) >> 1);
    at.mat = t / p.per_matrix;
    t -= at.mat * p.per_matrix;
    at.width = BN;
    if (EPI == kUpdate) {
        at.row = t % p.tiles_m * TM;
        at.col = t / p.tiles_m * BN + part * (BN / 2);
        if (halved) at.width = BN / 2;
        return at;
    }
    int i = 0;
    while (true) {
        const int n = min(p.tiles_n, (i * TM + TM - 1) / BN + 1);
        if (t < n) break;
        t -= n;
        ++i;
    }
    at.row = i * TM;
    at.col = t * BN;
    return at;
}

template <bool AMN, bool BMN, int EPI, int CG, int BN>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ns_gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                   const __grid_constant__ GemmParams p) {
    constexpr int kStages = stages_of(CG, BN), TM = kBM * CG;
    constexpr uint32_t kStage = stage_bytes(CG, BN);
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char* epi = base + kStages * kStage;
    GemmShared& S = *reinterpret_cast<GemmShared*>(epi + kEpiBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)cluster_rank() : 0;
    const int first = blockIdx.x / CG, stride = gridDim.x / CG;
    const bool by_tile = p.tiles > stride && p.K <= 8 * kBK;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            // (in a test of the waits one stage expects an arrival that does not come; a condition in the
            // loader's loop took 1 % of the projection)
            mbar_init(&S.full[i], p.debug_stall && (p.debug_stall - 1) % kStages == i ? 2 : 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], (by_tile ? 4 : kEpiWarps) * CG);
        }
        fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 1) alloc_columns<CG>(&S.tmem, 2 * BN);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();                        // both blocks' barriers are set up
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    after_previous();

    if (warp == 0 && lane == 0) {
        int it = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += stride) {
            TileAt at = tile_at<EPI, TM, BN>(p, t);
            at.row += rank * kBM;
            at.col += rank * (at.width / CG);
            // a halved tile's B in rows of K is copied whole all the same
            const uint32_t stage = kBM * 128 + (BMN ? at.width : BN) / CG * 128;
            for (int k = at.k0; k < at.k1; ++k, ++it) {
                const int s = it % kStages;
                ok = wait_one(&S.empty[s], ((it / kStages) & 1) ^ 1, &S.abort, p.status, p.limit);
                if (!ok) break;
                unsigned char *da = base + s * kStage, *db = da + kBM * 128;
                if (rank == 0) mbar_expect_tx(&S.full[s], CG * stage);
                const uint32_t bar = CG == 2 ? peer_addr(&S.full[s], 0) : 0;
                auto load = [&](unsigned char* dst, const CUtensorMap* m, int x, int y) {
                    if (CG == 2) tma_load_3d_pair(dst, m, bar, x, y, at.mat);
                    else tma_load_3d(dst, m, &S.full[s], x, y, at.mat);
                };
                if (AMN) {
                    for (int i = 0; i < kBM / 64; ++i) load(da + i * 8192, &ma, at.row + 64 * i, k * kBK);
                } else {
                    load(da, &ma, k * kBK, at.row);
                }
                if (BMN) {
                    for (int i = 0; i < at.width / CG / 64; ++i) load(db + i * 8192, &mb, at.col + 64 * i, k * kBK);
                } else {
                    load(db, &mb, k * kBK, at.col);
                }
            }
        }
        if (*(volatile int*)&S.abort && rank == 0)      // copies still in flight
            for (int i = max(0, it - kStages); i < it; ++i)
                drain(&S.full[i % kStages], (i / kStages) & 1, p.limit);
    } else if (warp == 1 && rank == 0) {
        // The whole warp walks the loop, so that descriptors stay in uniform registers, and one
        // elected lane issues: with a single lane in the loop a product left every 137 cycles
        // whatever its size.
        constexpr uint32_t step_a = (AMN ? 2048 : 32) >> 4, step_b = (BMN ? 2048 : 32) >> 4;
        const uint32_t base_u = __shfl_sync(0xffffffffu, smem_u32(base), 0);
        const uint64_t a0 = AMN ? sdesc(base_u, 8192, 1024, 2) : sdesc(base_u, 16, 1024, 2);
        const uint64_t b0 = BMN ? sdesc(base_u + kBM * 128, 8192, 1024, 2) : sdesc(base_u + kBM * 128, 16, 1024, 2);
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += stride, ++n) {
            const int acc = n & 1;
            ok = wait_warp(&S.acc_empty[acc], ((n >> 1) & 1) ^ 1, &S.abort, p.status, p.limit);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * BN;
            const TileAt at = tile_at<EPI, TM, BN>(p, t);
            const uint32_t id = at.width == BN ? idesc_f16(TM, BN, AMN, BMN) : idesc_f16(TM, BN / 2, AMN, BMN);
            for (int k = at.k0; k < at.k1; ++k) {
                ok = wait_warp(&S.full[s], phase, &S.abort, p.status, p.limit);
                if (!ok) break;
                tc_fence_after();
                const uint64_t da = a0 + s * (kStage >> 4), db = b0 + s * (kStage >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk) {
                        if (CG == 2) mma_pair(d, da + kk * step_a, db + kk * step_b, id, k > at.k0 || kk > 0);
                        else mma_bf16(d, da + kk * step_a, db + kk * step_b, id, k > at.k0 || kk > 0);
                    }
                    if (CG == 2) commit_pair(&S.empty[s]);
                    else mma_commit(&S.empty[s]);
                    if (k + 1 == at.k1) {
                        if (CG == 2) commit_pair(&S.acc_full[acc]);
                        else mma_commit(&S.acc_full[acc]);
                    }
                }
                __syncwarp();
                if (++s == kStages) { s = 0; phase ^= 1; }
            }
        }
        // after an abort: products still in flight (the commit of the stage before s)
        if (*(volatile int*)&S.abort && lane == 0 && (s > 0 || phase))
            drain(&S.empty[s ? s - 1 : kStages - 1], s ? phase : phase ^ 1, p.limit);
    } else if (warp >= 2) {
        const int part = warp & 3;                      // this warp's lanes of tensor memory
        const int team = (warp - 2) >> 2;
        const int turn = by_tile ? 0 : team, hop = by_tile ? 1 : 2;   // this warp's chunks
        unsigned char *hi = epi + (warp - 2) * 2 * kChunkBytes, *lo = hi + kChunkBytes;
        int n = 0;
        for (int t = first; t < p.tiles; t += stride, ++n) {
            if (by_tile && (n & 1) != team) continue;
            const TileAt at = tile_at<EPI, TM, BN>(p, t);
            const int acc = n & 1, row0 = at.row + rank * kBM + part * 32;
            const size_t mat = (size_t)at.mat * p.M * p.pitch;
            // chunks of 64 columns that have an element to write: a prefix
            int chunks = 0;
            if (row0 < p.M) chunks = max(0, min(at.width / 64, (p.N - at.col + 63) / 64));
            if (EPI != kUpdate && chunks > 0)
                chunks = min(chunks, max(0, (row0 + 31 - at.col) / 64 + (row0 + 31 >= at.col)));
            // rows of 128 bytes: lane l takes 16 bytes l % 8 of rows l / 8, l / 8 + 4, ..
            const int piece = lane & 7, prow = lane >> 3;
            auto fetch = [&](int c) {                   // the values to add to chunk c
                const int col = at.col + 64 * c + 8 * piece;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = prow + 4 * i;
                    const size_t o = mat + (size_t)(row0 + r) * p.pitch + col;
                    const bool in = row0 + r < p.M && col < p.pitch;
                    const uint32_t d = smem_u32(hi) + r * 128 + ((piece ^ (r & 7)) << 4);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                                 "l"(in ? p.in_hi + o : p.in_hi), "r"(in ? 16 : 0) : "memory");
                    if (EPI == kUpdate)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + kChunkBytes),
                                     "l"(in ? p.lo + o : p.lo), "r"(in ? 16 : 0) : "memory");
                }
            };
            if (EPI != kGram && turn < chunks) fetch(turn);
            if (!wait_warp(&S.acc_full[acc], (n >> 1) & 1, &S.abort, p.status, p.limit)) break;
            tc_fence_after();
            for (int c = turn; c < chunks; c += hop) {
                const int col0 = at.col + 64 * c;
                if (EPI != kGram) {
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    __syncwarp();
                }
                const bool mirror = EPI != kUpdate && row0 > col0 + 63;
                const int row = row0 + lane;
                const float* diag = p.diag + (size_t)at.mat * p.diag_n;
                float keep = p.beta, keep_lo = p.beta;
                float* cols = S.cols[warp - 2];         // by column: this chunk's 64
                if (EPI == kUpdate && p.by_column) {
#pragma unroll
                    for (int i = 0; i < 64; i += 32)
                        cols[i + lane] = col0 + i + lane < p.N ? diag[col0 + i + lane] : 0.f;
                    __syncwarp();
                } else if (EPI == kUpdate && row < p.M) {
                    keep = fmaf(p.diag_scale, diag[row], keep);
                    keep_lo = fmaf(p.diag_lo, diag[row], keep_lo);
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float v[32];
                    const uint32_t ta = tmem_addr(tmem, part * 32, acc * BN + 64 * c + 32 * q);
                    tmem_ld16(ta, *reinterpret_cast<float(*)[16]>(v));
                    tmem_ld16(ta + 16, *reinterpret_cast<float(*)[16]>(v + 16));
                    tmem_wait_ld();
                    if (EPI == kGram && p.splits > 1) {
                        float* to = p.parts + (((size_t)at.split * p.batch + at.mat) * p.M + row) * p.part_pitch;
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const int col = col0 + 32 * q + i;
                            if (row < p.M && col < p.part_pitch)
                                *reinterpret_cast<float4*>(to + col) =
                                    make_float4(v[i] * p.alpha, v[i + 1] * p.alpha, v[i + 2] * p.alpha,
                                                v[i + 3] * p.alpha);
                        }
                        continue;
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t o = lane * 128 + (((4 * q + h) ^ (lane & 7)) << 4);
                        uint4* at_hi = reinterpret_cast<uint4*>(hi + o);
                        uint4* at_lo = reinterpret_cast<uint4*>(lo + o);
                        float* f = v + 8 * h;
                        uint32_t w[4], z[4];
                        if (EPI == kGram) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] *= p.alpha;
                        } else {
                            const uint4 u = *at_hi;
                            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
                            if (EPI == kUpdate) {
                                const uint4 y = *at_lo;
                                z[0] = y.x; z[1] = y.y; z[2] = y.z; z[3] = y.w;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 x = half2_floats(w[i]);
                                float b0 = keep, b1 = keep;
                                float2 add = make_float2(0.f, 0.f);
                                if (EPI == kUpdate) {
                                    const float2 y = half2_floats(z[i]);
                                    float c0 = keep_lo, c1 = keep_lo;
                                    if (p.by_column) {
                                        const float2 e =
                                            *reinterpret_cast<const float2*>(cols + 32 * q + 8 * h + 2 * i);
                                        b0 = fmaf(p.diag_scale, e.x, b0);
                                        b1 = fmaf(p.diag_scale, e.y, b1);
                                        c0 = fmaf(p.diag_lo, e.x, c0);
                                        c1 = fmaf(p.diag_lo, e.y, c1);
                                    }
                                    add = make_float2(c0 * y.x, c1 * y.y);
                                }
                                f[2 * i] = fmaf(p.alpha, f[2 * i], fmaf(b0, x.x, add.x));
                                f[2 * i + 1] = fmaf(p.alpha, f[2 * i + 1], fmaf(b1, x.y, add.y));
                            }
                            if (EPI == kSquare && col0 + 32 * q + 8 * h == (row & ~7) && row < p.M) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (i == (row & 7)) {
                                        p.diag[(size_t)at.mat * p.diag_n + row] = f[i];
                                        f[i] = 0.f;
                                    }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (EPI == kUpdate && p.last) {
                                w[i] = bf162_bits(f[2 * i] * kUnscale, f[2 * i + 1] * kUnscale);
                            } else {
                                w[i] = half2_bits(f[2 * i], f[2 * i + 1]);
                                if (EPI == kUpdate) {
                                    const float2 x = half2_floats(w[i]);
                                    z[i] = half2_bits(f[2 * i] - x.x, f[2 * i + 1] - x.y);
                                }
                            }
                        }
                        *at_hi = make_uint4(w[0], w[1], w[2], w[3]);
                        if (EPI == kUpdate) {
                            if (!p.last) *at_lo = make_uint4(z[0], z[1], z[2], z[3]);
                        } else if (mirror) {            // [64 columns][32 rows]
                            __half* m = reinterpret_cast<__half*>(lo) + (32 * q + 8 * h) * 32 + lane;
#pragma unroll
                            for (int i = 0; i < 8; ++i) m[i * 32] = __float2half_rn(f[i]);
                        }
                    }
                }
                __syncwarp();
                if (EPI == kGram && p.splits > 1) continue;
                // out again, row by row; the columns between N and the pitch are never read
                const bool rows16 = EPI != kUpdate || !p.last || p.N % 8 == 0;
                if (rows16) {
                    const int col = col0 + 8 * piece, width = EPI == kUpdate && p.last ? p.N : p.pitch;
                    __half* o_hi = EPI == kUpdate && p.last
                                       ? reinterpret_cast<__half*>(p.last) + (size_t)at.mat * p.M * p.N
                                       : p.out_hi + mat;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = prow + 4 * i;
                        const uint32_t o = r * 128 + ((piece ^ (r & 7)) << 4);
                        if (row0 + r < p.M && col < width) {
                            const size_t g = (size_t)(row0 + r) * width + col;
                            *reinterpret_cast<uint4*>(o_hi + g) = *reinterpret_cast<uint4*>(hi + o);
                            if (EPI == kUpdate && !p.last)
                                *reinterpret_cast<uint4*>(p.lo + mat + g) = *reinterpret_cast<uint4*>(lo + o);
                        }
                    }
                } else {
                    __nv_bfloat16* o = p.last + ((size_t)at.mat * p.M + row0) * p.N + col0;
                    for (int r = 0; r < 32 && row0 + r < p.M; ++r)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int e = lane + 32 * i;
                            if (col0 + e < p.N)
                                o[(size_t)r * p.N + e] = *reinterpret_cast<__nv_bfloat16*>(
                                    hi + r * 128 + (((e >> 3) ^ (r & 7)) << 4) + (e & 7) * 2);
                        }
                }
                if (mirror) {                           // rows of 64 bytes, 4 lanes each
                    const int x = row0 + 8 * (lane & 3);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = (lane >> 2) + 8 * i;
                        if (x < p.pitch)
                            *reinterpret_cast<uint4*>(p.out_hi + mat + (size_t)(col0 + r) * p.pitch + x) =
                                *reinterpret_cast<uint4*>(lo + r * 64 + (lane & 3) * 16);
                    }
                }
                __syncwarp();
                if (EPI != kGram && c + hop < chunks) fetch(c + hop);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) mbar_arrive_at(peer_addr(&S.acc_empty[acc], 0));
                else mbar_arrive(&S.acc_empty[acc]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();                        // no arrival at a block that has left
    tc_fence_after();
    if (warp == 1) free_columns<CG>(tmem, 2 * BN);
}

// A from the parts' sums, in the parts' order: a block takes 32 x 32 values on or below the
// diagonal and writes them and their mirror image.
__global__ void __launch_bounds__(256) ns_join_kernel(const float* parts, int splits, int batch, int n,
                                                      int part_pitch, int pitch, __half* A) {
    __shared__ float tile[32][33];
    after_previous();
    const int r0 = blockIdx.y * 32, c0 = blockIdx.x * 32;
    if (c0 > r0) return;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const size_t mat = blockIdx.z;
    A += mat * n * pitch;
    for (int y = ty; y < 32; y += 8) {
        const int r = r0 + y, c = c0 + tx;
        float t = 0.f;
        if (r < n && c <= r)
            for (int i = 0; i < splits; ++i) t += parts[(((size_t)i * batch + mat) * n + r) * part_pitch + c];
        tile[y][tx] = t;
        if (r < n && c <= r) A[(size_t)r * pitch + c] = __float2half_rn(t);
    }
    __syncthreads();
    for (int y = ty; y < 32; y += 8) {
        const int r = c0 + y, c = r0 + tx;              // the mirrored element, of row r < c
        if (c < n && r < c) A[(size_t)r * pitch + c] = __float2half_rn(tile[tx][y]);
    }
}

// ----------------------------------------------------------------------------- host

int pitch_of(int n) { return (n + 7) / 8 * 8; }

struct Workspace {
    size_t hi[2], lo, a, b, diag, part, parts, total;  // X as hi (two in turn) + lo (in place), A, B and its
                                                // diagonal, norm sums, A by parts of K
};

// Tiles of one matrix.
int tiles_of(int epi, int M, int N, int TM, int BN) {
    const int tm = (M + TM - 1) / TM, tn = (N + BN - 1) / BN;
    if (epi == kUpdate) return tm * tn;
    int all = 0;
    for (int i = 0; i < tm; ++i) {
        const int n = (i * TM + TM - 1) / BN + 1;
        all += n < tn ? n : tn;
    }
    return all;
}

// Parts of K for A = X X^T, r x r from l columns: as many as fill the SMs with tiles of 128 x 64,
// of four blocks of K at least; 1 where the tiles alone come near that.
int split_of(int batch, int r, int l) {
    const long long tiles = (long long)tiles_of(kGram, r, r, kBM, 64) * batch;
    const int kblocks = (l + kBK - 1) / kBK;
    if (tiles > 50 || kblocks < 16) return 1;
    int s = (int)(152 / tiles);
    if (s > kblocks / 4) s = kblocks / 4;
    if (s > 16) s = 16;
    const int each = (kblocks + s - 1) / s;
    return (kblocks + each - 1) / each;                 // no part is empty
}

Workspace layout(int batch, int m, int n) {
    Workspace w{};
    const size_t xs = (size_t)batch * m * pitch_of(n) * 2;
    const size_t rs = (size_t)(m < n ? m : n), as = (size_t)batch * rs * pitch_of((int)rs) * 2;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += (bytes + 255) / 256 * 256;
        return at;
    };
    for (size_t& o : w.hi) o = take(xs);
    w.lo = take(xs);
    w.a = take(as);
    w.b = take(as);
    w.diag = take((size_t)batch * rs * sizeof(float));
    w.part = take((size_t)batch * kNormBlocks * sizeof(float));
    const int splits = split_of(batch, (int)rs, m < n ? n : m);
    if (splits > 1) w.parts = take((size_t)splits * batch * rs * ((rs + 3) / 4 * 4) * sizeof(float));
    w.total = off;
    return w;
}

// The most that a step multiplies a singular value by, for singular values of 0 to `top`, and the largest
// that it leaves.
struct Reach {
    float most, next;
};
Reach reach(const float* c, float top) {
    Reach r{0.f, 0.f};
    for (int i = 0; i <= 64; ++i) {
        const float x = top * i / 64, y = x * x, p = std::fabs(c[0] + (c[1] + c[2] * y) * y);
        r.most = p > r.most ? p : r.most;
        r.next = x * p > r.next ? x * p : r.next;
    }
    return r;
}

// The steps with the powers of two that their operands are stored times, from bounds on the singular
// values: X (at most `top`) times sx and A (at most top^2) times sa so that the bounds come to between 2^10 and
// 2^11, and B (an entry is at most its largest eigenvalue, the polynomial less a) times sb so that its
// bound does to between 2^11 and 2^12.  With the default coefficients all three are 2^10 in every step.  The
// last X is in fp32 and times 2^10.
void operand_scales(const float* coeffs, int steps, NsStep* out) {
    auto power = [](double bound, int to) {            // 2^(to - floor(log2 bound)), 2^to for 0 and infinity
        int e = 0;
        if (bound > 0. && std::isfinite(bound)) std::frexp(bound, &e), --e;
        return std::ldexp(1., to - (e < -100 ? -100 : (e > 100 ? 100 : e)));
    };
    double top = 1., sx = kScale;
    for (int k = 0; k < steps; ++k) {
        const double a = coeffs[3 * k], b = coeffs[3 * k + 1], c = coeffs[3 * k + 2];
        double next = 0., most = 0.;                    // of X', of B
        for (int i = 0; i <= 64; ++i) {
            const double x = top * i / 64, y = x * x, p = b * y + c * y * y;
            most = std::fmax(most, std::fabs(p));
            next = std::fmax(next, x * std::fabs(a + p));
        }
        const double sa = power(top * top, 10), sb = power(most, 11);
        top = std::fmin(1.01 * next, 1e60);
        const double sy = k + 1 == steps ? kScale : power(top, 10);
        out[k] = {(float)(sa / (sx * sx)), (float)(b * sb / sa), (float)(c * sb / (sa * sa)), (float)(a * sy / sx),
                  (float)(sy / (sx * sb))};
        sx = sy;
    }
}

// The first step after which the steps to come multiply a singular value by less than this.
constexpr float kLateGrowth = 8.f;
int late_step(const float* coeffs, int steps) {
    float most[kNsMaxSteps], top = 1.f, after = 1.f;
    for (int k = 0; k < steps; ++k) {
        const Reach r = reach(coeffs + 3 * k, top);
        most[k] = r.most;
        top = 1.01f * r.next;
    }
    int k = steps;
    while (k > 0 && after < kLateGrowth) after *= most[--k];
    return k;
}

// Whether the steps may run on A alone: bounds on the operands (fp16, scaled; from above against
// overflow, from below against what lo cannot hold) and on the growth of a rounding, from the
// polynomials' values over the range of the singular values.
bool tame(const float* coeffs, int steps) {
    float top = 1.f, grown = 1.f;                       // of the singular values, of Q
    for (int k = 0; k < steps; ++k) {
        const Reach r = reach(coeffs + 3 * k, top);
        grown *= r.most;
        if (!(top >= 0.0625f && top * top <= 48.f && r.most <= 48.f && r.most * top * top <= 48.f)) return false;
        if (!(grown >= 0.25f && grown <= 1024.f)) return false;
        top = 1.01f * r.next;
    }
    return steps > 0;
}

GramPlan gram_plan(int batch, int m, int n, size_t* bytes) {
    GramPlan p{};
    const int r = m < n ? m : n, l = m < n ? n : m;
    p.rp = r <= 64 ? 64 : 128;
    p.chunks = (l + kSide - 1) / kSide;
    // About as many blocks as run at a time; where that is one an SM, the cut with the fewest rounds
    // of blocks times a block's chunks and set-up (23 x 7452 x 117: 163 us, 190 with 161 blocks).
    auto cut = [&](int resident, int* parts, int* each) {
        const int slots = 152 * resident, most = (slots + batch - 1) / batch;
        long long best = 0;
        for (int k = resident > 1 ? most : 1; k <= most; ++k) {
            const int e = k < p.chunks ? (p.chunks + k - 1) / k : 1, n = (p.chunks + e - 1) / e;
            const long long t = ((long long)batch * n + slots - 1) / slots * (e + 2);
            if (best && t >= best) continue;
            best = t;
            *parts = n;
            *each = e;
        }
    };
    cut(p.rp == 128 ? 2 : 4, &p.gram_parts, &p.gram_each);
    cut(p.rp == 128 ? 1 : m <= n ? 3 : 2, &p.apply_parts, &p.apply_each);
    const size_t mn = (size_t)m * n;
    p.norm_parts = (int)((mn + 4095) / 4096 < kNormBlocks ? (mn + 4095) / 4096 : kNormBlocks);
    size_t off = 0;
    auto take = [&](size_t b) {
        const size_t at = off;
        off += (b + 255) / 256 * 256;
        return at;
    };
    p.norm = reinterpret_cast<float*>(take((size_t)batch * p.norm_parts * 4));
    p.sums = reinterpret_cast<float*>(take((size_t)batch * p.gram_parts * p.rp * p.rp * 4));
    p.q = reinterpret_cast<unsigned char*>(take((size_t)batch * p.rp * p.rp * 4));
    *bytes = off;
    return p;
}

// Whether a call stays on chip: one block a matrix, or, with a short side of up to 64, a cluster of
// blocks of 128 of the long side, up to two blocks for each SM (2 x 709 x 37: 27 us so, 40 by its
// A alone; 1 x 64 x 256: 25 and 32; but 20 x 128 x 1024: 79 and 65).
bool small(int batch, int m, int n) {
    const int r = m < n ? m : n, ranks = ((m < n ? n : m) + kSide - 1) / kSide;
    return r <= kSide && (ranks == 1 || (r <= 64 && ranks <= kMaxCluster && (long long)batch * ranks <= 2 * 152));
}

// A stored fp16 matrix batch: [batch][rows][pitch].
struct Mat {
    __half* p;
    int rows, cols, pitch, batch;
    bool map(CUtensorMap* m, unsigned bx, unsigned by) const {
        const unsigned long long row = (unsigned long long)pitch * 2;
        return make_tma_map(m, TmaType::f16, p,
                            {(unsigned long long)cols, (unsigned long long)rows, (unsigned long long)batch},
                            {row, row * rows}, {bx, by, 1u}, true);
    }
};

// Launches a kernel in clusters of `cluster` blocks; `overlap`: its set-up may run beside the
// kernel before (after_previous).
template <typename... P, typename... A>
cudaError_t launch_in_clusters(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                               int cluster, bool overlap, const A&... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = overlap;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

template <bool AMN, bool BMN, int EPI, int CG, int BN>
cudaError_t gemm_tiles(const Mat& A, const Mat& B, GemmParams p, cudaStream_t s) {
    p.tiles_m = (p.M + kBM * CG - 1) / (kBM * CG);
    p.tiles_n = (p.N + BN - 1) / BN;
    p.per_matrix = tiles_of(EPI, p.M, p.N, kBM * CG, BN);
    const long long tiles = (long long)p.per_matrix * p.batch * (EPI == kGram && p.splits > 1 ? p.splits : 1);
    if (tiles > (1LL << 30)) return cudaErrorInvalidValue;
    p.tiles = p.whole = (int)tiles;
    if (kHalves<EPI, kBM * CG, BN>) {
        const int rest = p.tiles % (152 / CG);
        if (rest <= 152 / CG / 2) {
            p.whole -= rest;
            p.tiles += rest;
        }
    }
    CUtensorMap ma, mb;
    if (!A.map(&ma, 64, AMN ? 64 : kBM) || !B.map(&mb, 64, BMN ? 64 : BN / CG)) return cudaErrorInvalidValue;
    constexpr int smem = 1024 + stages_of(CG, BN) * stage_bytes(CG, BN) + kEpiBytes + sizeof(GemmShared);
    static_assert(smem <= 232448, "shared memory of a block");
    auto kernel = ns_gemm_kernel<AMN, BMN, EPI, CG, BN>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_in_clusters(kernel, dim3(CG * (p.tiles < 152 / CG ? p.tiles : 152 / CG)), dim3(kGemmThreads), smem, s,
                              CG, true, ma, mb, p);
}

// The tile that takes the least time by this count: rounds of tiles over the SMs times a tile's
// blocks of K (cycles for its copies or products, whichever is more) and its start and epilogue.
template <bool AMN, bool BMN, int EPI>
cudaError_t gemm(const Mat& A, const Mat& B, const GemmParams& p, cudaStream_t s) {
    if (EPI == kGram && p.splits > 1) return gemm_tiles<AMN, BMN, EPI, 1, 64>(A, B, p, s);
    auto cost = [&](int CG, int BN, double block) {
        const long long tiles = (long long)tiles_of(EPI, p.M, p.N, kBM * CG, BN) * p.batch;
        const long long slots = 152 / CG, rest = tiles % slots;
        const bool halves = EPI == kUpdate && CG == 2 && BN == 256 && rest <= slots / 2;
        const double rounds = (double)(tiles / slots) + (rest == 0 ? 0. : (halves ? 0.6 : 1.));
        return rounds * ((p.K + kBK - 1) / kBK * block + 20.0 * BN) + 4000;
    };
    const double c64 = cost(1, 64, 490), c128 = cost(1, 128, 650), p128 = cost(2, 128, 490),
                 p256 = cost(2, 256, 660);
    if (p256 <= p128 && p256 <= c128 && p256 <= c64)
        return gemm_tiles<AMN, BMN, EPI, 2, 256>(A, B, p, s);
    if (p128 <= c128 && p128 <= c64) return gemm_tiles<AMN, BMN, EPI, 2, 128>(A, B, p, s);
    if (c128 <= c64) return gemm_tiles<AMN, BMN, EPI, 1, 128>(A, B, p, s);
    return gemm_tiles<AMN, BMN, EPI, 1, 64>(A, B, p, s);
}

template <int RP>
cudaError_t gram_steps(const OrthoArgs& a, const GramPlan& p, cudaStream_t s, int* launches) {
    *launches = 4;
    auto launch = [&](void (*kernel)(OrthoArgs, GramPlan), int blocks, int smem) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        return launch_in_clusters(kernel, dim3(blocks), dim3(kGramThreads<RP>), smem, s, 1, true, a, p);
    };
    cudaError_t e = launch(ns_gram_kernel<RP>, a.batch * p.gram_parts, kGramSmem<RP>);
    if (e == cudaSuccess && p.gram_parts > kFewParts) {
        ++*launches;
        e = launch_in_clusters(ns_sum_kernel, dim3(RP * RP / 256, a.batch), dim3(256), 0, s, 1, true, p);
    }
    if (e == cudaSuccess) e = launch(ns_poly_kernel<RP>, a.batch, kPolySmem<RP>);
    if (e == cudaSuccess) e = launch(ns_apply_kernel<RP>, a.batch * p.apply_parts, kApplySmem<RP>);
    return e;
}

}  // namespace

size_t ortho_workspace_bytes(int batch, int m, int n) {
    if (small(batch, m, n)) return 0;
    size_t bytes = 0;
    if (m <= kSide || n <= kSide) gram_plan(batch, m, n, &bytes);
    const size_t products = layout(batch, m, n).total;
    return bytes > products ? bytes : products;
}

cudaError_t ortho_launch(const OrthoArgs& in, cudaStream_t s, int* launches) {
    OrthoArgs a = in;
    if (a.wait_cycles <= 0) a.wait_cycles = kWaitCycles;
    a.late = late_step(a.coeffs, a.steps);
    operand_scales(a.coeffs, a.steps, a.step);
    if (small(a.batch, a.m, a.n)) {
        constexpr int smem = 1024 + 2 * kOperandBytes + sizeof(SmallShared), shares = kSide * kSide * 4;
        const int ranks = ((a.m > a.n ? a.m : a.n) + kSide - 1) / kSide;
        *launches = 1;
        cudaError_t e;
        if (ranks == 1) {
            e = cudaFuncSetAttribute(ns_small_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            ns_small_kernel<false><<<a.batch, kSmallThreads, smem, s>>>(a);
            return cudaGetLastError();
        }
        e = cudaFuncSetAttribute(ns_small_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem + shares);
        if (e != cudaSuccess) return e;
        return launch_in_clusters(ns_small_kernel<true>, dim3(a.batch * ranks), dim3(kSmallThreads), smem + shares, s,
                                  ranks, false, a);
    }
    if ((a.m <= kSide || a.n <= kSide) && tame(a.coeffs, a.steps)) {
        size_t bytes;
        GramPlan p = gram_plan(a.batch, a.m, a.n, &bytes);
        char* ws = static_cast<char*>(a.workspace);
        p.norm = reinterpret_cast<float*>(ws + reinterpret_cast<size_t>(p.norm));
        p.sums = reinterpret_cast<float*>(ws + reinterpret_cast<size_t>(p.sums));
        p.q = reinterpret_cast<unsigned char*>(ws + reinterpret_cast<size_t>(p.q));
        ns_norm_kernel<<<dim3(p.norm_parts, a.batch), 256, 0, s>>>(a, p.norm);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        return p.rp == 64 ? gram_steps<64>(a, p, s, launches) : gram_steps<128>(a, p, s, launches);
    }
    const Workspace w = layout(a.batch, a.m, a.n);
    char* ws = static_cast<char*>(a.workspace);
    const bool wide = a.m <= a.n;
    const int r = wide ? a.m : a.n, l = wide ? a.n : a.m;
    const int xp = pitch_of(a.n), ap = pitch_of(r);
    // every tile reads all of hi's rows, so the new one goes elsewhere; a value of lo is read and
    // written by the same warp
    const Mat hi[2] = {{reinterpret_cast<__half*>(ws + w.hi[0]), a.m, a.n, xp, a.batch},
                       {reinterpret_cast<__half*>(ws + w.hi[1]), a.m, a.n, xp, a.batch}};
    __half* lo = reinterpret_cast<__half*>(ws + w.lo);
    const Mat A{reinterpret_cast<__half*>(ws + w.a), r, r, ap, a.batch};
    const Mat B{reinterpret_cast<__half*>(ws + w.b), r, r, ap, a.batch};
    float* part = reinterpret_cast<float*>(ws + w.part);
    const int splits = split_of(a.batch, r, l);

    const size_t mn = (size_t)a.m * a.n;
    size_t blocks = (mn + 4095) / 4096;
    if (blocks > kNormBlocks) blocks = kNormBlocks;
    const dim3 grid((unsigned)blocks, a.batch);
    ns_norm_kernel<<<grid, 256, 0, s>>>(a, part);
    size_t fill = (mn + 4095) / 4096;
    if (fill > 2048) fill = 2048;
    ns_start_kernel<<<dim3((unsigned)fill, a.batch), 256, 0, s>>>(
        a, part, (int)blocks, xp, hi[0].p, lo);
    *launches = 2;
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.steps == 0) {
        ns_round_kernel<<<dim3((unsigned)fill, a.batch), 256, 0, s>>>(
            a.m, a.n, xp, hi[0].p, lo, (__nv_bfloat16*)a.out);
        ++*launches;
        return cudaGetLastError();
    }
    for (int i = 0; i < a.steps; ++i) {
        const NsStep& c = a.step[i];
        const Mat &x = hi[i & 1], &y = hi[(i & 1) ^ 1];
        GemmParams p{};
        p.batch = a.batch;
        p.status = a.status;
        p.limit = a.wait_cycles;
        p.debug_stall = i == 0 ? a.debug_stall : 0;
        p.M = p.N = r;
        p.K = l;
        p.alpha = c.a;
        p.pitch = ap;
        p.out_hi = A.p;
        p.splits = splits;
        p.split_blocks = ((l + kBK - 1) / kBK + splits - 1) / splits;
        p.parts = reinterpret_cast<float*>(ws + w.parts);
        p.part_pitch = (r + 3) / 4 * 4;
        e = wide ? gemm<false, false, kGram>(x, x, p, s) : gemm<true, true, kGram>(x, x, p, s);
        if (e != cudaSuccess) return e;
        if (splits > 1) {
            const unsigned t = (r + 31) / 32;
            e = launch_in_clusters(ns_join_kernel, dim3(t, t, a.batch), dim3(256), 0, s, 1, true, (const float*)p.parts, splits,
                             a.batch, r, p.part_pitch, ap, A.p);
            if (e != cudaSuccess) return e;
            ++*launches;
        }
        p.K = r;
        p.alpha = c.c2;
        p.beta = c.b1;
        p.in_hi = A.p;
        p.out_hi = B.p;
        p.diag = reinterpret_cast<float*>(ws + w.diag);
        p.diag_n = r;
        p.debug_stall = 0;
        e = gemm<false, false, kSquare>(A, A, p, s);
        if (e != cudaSuccess) return e;
        p.M = a.m;
        p.N = a.n;
        p.alpha = p.diag_scale = c.b;
        p.diag_lo = i < a.late ? 0.f : p.diag_scale;
        p.by_column = !wide;
        p.beta = c.keep;
        p.pitch = xp;
        p.in_hi = x.p;
        p.lo = lo;
        p.out_hi = y.p;
        p.last = i + 1 == a.steps ? static_cast<__nv_bfloat16*>(a.out) : nullptr;
        e = wide ? gemm<false, true, kUpdate>(B, x, p, s) : gemm<false, false, kUpdate>(x, B, p, s);
        if (e != cudaSuccess) return e;
        *launches += 3;
    }
    return cudaSuccess;
}

}  // namespace ttm
