// Gated feed-forward block: g | u = x W_in, h = act(g) u, y = h W_out (+ residual), and its gradient
//   dh = dy W_out^T,  dg = dh u act'(g),  du = dh act(g),  dx = [dg | du] W_in^T,
//   dW_in = x^T [dg | du],  dW_out = h^T dy.
// Bound by the tensor cores: 6 N D F operations forward, 12 N D F in the gradient, on bf16 operands with fp32 sums.
//
// Products (ffn_gemm_kernel): tiles of 256 x 256 by two blocks (a cluster), M = 256 on tcgen05, K in blocks of
// 64.  Each block copies in 128 rows of A and 128 of B, one issues products over both, each keeps its rows' sums
// in tensor memory, in two sets, so that one tile's epilogue runs beside the next one's products.  Every operand is
// read as it lies in memory (rows of K, or K as rows: the transposes of the formulas cost nothing).
//   kGated:     B is 128 columns of W_g beside the same 128 of W_u, one from each block, so that a thread of the
//               epilogue has g and u of the same place; out go h and, if wanted, g and u
//   kStore:     y (+ residual), dx, dW_in, dW_out
//   kGatedBack: dh stays in tensor memory; g and u come in a piece ahead, dg, du and h leave
// What bounds a tile is how far ahead the copies run: 32 KB a block of K and 2000 cycles until they land; with four
// stages a block of K took 900 cycles, with five 680, with six 560, where the tensor cores need 512.  So the epilogue has
// little shared memory: 32 rows by 32 columns a warp at a time, one result after the other through two places (rows of 64
// bytes, swizzled: free of conflicts), from where rows of 64 bytes leave.  (By tensor copies every result waits for a
// fence and for the copy before it: 4700 cycles for kGatedBack's three, of which 1700 are arithmetic.)  What it reads goes
// to registers a piece ahead.
// Measured, 2048 x 5504: forward of 32768 rows 1330 to 1413 us, 1.57 to 1.67 PFLOP/s, gradient of 16384 rows 1393 to 1464
// us, 1.51 to 1.59 PFLOP/s, by the card, both under the power limit (1.44 to 1.6 GHz); the tensor pipe is busy 87 to 95 % of a kernel, 62 % of kGatedBack's, whose
// epilogue (two results and h out, g and u in) is as long as the products.
//
// Roundings: g and u enter the activation in fp32; h, dg and du are rounded to bf16 once, as operands of the next
// product (half a step, 2^-8 of a value at most: the same as rounding the result, and what the tensor cores
// take); sums are fp32 throughout.  The gradient's h comes from the saved bf16 g and u, another half step each.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "../../include/ttm.h"
#include "known_clusters.h"
#include "pairs.cuh"
#include "tc_pair.cuh"
#include "tc_ptx.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

using namespace tc;
using bf16 = __nv_bfloat16;

constexpr long long kWaitCycles = 4000000000LL;   // default limit, ~2 s at 2 GHz
constexpr int kSms = 152, kPairs = kSms / 2;

// Values in pairs, as bf16 in words.
template <int N>
__device__ __forceinline__ void unpack(const uint32_t* w, f2 (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = pair_of_bf16(w[i]);
}
__device__ __forceinline__ void unpack(const uint4& u, f2 (&f)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    unpack<4>(w, f);
}
__device__ __forceinline__ void unpack(const uint2& u, f2 (&f)[2]) {
    const uint32_t w[2] = {u.x, u.y};
    unpack<2>(w, f);
}
__device__ __forceinline__ uint4 pack(const f2 (&f)[4]) {
    return make_uint4(bf16_of_pair(f[0]), bf16_of_pair(f[1]), bf16_of_pair(f[2]), bf16_of_pair(f[3]));
}
__device__ __forceinline__ uint2 pack(const f2 (&f)[2]) { return make_uint2(bf16_of_pair(f[0]), bf16_of_pair(f[1])); }

// ------------------------------------------------------------------------ activation

// act(g) and, where kSlope, its derivative, of two values.  GELU: with z = |g| / sqrt(2), the upper tail of the normal
// distribution is erfc(z) / 2 = exp(-z^2) P(1 / (1 + 0.425 z)), P a polynomial fitted to exp(z^2) erfc(z) / 2 over the z
// that matter (2e-6 of itself at most, by iterated least squares on the relative error); the density's exponential is
// the same one.
template <bool kSlope>
__device__ __forceinline__ f2 act(f2 g, int gelu, f2& slope) {
    if (gelu) {
        float a, b, ea, eb, ta, tb, pa, pb;
        split(mul(mul(g, g), splat<f2>(-0.72134752f)), a, b);                                    // -g^2 / 2 in base 2
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(ea) : "f"(a));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(eb) : "f"(b));
        split(g, a, b);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ta) : "f"(fmaf(fabsf(a), 0.425f * 0.70710678f, 1.f)));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(tb) : "f"(fmaf(fabsf(b), 0.425f * 0.70710678f, 1.f)));
        const f2 t = pair(ta, tb), e = pair(ea, eb);
        f2 p = splat<f2>(-0.08400925f);
        p = fma(p, t, splat<f2>(0.23711844f));
        p = fma(p, t, splat<f2>(-0.04467765f));
        p = fma(p, t, splat<f2>(0.16266398f));
        p = fma(p, t, splat<f2>(0.10760187f));
        p = fma(p, t, splat<f2>(0.12137473f));
        p = fma(p, t, splat<f2>(-7.3115713e-5f));
        split(mul(e, p), pa, pb);                       // the tail
        const f2 c = pair(a < 0.f ? pa : 1.f - pa, b < 0.f ? pb : 1.f - pb);
        if (kSlope) slope = fma(mul(g, splat<f2>(0.39894228f)), e, c);
        return mul(g, c);
    }
    const f2 s = fast_logistic(g);
    if (kSlope) slope = mul(s, fma(g, sub(splat<f2>(1.f), s), splat<f2>(1.f)));
    return mul(g, s);
}

// -------------------------------------------------------------------------- products

enum { kStore, kGated, kGatedBack };
constexpr int kBM = 128, kBK = 64, kTile = 256, kEpiWarps = 8, kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kOperand = kBM * kBK * 2, kStageBytes = 2 * kOperand;      // of a block: 128 rows of A, 128 of B
constexpr uint32_t kPiece = 32 * 32 * 2;                                      // 32 rows x 32 columns
constexpr uint32_t kEpiBytes = kEpiWarps * 2 * kPiece;
constexpr int kStages = 6;
constexpr int kRowGroup = 8;            // row tiles that share their way through the columns

struct Problem {                        // one product
    int M, N, K;                        // kGated, kGatedBack: N = F
    int tiles_m, tiles;
    bf16 *out, *h;                      // kStore: result; kGated: gu (or NULL) and h; kGatedBack: dgu and h
    const bf16* add;                    // kStore: residual or NULL; kGatedBack: gu
    long long add_row;
};
struct Maps {
    CUtensorMap a, b;
};
struct GemmParams {
    Problem q[2];
    int tile0, tiles;                   // this launch's tiles: from .. to
    int splits;                         // SPLIT: pairs of a cluster that share a tile's K
    int beside;                         // the second of two launches of one product, which runs beside the first
    int gelu;
    int* status;
    long long limit;
    int debug_stall;                    // stage (modulo their number) + 1 that never fills; 0: none
};
struct GemmShared {
    uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    uint32_t tmem;
    int abort;
};
constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiBytes + sizeof(GemmShared);

struct TileAt {
    int row, col, which;
};

// Tiles go through kRowGroup row tiles at a time, column by column, so that the tiles at work share rows of A and
// the columns of B come round while they are in the L2 cache.
template <int MODE>
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, int t) {
    TileAt at;
    at.which = t >= p.q[0].tiles;
    if (at.which) t -= p.q[0].tiles;
    const Problem& q = p.q[at.which];
    const int tiles_n = q.tiles / q.tiles_m, group = t / (kRowGroup * tiles_n), first = group * kRowGroup;
    const int rows = min(kRowGroup, q.tiles_m - first), r = t - group * kRowGroup * tiles_n;
    at.row = (first + r % rows) * kTile;
    at.col = r / rows * (MODE == kGated ? kTile / 2 : kTile);
    return at;
}

// 16 bytes j of row r of a piece.
__device__ __forceinline__ uint4* piece_at(unsigned char* piece, int r, int j) {
    return reinterpret_cast<uint4*>(piece + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void load_sums(uint32_t at, float (&v)[32]) {
    tmem_ld16(at, *reinterpret_cast<float(*)[16]>(v));
    tmem_ld16(at + 16, *reinterpret_cast<float(*)[16]>(v + 16));
}

// Blocks of K [from, to) of a pair of the cluster.
struct Share {
    int from, to;
};
template <bool SPLIT>
__device__ __forceinline__ Share share_of(const GemmParams& p, int which, int pair) {
    const int kblocks = (p.q[which].K + kBK - 1) / kBK;
    if (!SPLIT) return {0, kblocks};
    const int each = (kblocks + p.splits - 1) / p.splits;
    return {min(kblocks, pair * each), min(kblocks, (pair + 1) * each)};
}

// SPLIT: a cluster of 2 to 4 pairs has one tile, each pair a share of its K.  The pairs leave their sums where the
// operands lay, and each takes its share of the pieces through the epilogue, summed over the pairs in their
// order.
template <bool AMN, bool BMN, int MODE, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ Maps m0, const __grid_constant__ Maps m1,
                    const __grid_constant__ GemmParams p) {
    constexpr int kS = kStages;
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    unsigned char* epi = base + kS * kStageBytes;
    GemmShared& S = *reinterpret_cast<GemmShared*>(epi + kEpiBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int member = (int)cluster_rank(), pair_of = SPLIT ? member >> 1 : 0;
    const int rank = member & 1, lead = SPLIT ? member & ~1 : 0;
    const uint16_t both = (uint16_t)(3 << lead);
    const int width = SPLIT ? 2 * p.splits : 2, first = p.tile0 + (int)blockIdx.x / width, stride = (int)gridDim.x / width;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kS; ++i) {
            // (in a test of the waits one stage expects an arrival that does not come)
            mbar_init(&S.full[i], p.debug_stall && (p.debug_stall - 1) % kS == i ? 2 : 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&S.acc_full[i], 1);
            mbar_init(&S.acc_empty[i], 2 * kEpiWarps);
        }
        fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 1) alloc_columns<2>(&S.tmem, 2 * kTile);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                     // both blocks' barriers are set up
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    // A launch starts its successor's set-up only when all before it has ended, so that one that runs beside it finds
    // the operands written, and needs to wait for it only before its own end, which the next launch goes by.
    if (!p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    if (warp == 0 && lane == 0) {
        int it = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += stride) {
            const TileAt at = tile_at<MODE>(p, t);
            const CUtensorMap *ma = at.which ? &m1.a : &m0.a, *mb = at.which ? &m1.b : &m0.b;
            const Share own = share_of<SPLIT>(p, at.which, pair_of);
            const int row = at.row + rank * kBM, col = MODE == kGated ? at.col : at.col + rank * (kTile / 2);
            for (int k = own.from; k < own.to; ++k, ++it) {
                const int s = it % kS;
                ok = wait_one(&S.empty[s], ((it / kS) & 1) ^ 1, &S.abort, p.status, p.limit);
                if (!ok) break;
                unsigned char *da = base + s * kStageBytes, *db = da + kOperand;
                if (rank == 0) mbar_expect_tx(&S.full[s], 2 * kStageBytes);
                const uint32_t bar = peer_addr(&S.full[s], lead);
                if (AMN) {
                    for (int i = 0; i < 2; ++i) tma_load_3d_pair(da + i * 8192, ma, bar, row + 64 * i, k * kBK, 0);
                } else {
                    tma_load_3d_pair(da, ma, bar, k * kBK, row, 0);
                }
                if (MODE == kGated) {                   // W_in as [D][2][F]: one block W_g, the other W_u
                    for (int i = 0; i < 2; ++i) tma_load_3d_pair(db + i * 8192, mb, bar, col + 64 * i, rank, k * kBK);
                } else if (BMN) {
                    for (int i = 0; i < 2; ++i) tma_load_3d_pair(db + i * 8192, mb, bar, col + 64 * i, k * kBK, 0);
                } else {
                    tma_load_3d_pair(db, mb, bar, k * kBK, col, 0);
                }
            }
        }
        if (*(volatile int*)&S.abort && rank == 0)      // copies still in flight
            for (int i = max(0, it - kS); i < it; ++i) drain(&S.full[i % kS], (i / kS) & 1, p.limit);
    } else if (warp == 1 && rank == 0) {
        // The whole warp walks the loop, so that descriptors stay in uniform registers, and one elected lane issues.
        constexpr uint32_t step_a = (AMN ? 2048 : 32) >> 4, step_b = (BMN ? 2048 : 32) >> 4;
        constexpr uint32_t id = idesc_bf16_f32(kTile, kTile, AMN, BMN);
        const uint32_t base_u = __shfl_sync(0xffffffffu, smem_u32(base), 0);
        const uint64_t a0 = AMN ? sdesc(base_u, 8192, 1024, 2) : sdesc(base_u, 16, 1024, 2);
        const uint64_t b0 = BMN ? sdesc(base_u + kOperand, 8192, 1024, 2) : sdesc(base_u + kOperand, 16, 1024, 2);
        int s = 0, n = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = first; t < p.tiles && ok; t += stride, ++n) {
            const int acc = n & 1;
            ok = wait_warp(&S.acc_empty[acc], ((n >> 1) & 1) ^ 1, &S.abort, p.status, p.limit);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + acc * kTile;
            const Share own = share_of<SPLIT>(p, t >= p.q[0].tiles, pair_of);
            for (int k = own.from; k < own.to; ++k) {
                ok = wait_warp(&S.full[s], phase, &S.abort, p.status, p.limit);
                if (!ok) break;
                tc_fence_after();
                const uint64_t da = a0 + s * (kStageBytes >> 4), db = b0 + s * (kStageBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        mma_pair(d, da + kk * step_a, db + kk * step_b, id, k > own.from || kk > 0);
                    commit_pair(&S.empty[s], both);
                    if (k + 1 == own.to) commit_pair(&S.acc_full[acc], both);
                }
                __syncwarp();
                if (++s == kS) { s = 0; phase ^= 1; }
            }
        }
        // after an abort: products still in flight (the commit of the stage before s)
        if (*(volatile int*)&S.abort && lane == 0 && (s > 0 || phase))
            drain(&S.empty[s ? s - 1 : kS - 1], s ? phase : phase ^ 1, p.limit);
    }

    // ------ epilogue: warps 2 .. 9
    constexpr int kIn = MODE == kGatedBack ? 8 : MODE == kStore ? 4 : 1;     // 16 bytes that a piece takes in, a lane
    const int part = warp & 3;                          // this warp's lanes of tensor memory
    const int team = (warp - 2) >> 2;                   // takes every other piece
    unsigned char* mine = epi + (warp - 2) * 2 * kPiece;
    int turn = 0;
    bool ok = true;
    uint4 next[kIn] = {};                               // of the next piece: the residual, or g and u, four lanes to a row
    auto row_of = [&](const TileAt& at) { return at.row + rank * kBM + part * 32; };
    auto pieces_of = [&](const TileAt& at) {            // that hold a result
        const Problem& q = p.q[at.which];
        const int all = MODE == kGated ? kTile / 2 : kTile;
        return row_of(at) < q.M ? (min(all, q.N - at.col) + 31) / 32 : 0;
    };
    auto read = [&](const TileAt& at, int c, int pieces) {
        const Problem& q = p.q[at.which];
        if (MODE == kGated || !q.add || c >= pieces) return;
        // places outside read the nearest ones inside: a load under a condition would be waited for at once
        const int row0 = row_of(at) + (lane >> 2), x = min(at.col + 32 * c + 8 * (lane & 3), q.N - 8);
#pragma unroll
        for (int i = 0; i < kIn / (MODE == kGatedBack ? 2 : 1); ++i) {
            const bf16* from = q.add + min(row0 + 8 * i, q.M - 1) * q.add_row + x;
            next[i] = *reinterpret_cast<const uint4*>(from);
            if constexpr (MODE == kGatedBack) next[4 + i] = *reinterpret_cast<const uint4*>(from + q.N);
        }
    };
    // What was read, a row a lane.
    auto turned = [&](uint4 (&now)[kIn]) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kIn; ++i) *piece_at(mine + i / 4 * kPiece, 8 * (i & 3) + (lane >> 2), lane & 3) = next[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kIn; ++i) now[i] = *piece_at(mine + i / 4 * kPiece, lane, i & 3);
    };
    // 32 columns of results of this warp's 32 rows, to `to` (rows `pitch` apart) where they are of the matrix, by way of one
    // place or the other: lanes with a row each write them, four lanes to a row take them out.
    auto emit = [&](const uint4 (&r)[4], bf16* to, long long pitch, int rows, int columns) {
        unsigned char* place = mine + (turn & 1) * kPiece;
        ++turn;
#pragma unroll
        for (int j = 0; j < 4; ++j) *piece_at(place, lane, j) = r[j];
        __syncwarp();
        const int j = lane & 3;
        bf16* at = to + (lane >> 2) * pitch + 8 * j;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 8 * i + (lane >> 2);
            if (row < rows && 8 * j < columns) *reinterpret_cast<uint4*>(at + 8 * i * pitch) = *piece_at(place, row, j);
        }
    };
    // Piece c with its sums (kGated: of g in v, of u in up); `after`: the next piece of this warp.
    auto piece = [&](const TileAt& at, int c, int after, int pieces, float (&v)[32], float (&up)[MODE == kGated ? 32 : 1]) {
        const Problem& q = p.q[at.which];
        const int x = at.col + 32 * c, row0 = row_of(at), rows = q.M - row0, columns = q.N - x;
        uint4 now[kIn], r0[4], r1[4], r2[4];
        if (MODE != kGated && q.add) turned(now);
        read(at, after, pieces);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f2 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = pair(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
            if constexpr (MODE == kStore) {
                if (q.add) {
                    f2 r[4];
                    unpack(now[j], r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[i] = add(f[i], r[i]);
                }
                r0[j] = pack(f);
            } else if constexpr (MODE == kGated) {
                f2 u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) u[i] = pair(up[8 * j + 2 * i], up[8 * j + 2 * i + 1]);
                r0[j] = pack(f);
                r1[j] = pack(u);
                f2 unused;
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = mul(act<false>(f[i], p.gelu, unused), u[i]);
                r2[j] = pack(f);
            } else {
                f2 g[4], u[4], h[4];
                unpack(now[j], g);
                unpack(now[4 + j], u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f2 slope;
                    const f2 a = act<true>(g[i], p.gelu, slope);
                    h[i] = mul(a, u[i]);
                    g[i] = mul(mul(f[i], u[i]), slope);
                    u[i] = mul(f[i], a);
                }
                r0[j] = pack(g);
                r1[j] = pack(u);
                r2[j] = pack(h);
            }
        }
        if constexpr (MODE == kStore) {
            emit(r0, q.out + (long long)row0 * q.N + x, q.N, rows, columns);
        } else {
            if (MODE == kGatedBack || q.out) {
                bf16* to = q.out + (long long)row0 * 2 * q.N + x;
                emit(r0, to, 2 * q.N, rows, columns);
                emit(r1, to + q.N, 2 * q.N, rows, columns);
            }
            emit(r2, q.h + (long long)row0 * q.N + x, q.N, rows, columns);
        }
    };
    if constexpr (!SPLIT) {
        if (warp >= 2) {
            int n = 0;
            for (int t = first; t < p.tiles && ok; t += stride, ++n) {
                const TileAt at = tile_at<MODE>(p, t);
                const int acc = n & 1, pieces = pieces_of(at);
                read(at, team, pieces);
                ok = wait_warp(&S.acc_full[acc], (n >> 1) & 1, &S.abort, p.status, p.limit);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sums = tmem_addr(tmem, part * 32, acc * kTile);
                auto give_back = [&] {                  // this warp has read its sums
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_relaxed_at(peer_addr(&S.acc_empty[acc], 0));
                };
                if (team >= pieces) give_back();
                for (int c = team; c < pieces; c += 2) {
                    float v[32], up[MODE == kGated ? 32 : 1];
                    load_sums(sums + 32 * c, v);
                    if constexpr (MODE == kGated) load_sums(sums + kTile / 2 + 32 * c, up);
                    tmem_wait_ld();
                    if (c + 2 >= pieces) give_back();
                    piece(at, c, c + 2, pieces, v, up);
                }
            }
        }
    } else {
        // one tile: its sums as [column][128 rows] over the stages, which nothing reads any more
        float* sums = reinterpret_cast<float*>(base);
        const TileAt at = tile_at<MODE>(p, first);
        const int pieces = pieces_of(at), step = 2 * p.splits, begin = 2 * pair_of + team;
        if (warp >= 2) {
            read(at, begin, pieces);
            ok = wait_warp(&S.acc_full[0], 0, &S.abort, p.status, p.limit);
            if (ok) {
                tc_fence_after();
                for (int c = team; c < kTile / 32; c += 2) {
                    float v[32];
                    load_sums(tmem_addr(tmem, part * 32, 32 * c), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) sums[(32 * c + i) * kBM + part * 32 + lane] = v[i];
                }
            }
            tc_fence_before();
        }
        __syncwarp();
        cluster_sync();
        if (warp >= 2 && ok) {
            for (int c = begin; c < pieces; c += step) {
                float v[32] = {}, up[MODE == kGated ? 32 : 1] = {};
                for (int q = 0; q < p.splits; ++q) {
                    const uint32_t from = peer_addr(sums + 32 * c * kBM + part * 32 + lane, 2 * q + rank);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += peer_load(from + i * kBM * 4);
                    if constexpr (MODE == kGated) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) up[i] += peer_load(from + (kTile / 2 + i) * kBM * 4);
                    }
                }
                piece(at, c, c + step, pieces, v, up);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                     // no arrival at a block that has left
    tc_fence_after();
    if (warp == 1) free_columns<2>(tmem, 2 * kTile);
    if (p.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------- products of few rows

// Few rows: the weights are what is read, and the rows too few for a tile's first side.  So the product is turned: 128
// of the weights' columns are the 128 rows of the first operand, the rows of x the second operand's, 16 to 128 of
// them (more take another block).  A cluster of up to 8 blocks shares a tile's K, so that all SMs read weights however
// few the tiles are; each leaves its sums in shared memory, and a share of the results is added up over the blocks in
// their order, put through the epilogue and written by each.  The second kernel of a call starts on its weights while
// the first one finishes.  16 x 2048 x 5504: 19.7 us a call,
// 67.6 MB of weights at 3.4 TB/s with both launches (6.5 TB/s while they stream).
constexpr int kNarrow = 128, kNarrowThreads = 256, kNarrowStages = 6, kNarrowSmem = 110 * 1024;     // two blocks an SM

struct NarrowParams {
    int N, wide, K;                     // rows; columns of the result (kGated: F); K
    int F, kblocks;                     // kGated, kGatedBack: F; blocks of K of a block of the cluster
    int bn, stages;                     // rows, padded to 16
    int gelu, second;                   // second: of a call's kernels
    bf16 *out, *gu, *h;                 // kStore: result; kGated: h and gu (or NULL); kGatedBack: dgu, gu read, h
    const bf16* add;                    // kStore: residual or NULL
    long long add_row;
    int* status;
    long long limit;
    int debug_stall;
};
struct NarrowShared {
    uint64_t full[kNarrowStages], empty[kNarrowStages], done;
    uint32_t tmem;
    int abort;
};

template <bool WMN, int MODE>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    ffn_narrow_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mx,
                      const __grid_constant__ NarrowParams p) {
    __shared__ NarrowShared S;
    extern __shared__ unsigned char raw[];
    unsigned char* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int tile = blockIdx.x / ranks, row0 = blockIdx.y * p.bn;
    const int first = MODE == kGated ? tile * 64 : tile * 128;       // column of the result (kGated: f)
    const int k0 = rank * p.kblocks, k1 = min((p.K + kBK - 1) / kBK, k0 + p.kblocks);
    const uint32_t stage = kOperand + p.bn * 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&S.full[i], p.debug_stall && (p.debug_stall - 1) % p.stages == i ? 2 : 1);
            mbar_init(&S.empty[i], 1);
        }
        mbar_init(&S.done, 1);
        fence_mbar_init();
        S.abort = 0;
    }
    if (warp == 1) tmem_alloc(&S.tmem, kNarrow);
    if (warp == 2 && lane == 0) {
        tma_prefetch_desc(&mw);
        tma_prefetch_desc(&mx);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    if (warp == 0 && lane == 0) {
        auto weights = [&](int k, int s) {
            unsigned char* to = base + s * stage;
            mbar_expect_tx(&S.full[s], stage);
            for (int i = 0; i < (WMN ? 2 : 1); ++i) {
                if (MODE == kGated) tma_load_3d(to + i * 8192, &mw, &S.full[s], first, i, k * kBK);
                else if (WMN) tma_load_3d(to + i * 8192, &mw, &S.full[s], first + 64 * i, k * kBK, 0);
                else tma_load_3d(to, &mw, &S.full[s], k * kBK, first, 0);
            }
        };
        // A call's second kernel needs its first one's results, but not for the weights, whose first stages are on
        // their way before its end.  The first kernel lets the second one start only when all before it has ended,
        // whatever wrote the weights among it.
        const int ahead = max(0, min(p.stages, k1 - k0));
        if (p.second)
            for (int i = 0; i < ahead; ++i) weights(k0 + i, i);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;");
        if (!p.second)
            for (int i = 0; i < ahead; ++i) weights(k0 + i, i);
        int it = 0;
        bool ok = true;
        for (int k = k0; k < k1; ++k, ++it) {
            const int s = it % p.stages;
            if (it >= p.stages) {
                ok = wait_one(&S.empty[s], ((it / p.stages) & 1) ^ 1, &S.abort, p.status, p.limit);
                if (!ok) break;
                weights(k, s);
            }
            tma_load_3d(base + s * stage + kOperand, &mx, &S.full[s], k * kBK, row0, 0);
        }
        if (*(volatile int*)&S.abort)                   // copies still in flight
            for (int i = max(0, it - p.stages); i < it; ++i) drain(&S.full[i % p.stages], (i / p.stages) & 1, p.limit);
    } else if (warp == 1) {
        constexpr uint32_t step = (WMN ? 2048 : 32) >> 4;
        const uint32_t id = idesc_bf16_f32(128, p.bn, WMN, 0);
        const uint32_t base_u = __shfl_sync(0xffffffffu, smem_u32(base), 0);
        const uint64_t a0 = WMN ? sdesc(base_u, 8192, 1024, 2) : sdesc(base_u, 16, 1024, 2);
        const uint64_t b0 = sdesc(base_u + kOperand, 16, 1024, 2);
        // (x comes after this too: the limit of a wait counts from the end of the kernel before, however long that runs)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int k = k0; k < k1; ++k) {
            ok = wait_warp(&S.full[s], phase, &S.abort, p.status, p.limit);
            if (!ok) break;
            tc_fence_after();
            const uint64_t da = a0 + s * (stage >> 4), db = b0 + s * (stage >> 4);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) mma_bf16(tmem, da + kk * step, db + kk * 2, id, k > k0 || kk > 0);
                mma_commit(&S.empty[s]);
                if (k + 1 == k1) mma_commit(&S.done);
            }
            __syncwarp();
            if (++s == p.stages) { s = 0; phase ^= 1; }
        }
        if (ok && k1 > k0) ok = wait_warp(&S.done, 0, &S.abort, p.status, p.limit);
        if (!ok && lane == 0 && (s > 0 || phase)) drain(&S.empty[s ? s - 1 : p.stages - 1], s ? phase : phase ^ 1, p.limit);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // sums as [row of x][128 columns], over the stages that nothing reads any more
    float* sums = reinterpret_cast<float*>(base);
    const bool good = *(volatile int*)&S.abort == 0;
    if (good) {
        const int part = warp & 3, half = p.bn / 2;
        for (int c = (warp >> 2) * half; c < ((warp >> 2) + 1) * half; c += 8) {
            float v[8];
            tmem_ld8(tmem_addr(tmem, part * 32, c), v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[(c + i) * 128 + part * 32 + lane] = k1 > k0 ? v[i] : 0.f;
        }
    }
    tc_fence_before();
    cluster_sync();
    asm volatile("griddepcontrol.wait;" ::: "memory");     // (long over: for the residual, g and u, read by every thread)
    if (good) {
        constexpr int kGroups = MODE == kGated ? 16 : 32;            // of 4 columns
        const int items = min(p.bn, p.N - row0) * kGroups, share = (items + ranks - 1) / ranks;
        const int last = min(items, (rank + 1) * share);
        for (int i = rank * share + (int)threadIdx.x; i < last; i += kNarrowThreads) {
            const int t = i / kGroups, g4 = i % kGroups * 4, col = first + g4;
            const long long row = row0 + t;
            if (col >= p.wide) continue;
            f2 v[2] = {splat<f2>(0.f), splat<f2>(0.f)}, u[2] = {v[0], v[0]};
            for (int q0 = 0; q0 < ranks; q0 += 4) {                  // four blocks' sums on their way together
                float4 a[4], b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = b[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (q0 + q >= ranks) continue;
                    const uint32_t at = peer_addr(sums + t * 128 + g4, q0 + q);
                    a[q] = peer_load4(at);
                    if constexpr (MODE == kGated) b[q] = peer_load4(at + 256);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v[0] = add(v[0], pair(a[q].x, a[q].y));
                    v[1] = add(v[1], pair(a[q].z, a[q].w));
                    if constexpr (MODE == kGated) {
                        u[0] = add(u[0], pair(b[q].x, b[q].y));
                        u[1] = add(u[1], pair(b[q].z, b[q].w));
                    }
                }
            }
            if constexpr (MODE == kStore) {
                if (p.add) {
                    f2 r[2];
                    unpack(*reinterpret_cast<const uint2*>(p.add + row * p.add_row + col), r);
#pragma unroll
                    for (int j = 0; j < 2; ++j) v[j] = add(v[j], r[j]);
                }
                *reinterpret_cast<uint2*>(p.out + row * p.wide + col) = pack(v);
            } else {
                bf16* gu = p.gu + row * 2 * p.F + col;
                uint2* h = reinterpret_cast<uint2*>(p.h + row * p.F + col);
                if constexpr (MODE == kGated) {
                    if (p.gu) {
                        *reinterpret_cast<uint2*>(gu) = pack(v);
                        *reinterpret_cast<uint2*>(gu + p.F) = pack(u);
                    }
                    f2 unused;
#pragma unroll
                    for (int j = 0; j < 2; ++j) v[j] = mul(act<false>(v[j], p.gelu, unused), u[j]);
                    *h = pack(v);
                } else {
                    f2 g[2], hh[2];
                    unpack(*reinterpret_cast<const uint2*>(gu), g);
                    unpack(*reinterpret_cast<const uint2*>(gu + p.F), u);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f2 slope;
                        const f2 a = act<true>(g[j], p.gelu, slope);
                        hh[j] = mul(a, u[j]);
                        g[j] = mul(mul(v[j], u[j]), slope);
                        u[j] = mul(v[j], a);
                    }
                    bf16* dgu = p.out + row * 2 * p.F + col;
                    *reinterpret_cast<uint2*>(dgu) = pack(g);
                    *reinterpret_cast<uint2*>(dgu + p.F) = pack(u);
                    *h = pack(hh);
                }
            }
        }
    }
    cluster_sync();                                     // no block leaves while its sums are read
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kNarrow);
}

// ----------------------------------------------------------------------------- host

// A matrix in memory: rows of `cols` values, `pitch` apart.
struct Matrix {
    const void* p;
    long long rows, cols, pitch;
    // Copies of 64 values by `down` rows.
    bool map(CUtensorMap* m, int down) const {
        const unsigned long long dims[3] = {(unsigned long long)cols, (unsigned long long)rows, 1};
        const unsigned long long row = (unsigned long long)pitch * 2, strides[2] = {row, row * (unsigned long long)rows};
        const unsigned box[3] = {64, (unsigned)down, 1};
        return make_tma_map(m, TmaType::bf16, p, dims, strides, box, true);
    }
    // Rows of 2F as [rows][2][F].
    bool halves(CUtensorMap* m, int down) const {
        const unsigned long long dims[3] = {(unsigned long long)cols / 2, 2, (unsigned long long)rows};
        const unsigned long long strides[2] = {(unsigned long long)cols, (unsigned long long)cols * 2};
        const unsigned box[3] = {64, 1, (unsigned)down};
        return make_tma_map(m, TmaType::bf16, p, dims, strides, box, true);
    }
    // As an operand: rows of K, or (mn) K as rows.
    bool operand(CUtensorMap* m, bool mn) const { return map(m, mn ? 64 : kBM); }
};

bool problem(Problem& q, int M, int N, int K, int mode) {
    q.M = M; q.N = N; q.K = K;
    q.tiles_m = (M + kTile - 1) / kTile;
    const int wide = mode == kGated ? kTile / 2 : kTile;
    const long long tiles = (long long)q.tiles_m * ((N + wide - 1) / wide);
    q.tiles = (int)tiles;
    return tiles < (1LL << 30);
}

// Clusters of `width` blocks that run at once (a cluster stays within a group of SMs), asked once for a kernel, device and
// width.
cudaError_t clusters_at_once(const void* kernel, KnownClusters& known, int width, int threads, int smem, int& n) {
    int device;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return known.get(device, width, n, [&](int* out) {
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = width;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(width);
        c.blockDim = dim3(threads);
        c.dynamicSmemBytes = smem;
        c.attrs = at;
        c.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(out, kernel, &c);
    });
}

// How a product's tiles are gone through: whole rounds by the pairs, the rest in one more round or with K shared by
// clusters of 2 to 4 pairs (20 tiles of a last round leave 56 pairs idle).
struct Plan {
    int whole, splits;                  // tiles of the first launch; pairs on a tile in the second, 1 for none
};

// Counted in blocks of K of a pair: a round takes its blocks of K and the epilogue of the last tile (6), tiles that share K
// the passing on of their sums too (4 more).
template <bool AMN, bool BMN, int MODE>
cudaError_t plan_of(const GemmParams& p, Plan& plan) {
    const int K = p.q[0].K > p.q[1].K ? p.q[0].K : p.q[1].K, kblocks = (K + kBK - 1) / kBK;
    const int whole = p.tiles / kPairs * kPairs, rest = p.tiles - whole;
    plan = {p.tiles, 1};
    if (rest == 0) return cudaSuccess;
    static KnownClusters known;
    const void* kernel = reinterpret_cast<const void*>(ffn_gemm_kernel<AMN, BMN, MODE, true>);
    int least = kblocks + (whole ? 0 : 6);
    for (int n = 2; n <= 4; ++n) {
        const int each = (kblocks + n - 1) / n;
        if (each < 4 || (kblocks + each - 1) / each != n) continue;
        int at_once;
        const cudaError_t e = clusters_at_once(kernel, known, 2 * n, kThreads, kSmem, at_once);
        if (e != cudaSuccess) return e;
        if (at_once < 1) continue;
        const int cost = (rest + at_once - 1) / at_once * (each + 10);
        if (cost < least) {
            least = cost;
            plan = {whole, n};
        }
    }
    return cudaSuccess;
}

template <bool AMN, bool BMN, int MODE, bool SPLIT>
cudaError_t launch(const Maps& m0, const Maps& m1, const GemmParams& p, int blocks, cudaStream_t s) {
    static_assert(kSmem <= 232448, "shared memory of a block");
    static_assert(!SPLIT || kStages * kStageBytes >= kTile * kBM * 4, "the sums of a block");
    return launch_in_clusters(ffn_gemm_kernel<AMN, BMN, MODE, SPLIT>, dim3(blocks), dim3(kThreads), kSmem, s,
                              SPLIT ? 2 * p.splits : 2, true, m0, m1, p);
}

template <bool AMN, bool BMN, int MODE>
cudaError_t gemm(const Maps& m0, const Maps& m1, GemmParams p, cudaStream_t s, int* launches) {
    cudaError_t e = cudaFuncSetAttribute(ffn_gemm_kernel<AMN, BMN, MODE, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(ffn_gemm_kernel<AMN, BMN, MODE, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const int all = p.tiles = p.q[0].tiles + p.q[1].tiles;
    Plan plan;
    e = plan_of<AMN, BMN, MODE>(p, plan);
    if (e != cudaSuccess) return e;
    if (plan.whole) {
        p.tiles = plan.whole;
        e = launch<AMN, BMN, MODE, false>(m0, m1, p, 2 * (plan.whole < kPairs ? plan.whole : kPairs), s);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    if (plan.whole == all) return cudaSuccess;
    p.beside = plan.whole > 0;
    p.tile0 = plan.whole;
    p.tiles = all;
    p.splits = plan.splits;
    if (plan.whole) p.debug_stall = 0;
    ++*launches;
    return launch<AMN, BMN, MODE, true>(m0, m1, p, 2 * p.splits * (all - p.tile0), s);
}

// Splits of K, of two blocks of K at least, by rounds of the clusters that run at once: a round takes its blocks of K, the
// set-up and epilogue (6) and the passing on of sums (2).  Two blocks share an SM (the query counts one where a kernel uses
// tensor memory); a launch that needs the second places (4 more) leaves none to the launch after it, whose weights could
// be on their way.  128 x 2048 x 1544 forward: 19 us with 125 blocks, 23.5 with 200; 16 x 2048 x 5504: 19.6 with 258, 22.2 with
// two thirds of them.
template <bool WMN, int MODE>
cudaError_t narrow(const CUtensorMap& mw, const Matrix& x, NarrowParams p, bool second, cudaStream_t s) {
    const int columns = MODE == kGated ? 64 : 128, tiles = (p.wide + columns - 1) / columns;
    const int kblocks = (p.K + kBK - 1) / kBK;
    const int parts = (p.N + kNarrow - 1) / kNarrow;
    const int rows = (p.N + parts - 1) / parts;
    p.bn = (rows + 15) / 16 * 16;
    auto kernel = ffn_narrow_kernel<WMN, MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNarrowSmem);
    if (e != cudaSuccess) return e;
    static KnownClusters known;
    int splits = 1;
    long long least = LLONG_MAX;
    for (int n = 1; n <= 8; ++n) {
        const int each = (kblocks + n - 1) / n;
        if (n > 1 && (each < 2 || (kblocks + each - 1) / each != n)) continue;
        int places;
        e = clusters_at_once(reinterpret_cast<const void*>(kernel), known, n, kNarrowThreads, kNarrowSmem, places);
        if (e != cudaSuccess) return e;
        if (places < 1) continue;
        const long long all = (long long)tiles * parts, rounds = (all + 2 * places - 1) / (2 * places);
        const long long cost = rounds * (each + (n > 1 ? 8 : 6)) + (all > places ? 4 : 0);
        if (cost <= least) {
            least = cost;
            splits = n;
        }
    }
    p.kblocks = (kblocks + splits - 1) / splits;
    p.second = second;
    const int stage = kOperand + p.bn * 128, room = kNarrowSmem - 1024;
    p.stages = room / stage < kNarrowStages ? room / stage : kNarrowStages;
    CUtensorMap mx;
    if (!x.map(&mx, p.bn)) return cudaErrorInvalidValue;
    return launch_in_clusters(kernel, dim3(tiles * splits, parts), dim3(kNarrowThreads), kNarrowSmem, s, splits, true, mw, mx, p);
}

// Whether a product of N rows takes the narrow kernel: always up to 128.  Up to 768 rows, parts of 128 read the weights
// again (from L2), which pays while the wide kernel's 256 x 256 tiles leave most pairs idle: with up to 48 parts of tiles
// (160 x 2048 x 5504 forward 29.2 us, wide 33.1; with the weights in L2 500 rows, 64 parts: 56.5 and 52.6), up to 152 where
// K is short and the parts of rows are few (250 x 768 x 2048 forward 16.3 and 25.9, input gradient 18.7 and 26.5; with the
// weights in L2 760 rows, 192 parts: 22.2 and 20.2; 760 x 2048 x 1544, second product: 36.8 and 28.6 in all), or where the
// tiles are a little more than a round of the pairs (330 x 2048 x 5504: 36.8 and 51.2).
bool few(int N, int K, int wide, int columns) {
    if (N <= kNarrow) return true;
    if (N > 6 * kNarrow) return false;
    const long long of_rows = (N + kNarrow - 1) / kNarrow, parts = (wide + columns - 1) / columns * of_rows;
    const long long tiles = (long long)((wide + 2 * columns - 1) / (2 * columns)) * ((N + kTile - 1) / kTile);
    return parts <= 48 || (parts <= 2 * kPairs && parts * of_rows * ((K + kBK - 1) / kBK) <= 6800) ||
           (tiles > kPairs && parts <= 4 * kPairs);
}

NarrowParams narrow_params(const FfnArgs& a) {
    NarrowParams p{};
    p.N = a.N;
    p.F = a.F;
    p.gelu = a.gelu;
    p.status = a.status;
    p.limit = a.wait_cycles > 0 ? a.wait_cycles : kWaitCycles;
    return p;
}

GemmParams params(const FfnArgs& a) {
    GemmParams p{};
    p.gelu = a.gelu;
    p.status = a.status;
    p.limit = a.wait_cycles > 0 ? a.wait_cycles : kWaitCycles;
    return p;
}

}  // namespace

size_t ffn_workspace_bytes(int N, int D, int F, int backward) {
    return (size_t)N * F * 2 * (backward ? 3 : 1);
}

cudaError_t ffn_fwd_launch(const FfnArgs& a, cudaStream_t s, int* launches) {
    const long long N = a.N, D = a.D, F = a.F;
    const Matrix x{a.x, N, D, a.x_row}, wi{a.W_in, D, 2 * F, 2 * F}, wo{a.W_out, F, D, D}, h{a.workspace, N, F, F};
    *launches = 0;
    cudaError_t e;
    if (few(a.N, a.D, a.F, 64)) {
        NarrowParams p = narrow_params(a);
        CUtensorMap w;
        p.wide = a.F;
        p.K = a.D;
        p.h = static_cast<bf16*>(a.workspace);
        p.gu = static_cast<bf16*>(a.gu);
        p.debug_stall = a.debug_stall;
        if (!wi.halves(&w, 64)) return cudaErrorInvalidValue;
        e = narrow<true, kGated>(w, x, p, false, s);
        ++*launches;
    } else {
        GemmParams p = params(a);
        p.debug_stall = a.debug_stall;
        p.q[0].out = static_cast<bf16*>(a.gu);
        p.q[0].h = static_cast<bf16*>(a.workspace);
        Maps m{};
        if (!x.operand(&m.a, false) || !wi.halves(&m.b, 64) || !problem(p.q[0], a.N, a.F, a.D, kGated))
            return cudaErrorInvalidValue;
        e = gemm<false, true, kGated>(m, m, p, s, launches);
    }
    if (e != cudaSuccess) return e;
    if (few(a.N, a.F, a.D, 128)) {
        NarrowParams o = narrow_params(a);
        CUtensorMap w;
        o.wide = a.D;
        o.K = a.F;
        o.out = static_cast<bf16*>(a.y);
        o.add = static_cast<const bf16*>(a.residual);
        o.add_row = a.residual_row;
        if (!wo.operand(&w, true)) return cudaErrorInvalidValue;
        ++*launches;
        return narrow<true, kStore>(w, h, o, true, s);
    }
    GemmParams o = params(a);
    Maps n{};
    if (!h.operand(&n.a, false) || !wo.operand(&n.b, true) || !problem(o.q[0], a.N, a.D, a.F, kStore))
        return cudaErrorInvalidValue;
    o.q[0].out = static_cast<bf16*>(a.y);
    o.q[0].add = static_cast<const bf16*>(a.residual);
    o.q[0].add_row = a.residual_row;
    return gemm<false, true, kStore>(n, n, o, s, launches);
}

cudaError_t ffn_bwd_launch(const FfnArgs& a, cudaStream_t s, int* launches) {
    const long long N = a.N, D = a.D, F = a.F;
    char* ws = static_cast<char*>(a.workspace);
    const Matrix x{a.x, N, D, a.x_row}, wi{a.W_in, D, 2 * F, 2 * F}, wo{a.W_out, F, D, D}, dy{a.dy, N, D, a.dy_row},
        dgu{ws, N, 2 * F, 2 * F}, h{ws + (size_t)N * F * 4, N, F, F};
    *launches = 0;
    cudaError_t e;
    if (few(a.N, a.D, a.F, 128)) {
        NarrowParams p = narrow_params(a);
        CUtensorMap w;
        p.wide = a.F;
        p.K = a.D;
        p.out = static_cast<bf16*>(const_cast<void*>(dgu.p));
        p.h = static_cast<bf16*>(const_cast<void*>(h.p));
        p.gu = static_cast<bf16*>(a.gu);
        p.debug_stall = a.debug_stall;
        if (!wo.operand(&w, false)) return cudaErrorInvalidValue;
        e = narrow<false, kGatedBack>(w, dy, p, false, s);
        ++*launches;
    } else {
        GemmParams p = params(a);
        p.debug_stall = a.debug_stall;
        p.q[0].add = static_cast<const bf16*>(a.gu);
        p.q[0].add_row = 2LL * a.F;
        p.q[0].out = static_cast<bf16*>(const_cast<void*>(dgu.p));
        p.q[0].h = static_cast<bf16*>(const_cast<void*>(h.p));
        Maps m{};
        if (!dy.operand(&m.a, false) || !wo.operand(&m.b, false) ||
            !problem(p.q[0], a.N, a.F, a.D, kGatedBack))
            return cudaErrorInvalidValue;
        e = gemm<false, false, kGatedBack>(m, m, p, s, launches);
    }
    if (e != cudaSuccess) return e;
    if (a.dx && few(a.N, 2 * a.F, a.D, 128)) {
        NarrowParams o = narrow_params(a);
        CUtensorMap w;
        o.wide = a.D;
        o.K = 2 * a.F;
        o.out = static_cast<bf16*>(a.dx);
        if (!wi.operand(&w, false)) return cudaErrorInvalidValue;
        e = narrow<false, kStore>(w, dgu, o, true, s);
        if (e != cudaSuccess) return e;
        ++*launches;
    } else if (a.dx) {
        GemmParams o = params(a);
        Maps n{};
        if (!dgu.operand(&n.a, false) || !wi.operand(&n.b, false) || !problem(o.q[0], a.N, a.D, 2 * a.F, kStore))
            return cudaErrorInvalidValue;
        o.q[0].out = static_cast<bf16*>(a.dx);
        e = gemm<false, false, kStore>(n, n, o, s, launches);
        if (e != cudaSuccess) return e;
    }
    if (!a.dW_in && !a.dW_out) return cudaSuccess;
    // both weights' products together: few tiles each, so that one's last round fills up with the other's
    GemmParams o = params(a);
    Maps n[2] = {};
    int k = 0;
    if (a.dW_in) {
        if (!x.operand(&n[k].a, true) || !dgu.operand(&n[k].b, true) || !problem(o.q[k], a.D, 2 * a.F, a.N, kStore))
            return cudaErrorInvalidValue;
        o.q[k++].out = static_cast<bf16*>(a.dW_in);
    }
    if (a.dW_out) {
        if (!h.operand(&n[k].a, true) || !dy.operand(&n[k].b, true) || !problem(o.q[k], a.F, a.D, a.N, kStore))
            return cudaErrorInvalidValue;
        o.q[k].out = static_cast<bf16*>(a.dW_out);
    }
    return gemm<true, true, kStore>(n[0], n[1], o, s, launches);
}

}  // namespace ttm
