// Gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t, its gradient and its
// decode step.
//
// Mathematics.  With a_t = exp(g_t), a run of tokens acts on the state before it
// as the affine map h -> A h + H, A the product of the run's a_t and H its result
// from zero; two runs in a row give (A2 A1, A2 H1 + H2), which is associative.  The
// gradient is the same recurrence from the last token on: with c_T = dh_last,
//   G_t = dh_t + c_{t+1},  c_t = a_t G_t,
//   dx_t = G_t,  dg_t = c_t h_{t-1} (summed over the channels for a token gate),  dh0 = c_0,
// so a run acts on c as c -> A c + H too and needs no gate of a neighbouring run.
//
// What bounds it: HBM.  Three tensors move in the forward direction (x, g, h), five
// in the gradient (g, h, dh, dx, dg), and each value takes a handful of operations.
// Every input is therefore read once: a block holds a tile of tokens in shared
// memory, takes its map (A, H) in a first pass over it, learns the state before the
// tile from the blocks of the tiles before, and writes the outputs in a second pass.
//
// Tile: 256 threads, each 4 channels times R consecutive tokens, CW threads side by
// side over a strip of channels and 256 / CW over the tokens (make_plan chooses CW).
// The runs of a warp are joined by shuffles, the eight warps' through shared memory.
//
// Measured, a gate per channel: bf16 forward 16 x 131072 x 128 258 us (6.3 TB/s, 92 % of what a copy
// reaches), 256 x 8192 x 128 238 us (6.8 TB/s); gradient 96 x 8192 x 64 83 us (6.1 TB/s); one tile,
// 2 x 777 x 768, 6.3 us; fp32 forward 16 x 65536 x 128 242 us (6.7 TB/s), gradient 96 x 8192 x 64 150 us (6.7
// TB/s).  A gate per token: forward 16 x 131072 x 128 bf16 238 us and 16 x 65536 x 128 fp32 206 us (4.6 and
// 5.2 TB/s: a token's arithmetic is the same for a third less of traffic), gradient 96 x 8192 x 64 bf16 83,
// fp32 108 us (3.7 and 5.7 TB/s: each token's sum over the channels besides).
//
// Between tiles (look-back), a lane per channel: a warp publishes its channels' map of
// the tile as soon as it has it, finds the nearest tile before whose end state is known,
// takes that state through the maps in between (read 8 at a time) and publishes its own
// end state.  Every end state is thus the tile's map applied to the one before, however
// far back a warp had to start: the result does not depend on timing.  A map is one
// 64-bit word and an end state one 32-bit word per channel, each its own flag (a bit
// pattern that the values never take marks an empty word), so neither side needs a
// fence: with release / acquire the two publications took 6600 of a tile's 23700 cycles.
// Tiles are handed out in order by a counter, so a block only ever waits for blocks
// that are already running.  The waits are bounded: one that runs out sets the
// device status word and the call's outputs are invalid.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/ttm.h"
#include "pairs.cuh"
#include "tc_ptx.cuh"
#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int V = 4;                          // channels of a thread
constexpr int kMaxLog = 4;                        // at most 16 threads over the channels
constexpr int kChans = V << kMaxLog;          // channels of a full strip
constexpr int kNear = 4, kBatch = 8;              // tiles a look-back takes with the hints; maps then
constexpr long long kWaitCycles = 4000000000LL;   // default limit, ~2 s at 2 GHz
constexpr long long kDrainCycles = 20000000LL;    // ~10 ms, for copies in flight

// R, the tokens of one thread in a tile: its two tensors (three in the gradient with a gate per
// channel, which gets half the tokens) take 64 (48) registers.
template <typename E, bool kToken, bool kBack>
constexpr int kRun = (sizeof(E) == 2 ? 16 : 8) / (kBack && !kToken ? 2 : 1);
template <typename E, bool kToken, bool kBack>
constexpr int kTileBytes = kThreads * kRun<E, kToken, kBack> * V * (int)sizeof(E);

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float v) { o = __float2bfloat16(v); }

// Four channels as they are stored.
template <typename E> struct Held;
template <> struct Held<float> {
    float4 u;
    __device__ __forceinline__ void load(const float* p) { u = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(f2 (&f)[2]) const { f[0] = pair(u.x, u.y); f[1] = pair(u.z, u.w); }
    __device__ __forceinline__ void set(const f2 (&f)[2]) { split(f[0], u.x, u.y); split(f[1], u.z, u.w); }
    __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = u; }
    __device__ __forceinline__ void repack() {}
};
template <> struct Held<__nv_bfloat16> {
    uint2 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void get(f2 (&f)[2]) const { f[0] = pair_of_bf16(u.x); f[1] = pair_of_bf16(u.y); }
    __device__ __forceinline__ void set(const f2 (&f)[2]) { u = make_uint2(bf16_of_pair(f[0]), bf16_of_pair(f[1])); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = u; }
    // forgets the unpacked values: cheaper to take again than to keep over the look-back
    __device__ __forceinline__ void repack() { asm volatile("" : "+r"(u.x), "+r"(u.y)); }
};
__device__ __forceinline__ void get4(const float* p, float (&f)[V]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
}
__device__ __forceinline__ void get4(const __nv_bfloat16* p, float (&f)[V]) {
    Held<__nv_bfloat16> h;
    f2 q[2];
    h.load(p);
    h.get(q);
    split(q[0], f[0], f[1]);
    split(q[1], f[2], f[3]);
}
__device__ __forceinline__ void put4(float* p, const float (&f)[V]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void put4(__nv_bfloat16* p, const float (&f)[V]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_of_pair(pair(f[0], f[1])), bf16_of_pair(pair(f[2], f[3])));
}

// exp of gates of type G; -infinity gives 0.  An fp32 gate takes expf (2 units in the last place).  A bf16
// gate takes the base-2 unit on the rounded product with log2 e, which adds |g| 2^-24 of the
// result, 2^-15 of what half a unit of the gate itself is worth.
template <typename G>
__device__ __forceinline__ float retention(float g) {
    if constexpr (sizeof(G) == 4) {
        return expf(g);
    } else {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(g * 1.44269504088896341f));
        return r;
    }
}

template <typename G>
__device__ __forceinline__ void retention(const f2 (&g)[2], f2 (&r)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float lo, hi;
        if constexpr (sizeof(G) == 4) {
            split(g[i], lo, hi);
            lo = expf(lo);
            hi = expf(hi);
        } else {
            split(mul(g[i], splat<f2>(1.44269504088896341f)), lo, hi);
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(lo));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(hi));
        }
        r[i] = pair(lo, hi);
    }
}

// R^2 c + H for the map (A, H) with R the root of A.  Growing gates may take A past fp32's range
// while A c is well inside it (gates of 0.05 over 2000 tokens, a state of 1e-30); the root has
// twice the range, which is that of A c for any state but zero, which stays out of the product.
__device__ __forceinline__ float apply(float R, float H, float c) {
    return c == 0.f ? H : fmaf(c * R, R, H);
}
// The root of a run's A (to 2^-23, once for the 4 to 16 retentions that A is the product of); an A of
// infinity times 0 is one that a forgetting gate (-infinity) has cut off.
__device__ __forceinline__ float root(float A) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(A));
    return A == A ? r : 0.f;
}

// ------------------------------------------------------------ global <-> shared

// Widest access all rows of a view allow, in bytes.
inline int access_width(const void* p, long long seq, long long tok, int es) {
    const unsigned long long m =
        reinterpret_cast<uintptr_t>(p) | (unsigned long long)seq * es | (unsigned long long)tok * es;
    return m % 16 == 0 ? 16 : (m % 8 == 0 ? 8 : (m % 4 == 0 ? 4 : es));
}

// Copies rows [0, rows) of `bytes` bytes at `pitch` bytes from global memory, wherever they
// start, into shared rows of `srow` bytes (a multiple of 8), 16 at a time; rows below `lo` or
// from `hi` on and bytes past the end read as zero.  Global memory is read in aligned 16-byte
// words that hold at least one byte of the row, and two of them shifted into place: 436 x
// 508 x 768 bf16 from rows of 771 values took 300 us in loads of two bytes.
__device__ __forceinline__ void load_rows(unsigned char* dst, int rows, int srow, const char* src,
                                          long long pitch, int lo, int hi, int bytes) {
    constexpr int kFlight = 4;                        // pairs of loads a thread has in flight
    const int per = max(1, srow / 16);                // threads a row, a power of two
    const int o = (threadIdx.x & (per - 1)) * 16, step = kThreads / per;
    const int left = bytes - o;                       // of the row, from this thread's bytes on
    for (int r = threadIdx.x / per; r < rows; r += kFlight * step) {
        uint4 u[kFlight], v[kFlight];
        int sh[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int q = r + k * step;
            const char* p = src + q * pitch + o;
            sh[k] = (int)(reinterpret_cast<uintptr_t>(p) & 15);
            const uint4* w = reinterpret_cast<const uint4*>(p - sh[k]);
            const bool in = q >= lo && q < hi && left > 0;
            u[k] = in ? w[0] : make_uint4(0, 0, 0, 0);
            v[k] = in && sh[k] + left > 16 && sh[k] ? w[1] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            uint32_t w[8] = {u[k].x, u[k].y, u[k].z, u[k].w, v[k].x, v[k].y, v[k].z, v[k].w};
            if (sh[k] & 8)
#pragma unroll
                for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
            if (sh[k] & 4)
#pragma unroll
                for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = __funnelshift_r(w[i], w[i + 1], (sh[k] & 3) * 8);
                if (left < 4 * i + 4) w[i] = left == 4 * i + 2 ? w[i] & 0xffffu : 0u;
            }
            const int q = r + k * step;
            if (q >= rows) continue;
            unsigned char* to = dst + q * srow + o;
            if (srow >= 16) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        }
    }
}

// Shared rows back to global memory where a row does not start on 16 bytes:
// neighbouring threads write neighbouring values.
template <typename U>
__device__ __forceinline__ void store_rows_by(char* dst, long long pitch, const unsigned char* src,
                                              int rows, int srow, int bytes) {
    const int per = srow / (int)sizeof(U), o = (threadIdx.x & (per - 1)) * (int)sizeof(U);
    if (o >= bytes) return;
#pragma unroll 8
    for (int r = threadIdx.x / per; r < rows; r += kThreads / per)
        *reinterpret_cast<U*>(dst + r * pitch + o) = *reinterpret_cast<const U*>(src + r * srow + o);
}
__device__ __forceinline__ void store_rows(char* dst, long long pitch, const unsigned char* src, int rows,
                                           int srow, int bytes, int width) {
    if (width == 8) store_rows_by<uint2>(dst, pitch, src, rows, srow, bytes);
    else if (width == 4) store_rows_by<uint32_t>(dst, pitch, src, rows, srow, bytes);
    else store_rows_by<unsigned short>(dst, pitch, src, rows, srow, bytes);
}

// ------------------------------------------------------------------- look-back

struct TilePlan {
    int cw_log;            // log2 of the threads side by side over the channels
    int tokens;            // of a tile
    int ntiles, ncols;     // tiles of a sequence, strips of channels
    unsigned* counter;     // hands out tiles in order; NULL when ntiles == 1
    unsigned long long* maps;   // [strip][tile][channel] in processing order: root of A low, H high word
    unsigned* ends;        // [strip][tile][channel]: state after the tile
    unsigned* hints;       // [strip][32 channels][tile]: kMapThere, kEndThere
    size_t words_bytes;    // of the counter, maps, ends and hints, all set to kEmpty before
    unsigned tiles;        // of all strips
    int tma, tma_out;      // inputs, outputs by tensor copies
    int x_first, g_first;  // x, g have their tokens further apart than their sequences
    int width_o;           // else: access width of the outputs' rows
    float* dg_part;        // token gate over several strips: [ncols][N T] partial sums
};

constexpr unsigned kEmpty = 0xffffffffu;   // as a float a NaN that full() never lets through
constexpr unsigned kMapThere = 1, kEndThere = 2;

__device__ __forceinline__ unsigned full(float v) {
    const unsigned u = __float_as_uint(v);
    return u == kEmpty ? 0x7fffffffu : u;
}
__device__ __forceinline__ unsigned load_word(const unsigned* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long load_word(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_word(unsigned* p, unsigned v) {
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ void publish_end(unsigned* p, float v) {
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(full(v)) : "memory");
}
__device__ __forceinline__ void publish_map(unsigned long long* p, float A, float H) {
    const unsigned long long w =
        (unsigned long long)full(H) << 32 | (unsigned long long)__float_as_uint(A);
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}
__device__ __forceinline__ bool has_map(unsigned long long w) { return (unsigned)(w >> 32) != kEmpty; }
__device__ __forceinline__ float apply_map(unsigned long long w, float s) {
    return apply(__uint_as_float((unsigned)w), __uint_as_float((unsigned)(w >> 32)), s);
}

// Shared memory behind the input tiles.
struct Joints {
    float a[kWarps][kChans], h[kWarps][kChans];   // map of each warp's tokens, by channel (roots)
    float carry[kChans];                          // state before the tile
    unsigned ticket;
    unsigned long long arrived;                   // mbarrier of the tensor copies
};

// Sums of v[0 .. 2N-1] over groups of 2D lanes by exchanging halves: lane l of a group is left
// with the sums of the values whose index agrees with it in the bits exchanged, in v[0 ..].
template <int N, int D>
__device__ __forceinline__ void scatter_sums(float* v) {
    const bool up = threadIdx.x & D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float mine = up ? v[i + N] : v[i], other = up ? v[i] : v[i + N];
        v[i] = mine + __shfl_xor_sync(0xffffffffu, other, D);
    }
    if constexpr (N > 1) scatter_sums<N / 2, D / 2>(v);
}

// One warp, a lane per channel (mine: the lane has one): the state before tile j > 0.
// maps and ends point to this lane's channel of tile j, `chans` words a tile; hints to
// the warp's word of tile j.  The words of the nearest four tiles come in the same round
// trip as the hints, which say in one load where the nearest end state of the 32 tiles
// before is and that the maps in between are out; they are not ordered with the words
// themselves, each of which is looked at until it is there.
__device__ __forceinline__ float look_back(const unsigned* hints, const unsigned long long* maps,
                                           const unsigned* ends, int chans, int j, bool mine, int* status,
                                           long long limit) {
    const int lane = threadIdx.x & 31;
    const long long t0 = clock64();
    auto late = [&]() {
        if (!__any_sync(0xffffffffu, clock64() - t0 > limit)) return false;
        if (lane == 0) atomicExch(status, TTM_ERR_TIMEOUT);
        return true;
    };
    int back;                                         // distance of the end state
    while (true) {
        const unsigned f = lane < j ? load_word(hints - 1 - lane) : kMapThere;
        unsigned ne[kNear];
        unsigned long long nm[kNear];
#pragma unroll
        for (int u = 0; u < kNear; ++u) {
            const bool in = mine && u < j;
            ne[u] = in ? load_word(ends - (long long)(u + 1) * chans) : (u < j ? 0u : kEmpty);
            nm[u] = in ? load_word(maps - (long long)(u + 1) * chans) : 0ull;
        }
        bool open = true;                             // every map nearer than u is there
#pragma unroll
        for (int u = 0; u < kNear; ++u) {
            if (open && __all_sync(0xffffffffu, ne[u] != kEmpty)) {
                float s = __uint_as_float(ne[u]);
#pragma unroll
                for (int w = kNear - 1; w >= 0; --w)
                    if (w < u) s = apply_map(nm[w], s);
                return s;
            }
            open = open && __all_sync(0xffffffffu, has_map(nm[u]));
        }
        const unsigned out = __ballot_sync(0xffffffffu, f != kEmpty);
        const unsigned end = __ballot_sync(0xffffffffu, f == kEndThere);
        back = __ffs(end);
        const unsigned nearer = (end & (0u - end)) - 1u;
        if (end && (out & nearer) == nearer) break;
        if (late()) return 0.f;
    }
    unsigned e;
    unsigned long long m[kBatch];
    int d = back - 1;                                 // distance of the next map
    float s = 0.f;
    bool first = true;
    do {
        while (true) {
            bool there = true;
            if (first) {
                e = mine ? load_word(ends - (long long)back * chans) : 0u;
                there = e != kEmpty;
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                m[u] = mine && d - u > 0 ? load_word(maps - (long long)(d - u) * chans) : 0ull;
                there = there && has_map(m[u]);
            }
            if (__all_sync(0xffffffffu, there)) break;
            if (late()) return 0.f;
        }
        if (first) s = __uint_as_float(e);
        first = false;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (d - u > 0) s = apply_map(m[u], s);
        d -= kBatch;
    } while (d > 0);
    return s;
}

// ------------------------------------------------------------------ tile kernel

// Blocks an SM: what registers and shared memory leave room for.
template <bool kToken, bool kBack> constexpr int kResident = kToken && !kBack ? 3 : 2;

// Persistent.  A block takes a tile from shared memory into registers, so that the next tile's
// copies run while it looks back and writes this one's results.
template <typename E, bool kToken, bool kBack>
__global__ void __launch_bounds__(kThreads, kResident<kToken, kBack>)
    glr_tile_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
                    const __grid_constant__ CUtensorMap mh, const __grid_constant__ CUtensorMap mo,
                    const __grid_constant__ CUtensorMap mog, const __grid_constant__ GlrArgs a,
                    const __grid_constant__ TilePlan p) {
    constexpr int R = kRun<E, kToken, kBack>;
    constexpr int kIns = 1 + (kToken ? 0 : 1) + (kBack ? 1 : 0);
    constexpr uint32_t kBytes = kTileBytes<E, kToken, kBack>;
    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char* sx = smem;                                        // x or dh
    unsigned char* sg = smem + (kToken ? 0 : kBytes);                // g (gate per channel)
    unsigned char* sh = smem + (kIns - 1) * kBytes;                  // gradient: h one token earlier
    unsigned char* so = smem + kIns * kBytes;                        // h or dx
    unsigned char* sog = so + kBytes;                                // gradient: dg (gate per channel)
    Joints& J = *reinterpret_cast<Joints*>(so + (kBack && !kToken ? 2 : 1) * kBytes);
    float* sgt = reinterpret_cast<float*>(&J + 1);    // token gate: a tile's retentions, two in turn
    uint64_t* arrived = reinterpret_cast<uint64_t*>(&J.arrived);

    const int tid = threadIdx.x, warp = tid >> 5;
    const int chans = V << p.cw_log, srow = chans * (int)sizeof(E);  // a strip's channels, their bytes
    const unsigned strips = (unsigned)a.N * p.ncols;
    // this thread's channels and run of tokens, in processing order
    const int cw = 1 << p.cw_log, ch = (tid & (cw - 1)) * V;
    const int place = tid >> p.cw_log, runs = kThreads >> p.cw_log;
    const int r0 = (kBack ? runs - 1 - place : place) * R;
    const int own = r0 * chans + ch;                  // its first value of a tile
    const int swarps = (chans + 31) / 32;             // warps with a lane per channel

    // Tiles in order, all strips of the first one first: from the counter (it starts at
    // kEmpty = -1), or, where no tile waits for another, every gridDim-th
    auto request = [&](unsigned ticket) {             // thread 0: the tile's tensor copies
        const unsigned strip = ticket % strips;
        const int j = ticket / strips, n = strip / p.ncols, c0 = (strip % p.ncols) * chans;
        const int t0 = (kBack ? p.ntiles - 1 - j : j) * p.tokens;
        // (a test of the waits has more announced than comes)
        tc::mbar_expect_tx(arrived, kIns * kBytes + (ticket + 1 == a.debug_stall ? 16u : 0u));
        const int box = min(p.tokens, 256);
        for (int r = 0; r < p.tokens; r += box) {
            tc::tma_load_3d(sx + r * srow, &mx, arrived, c0, p.x_first ? n : t0 + r, p.x_first ? t0 + r : n);
            if (!kToken)
                tc::tma_load_3d(sg + r * srow, &mg, arrived, c0, p.g_first ? n : t0 + r, p.g_first ? t0 + r : n);
            // row r of sh holds h of token t0 + r - 1; token -1 is h0, taken below
            if (kBack) tc::tma_load_3d(sh + r * srow, &mh, arrived, c0, t0 + r - 1, n);
        }
    };
    // token gate: copies of a tile's gates, waited for before the barrier that ends a tile
    auto request_gates = [&](unsigned ticket, unsigned turn) {
        const unsigned strip = ticket % strips;
        const int j = ticket / strips, t0 = (kBack ? p.ntiles - 1 - j : j) * p.tokens;
        const float* g = static_cast<const float*>(a.g) + (strip / p.ncols) * a.g_seq + (long long)t0 * a.g_tok;
        float* to = sgt + turn * p.tokens;
        for (int i = tid; i < p.tokens; i += kThreads) {
            const bool in = t0 + i < a.T;             // past the end: 0, which keeps the state
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(tc::smem_u32(to + i)),
                         "l"(in ? g + (long long)i * a.g_tok : static_cast<const float*>(a.g)), "r"(in ? 4 : 0)
                         : "memory");
        }
    };
    // waits for this thread's and leaves their retentions in their place, once a token for all channels
    auto gates_arrived = [&](bool any, unsigned turn) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (any)
            for (int i = tid; i < p.tokens; i += kThreads) {
                float& g = sgt[turn * p.tokens + i];
                g = retention<float>(g);
            }
    };
    if (tid == 0) {
        J.ticket = p.counter ? atomicAdd(p.counter, 1u) + 1u : blockIdx.x;
        if (p.tma) {
            tc::mbar_init(arrived, 1);
            tc::fence_mbar_init();
            if (J.ticket < p.tiles) request(J.ticket);
        }
    }
    __syncthreads();
    if (kToken) {
        if (J.ticket < p.tiles) request_gates(J.ticket, 0);
        gates_arrived(J.ticket < p.tiles, 0);
        __syncthreads();
    }

    unsigned phase = 0;
    for (unsigned ticket = J.ticket; ticket < p.tiles; ticket = J.ticket, phase ^= 1u) {
        const unsigned strip = ticket % strips;
        const int j = ticket / strips;                // place in processing order
        const size_t n = strip / p.ncols;
        const int c0 = (strip % p.ncols) * chans;
        const int t0 = (kBack ? p.ntiles - 1 - j : j) * p.tokens;
        const int ntok = min(p.tokens, a.T - t0);
        const int bytes = min(chans, a.D - c0) * (int)sizeof(E);
        const size_t row0 = n * a.T + t0;             // row of the contiguous tensors
        const bool live = c0 + ch < a.D;
        unsigned next = 0;
        if (tid == 0) next = p.counter ? atomicAdd(p.counter, 1u) + 1u : ticket + gridDim.x;

        bool late = false;                            // the copies did not come
        if (p.tma) {
            const long long since = clock64();
            while (!late && !tc::mbar_try_wait(arrived, phase))
                if (clock64() - since > a.wait_cycles) {
                    atomicExch(a.status, TTM_ERR_TIMEOUT);
                    late = true;
                }
        } else {
            load_rows(sx, p.tokens, srow,
                         reinterpret_cast<const char*>(static_cast<const E*>(a.x) + n * a.x_seq +
                                                       (long long)t0 * a.x_tok + c0),
                         a.x_tok * (long long)sizeof(E), 0, ntok, bytes);
            if (!kToken)
                load_rows(sg, p.tokens, srow,
                             reinterpret_cast<const char*>(static_cast<const E*>(a.g) + n * a.g_seq +
                                                           (long long)t0 * a.g_tok + c0),
                             a.g_tok * (long long)sizeof(E), 0, ntok, bytes);
            if (kBack)
                load_rows(sh, p.tokens, srow,
                             reinterpret_cast<const char*>(static_cast<const E*>(a.h) + c0) +
                                 ((long long)row0 - 1) * a.D * (long long)sizeof(E),
                             (long long)a.D * sizeof(E), t0 == 0 ? 1 : 0, ntok, bytes);
            __syncthreads();
        }
        Held<E> hx[R], hg[kToken ? 1 : R], hh[kBack ? R : 1];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            hx[q].load(reinterpret_cast<const E*>(sx) + own + q * chans);
            if (!kToken) hg[q].load(reinterpret_cast<const E*>(sg) + own + q * chans);
            if (kBack) hh[q].load(reinterpret_cast<const E*>(sh) + own + q * chans);
        }
        const float* gt = sgt + phase * p.tokens + r0;
        auto retain = [&](int q, f2 (&r)[2]) {        // of token r0 + q
            if constexpr (kToken) {
                r[0] = r[1] = splat<f2>(gt[q]);
            } else {
                f2 g[2];
                hg[q].get(g);
                retention<E>(g, r);
            }
        };

        // This run's map; from here on A is its root
        float A[V], H[V];
        {
            f2 mA[2] = {splat<f2>(1.f), splat<f2>(1.f)}, mH[2] = {splat<f2>(0.f), splat<f2>(0.f)};
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int q = kBack ? R - 1 - i : i;
                f2 x[2], r[2];
                hx[q].get(x);
                retain(q, r);
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    mH[v] = kBack ? mul(r[v], add(mH[v], x[v])) : fma(r[v], mH[v], x[v]);
                    mA[v] = mul(mA[v], r[v]);
                }
            }
            split(mA[0], A[0], A[1]);
            split(mA[1], A[2], A[3]);
            split(mH[0], H[0], H[1]);
            split(mH[1], H[2], H[3]);
            A[0] = root(A[0]);
#pragma unroll
            for (int v = 1; v < V; ++v) A[v] = kToken ? A[0] : root(A[v]);
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
            hx[q].repack();
            if (!kToken) hg[q].repack();
            if (kBack) hh[q].repack();
        }

        // Join over the runs of a warp (inclusive), then over the warps
        for (int d = cw; d < 32; d <<= 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float pa = __shfl_up_sync(0xffffffffu, A[v], d);
                const float ph = __shfl_up_sync(0xffffffffu, H[v], d);
                if ((tid & 31) >= d) {
                    H[v] = apply(A[v], H[v], ph);
                    A[v] *= pa;
                }
            }
        }
        if ((tid & 31) >= 32 - cw) {
            put4(&J.a[warp][ch], A);
            put4(&J.h[warp][ch], H);
        }
        if (cw < 32) {   // exclusive of this thread's own run
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = __shfl_up_sync(0xffffffffu, A[v], cw);
                H[v] = __shfl_up_sync(0xffffffffu, H[v], cw);
            }
        }
        if ((tid & 31) < cw) {
#pragma unroll
            for (int v = 0; v < V; ++v) { A[v] = 1.f; H[v] = 0.f; }
        }
        // Maps written, the tile is in registers.  If a thread's wait ran out the block hands out no
        // result and asks for no copy any more: it leaves once the last ones have had time to land.
        if (__syncthreads_or(late)) {
            if (tid == 0) {
                const long long since = clock64();
                while (!tc::mbar_try_wait(arrived, phase) &&
                       clock64() - since < max(a.wait_cycles, kDrainCycles)) {
                }
            }
            break;
        }

        if (tid == 0) {
            J.ticket = next;
            if (p.tma && next < p.tiles) request(next);
        }
        // A lane per channel: publish the tile's map, look back, publish the state after it.
        // Every state after a tile is that tile's map applied to the state before, wherever
        // the look-back started, so equal inputs give equal bits.
        if (warp < swarps) {
            const bool mine = tid < chans;
            float before = 0.f;
            if (j == 0) {
                const float* init = kBack ? a.dh_last : a.h0;
                if (init && mine && c0 + tid < a.D) before = init[n * a.D + c0 + tid];
            }
            if (p.counter) {
                const size_t word = ((size_t)strip * p.ntiles + j) * chans + tid;
                float mA = 1.f, mH = 0.f;
                if (mine) {
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        mH = apply(J.a[w][tid], J.h[w][tid], mH);
                        mA *= J.a[w][tid];
                    }
                }
                unsigned* hint = p.hints + ((size_t)strip * swarps + warp) * p.ntiles + j;
                const bool tell = j + 1 < p.ntiles;
                if (tell && j > 0) {
                    if (mine) publish_map(p.maps + word, mA, mH);
                    __syncwarp();
                    if ((tid & 31) == 0) store_word(hint, kMapThere);
                }
                if (j > 0)
                    before = look_back(hint, p.maps + word, p.ends + word, chans, j, mine, a.status,
                                       a.wait_cycles);
                if (tell) {
                    if (mine) publish_end(p.ends + word, apply(mA, mH, before));
                    __syncwarp();
                    if ((tid & 31) == 0) store_word(hint, kEndThere);
                }
            }
            if (mine) J.carry[tid] = before;
        }
        if (p.tma_out && tid == 0) tc::bulk_wait_read<0>();   // the results before have left
        __syncthreads();
        if (kToken && J.ticket < p.tiles) request_gates(J.ticket, phase ^ 1u);

        // State before this thread's run: the tile's, through the warps before, then the
        // runs before in this warp
        f2 s[2];
        {
            float f[V];
            get4(&J.carry[ch], f);
            for (int w = 0; w < warp; ++w) {
                float wa[V], wh[V];
                get4(&J.a[w][ch], wa);
                get4(&J.h[w][ch], wh);
#pragma unroll
                for (int v = 0; v < V; ++v) f[v] = apply(wa[v], wh[v], f[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = apply(A[v], H[v], f[v]);
            s[0] = pair(f[0], f[1]);
            s[1] = pair(f[2], f[3]);
        }
        float* dg = nullptr;                          // token gate: its gradient, or a strip's share
        if (kBack && kToken)
            dg = (p.ncols > 1 ? p.dg_part + (size_t)(strip % p.ncols) * a.N * a.T
                              : static_cast<float*>(a.dg)) + row0;
        float share[kBack && kToken ? R : 1];         // token gate: this thread's share of dg
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int q = kBack ? R - 1 - i : i;
            f2 x[2], r[2], o[2];
            hx[q].get(x);
            retain(q, r);
            if (!kBack) {
#pragma unroll
                for (int v = 0; v < 2; ++v) o[v] = s[v] = fma(r[v], s[v], x[v]);
            } else {
                f2 b[2];
                hh[q].get(b);
                if (q == 0 && t0 + r0 == 0 && a.h0 && live) {
                    float f[V];
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        f[v] = c0 + ch + v < a.D ? a.h0[n * a.D + c0 + ch + v] : 0.f;
                    b[0] = pair(f[0], f[1]);
                    b[1] = pair(f[2], f[3]);
                }
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    o[v] = add(x[v], s[v]);
                    s[v] = mul(r[v], o[v]);
                    b[v] = mul(b[v], s[v]);
                }
                if (kToken) {
                    share[q] = total(add(b[0], b[1]));
                } else {
                    Held<E> w;
                    w.set(b);
                    w.store(reinterpret_cast<E*>(sog) + own + q * chans);
                }
            }
            Held<E> w;
            w.set(o);
            w.store(reinterpret_cast<E*>(so) + own + q * chans);
        }

        if constexpr (kBack && kToken) {
            // over the cw threads of the strip's channels, lanes of one warp
            if (cw == 16) {
                if (R == 8) {                         // 16 lanes for 8 values: add their halves first
#pragma unroll
                    for (int q = 0; q < R; ++q) share[q] += __shfl_xor_sync(0xffffffffu, share[q], 8);
                }
                scatter_sums<R / 2, R / 2>(share);
                const int q = tid & (R - 1);
                if ((tid & 15) < R && r0 + q < ntok) dg[r0 + q] = share[0];
            } else {
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    for (int d = cw >> 1; d; d >>= 1) share[q] += __shfl_xor_sync(0xffffffffu, share[q], d);
                    if (ch == 0 && r0 + q < ntok) dg[r0 + q] = share[q];
                }
            }
        }

        // End of the strip: the tokens past T leave the state as it is
        float* end = kBack ? a.dh0 : a.h_last;
        if (j == p.ntiles - 1 && place == runs - 1 && end) {
            float f[V];
            split(s[0], f[0], f[1]);
            split(s[1], f[2], f[3]);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (c0 + ch + v < a.D) end[n * a.D + c0 + ch + v] = f[v];
        }
        if (p.tma_out) tc::fence_proxy_async_smem();
        if (kToken) gates_arrived(J.ticket < p.tiles, phase ^ 1);
        __syncthreads();
        if (p.tma_out) {
            if (tid == 0) {
                const int box = min(p.tokens, 256);
                for (int r = 0; r < ntok; r += box) {
                    tc::tma_store_3d(&mo, so + r * srow, c0, t0 + r, (int)n);
                    if (kBack && !kToken) tc::tma_store_3d(&mog, sog + r * srow, c0, t0 + r, (int)n);
                }
                tc::bulk_commit();
            }
        } else {
            char* o = reinterpret_cast<char*>(static_cast<E*>(kBack ? a.dx : a.h) + row0 * a.D + c0);
            store_rows(o, (long long)a.D * sizeof(E), so, ntok, srow, bytes, p.width_o);
            if (kBack && !kToken) {
                o = reinterpret_cast<char*>(static_cast<E*>(a.dg) + row0 * a.D + c0);
                store_rows(o, (long long)a.D * sizeof(E), sog, ntok, srow, bytes, p.width_o);
            }
        }
    }
    if (p.tma_out && tid == 0) tc::bulk_wait_read<0>();       // the block's shared memory goes with it
}

// dg of a token gate from the strips' partial sums, in the strips' order.
__global__ void glr_gate_sum_kernel(const float* part, int ncols, size_t n, float* dg) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int c = 0; c < ncols; ++c) s += part[c * n + i];
    dg[i] = s;
}

// W neighbouring channels, W = 1, 4 or 8, at once (16 bytes at most in one access).
template <typename E, int W>
__device__ __forceinline__ void get_wide(const E* p, float (&f)[W]) {
    if constexpr (W == 1) {
        f[0] = to_f(*p);
    } else if constexpr (sizeof(E) == 2 && W == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) get4(p + i, *reinterpret_cast<float(*)[4]>(f + i));
    }
}
template <typename E, int W>
__device__ __forceinline__ void put_wide(E* p, const float (&f)[W]) {
    if constexpr (W == 1) {
        put(*p, f[0]);
    } else if constexpr (sizeof(E) == 2 && W == 8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = bf16_of_pair(pair(f[2 * i], f[2 * i + 1]));
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) put4(p + i, *reinterpret_cast<const float(*)[4]>(f + i));
    }
}

// Token by token: one thread per W channels, the state in registers.  The outputs overlap no
// input, so the loads of B tokens go out together, ahead of their stores (1 x 128 x 64, bf16: 10 us
// against 25 with one token's loads at a time).
template <typename E, bool kToken, int W, int B>
__global__ void glr_serial_kernel(GlrArgs a, const float* start) {
    const int per = (a.D + W - 1) / W;
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (size_t)a.N * per) return;
    const size_t n = i / per;
    const int d = (int)(i % per) * W;
    const size_t nd = n * a.D + d;
    float s[W];
#pragma unroll
    for (int v = 0; v < W; ++v) s[v] = 0.f;
    if (start) get_wide(start + nd, s);
    const E* x = static_cast<const E*>(a.x) + n * a.x_seq + d;
    const E* gc = static_cast<const E*>(a.g) + n * a.g_seq + d;
    const float* gt = static_cast<const float*>(a.g) + n * a.g_seq;
    E* h = static_cast<E*>(a.h) + n * a.T * a.D + d;
    for (int t0 = 0; t0 < a.T; t0 += B) {
        float xv[B][W], gv[B][kToken ? 1 : W];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const long long t = min(t0 + b, a.T - 1);
            get_wide(x + t * a.x_tok, xv[b]);
            if constexpr (kToken) gv[b][0] = gt[t * a.g_tok];
            else get_wide(gc + t * a.g_tok, gv[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            if (t0 + b >= a.T) break;
            const float rt = kToken ? retention<float>(gv[b][0]) : 0.f;
#pragma unroll
            for (int v = 0; v < W; ++v) s[v] = fmaf(kToken ? rt : retention<E>(gv[b][v]), s[v], xv[b][v]);
            put_wide(h + (size_t)(t0 + b) * a.D, s);
        }
    }
    put_wide(a.h_last + nd, s);
}

// The gradient likewise, from the last token on (gates per channel: a token gate's sum over the
// channels is the tiles' work).
template <typename E, int W, int B>
__global__ void glr_serial_back_kernel(GlrArgs a) {
    const int per = (a.D + W - 1) / W;
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (size_t)a.N * per) return;
    const size_t n = i / per;
    const int d = (int)(i % per) * W;
    const size_t nd = n * a.D + d, at = n * a.T * a.D + d;
    float c[W], first[W];
#pragma unroll
    for (int v = 0; v < W; ++v) c[v] = first[v] = 0.f;
    if (a.dh_last) get_wide(a.dh_last + nd, c);
    if (a.h0) get_wide(a.h0 + nd, first);
    const E* dh = static_cast<const E*>(a.x) + n * a.x_seq + d;
    const E* g = static_cast<const E*>(a.g) + n * a.g_seq + d;
    const E* h = static_cast<const E*>(a.h) + at;
    E *dx = static_cast<E*>(a.dx) + at, *dg = static_cast<E*>(a.dg) + at;
    for (int t0 = a.T - 1; t0 >= 0; t0 -= B) {
        float G[B][W], gv[B][W], before[B][W];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const long long t = max(t0 - b, 0);
            get_wide(dh + t * a.x_tok, G[b]);
            get_wide(g + t * a.g_tok, gv[b]);
            get_wide(h + max(t - 1, 0ll) * a.D, before[b]);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int t = t0 - b;
            if (t < 0) break;
#pragma unroll
            for (int v = 0; v < W; ++v) {
                G[b][v] += c[v];
                c[v] = retention<E>(gv[b][v]) * G[b][v];
                before[b][v] = c[v] * (t > 0 ? before[b][v] : first[v]);
            }
            put_wide(dx + (size_t)t * a.D, G[b]);
            put_wide(dg + (size_t)t * a.D, before[b]);
        }
    }
    if (a.dh0) put_wide(a.dh0 + nd, c);
}

// ------------------------------------------------------------------------- host

// Channels a thread of the token by token kernels takes: 16 bytes where that still makes a thread
// for every lane of the GPU's SMs, else four, or one where the rows do not allow it.
int thread_width(const GlrArgs& a) {
    const int es = a.bf16 ? 2 : 4;
    int width = access_width(a.x, a.N > 1 ? a.x_seq : 0, a.T > 1 ? a.x_tok : 0, es);
    if (!a.gate_token)
        width = min(width, access_width(a.g, a.N > 1 ? a.g_seq : 0, a.T > 1 ? a.g_tok : 0, es));
    if (es == 2 && width == 16 && a.D % 8 == 0 && (size_t)a.N * a.D >= 8ull * 152 * 1024) return 8;
    return width >= V * es && a.D % V == 0 ? V : 1;
}

// Token by token where a sequence is short, where it is short against the number of tiles that
// sequences make, and where the channels alone keep the SMs busy: nothing is joined or waited for
// then.  A token takes 0.08 us (0.14 in the gradient), a round of tiles 3.3.  In us, by tokens and
// by tiles, bf16, forward / gradient: 1 x 16 x 64 2.3 / 3.4 and 3.6 / 3.4, 1 x 32 x 64 3.6 / 5.3 and
// 3.8 / 3.4; 64 x 48 x 768 5.2 / 7.5 and 10.7 / 9.0, 64 x 96 x 768 8.6 / 13.5 and 10.8 / 9.5;
// 200 x 128 x 2048 49 / 82 and 67 / 80; 512 x 512 x 2048 gradient 827 and 889.
bool by_tokens(const GlrArgs& a, bool back) {
    if (back && a.gate_token) return false;
    const size_t strips = (size_t)a.N * ((a.D + kChans - 1) / kChans);
    return a.T <= 16 || (a.T <= 128 && strips >= 16 * (size_t)a.T) ||
           (size_t)a.N * a.D >= thread_width(a) * (152ull * 1024);
}

TilePlan make_plan(const GlrArgs& a, int backward, size_t* bytes) {
    TilePlan p{};
    const int es = a.bf16 ? 2 : 4;
    const int run = backward && !a.gate_token
                        ? (a.bf16 ? kRun<__nv_bfloat16, false, true> : kRun<float, false, true>)
                        : (a.bf16 ? kRun<__nv_bfloat16, true, true> : kRun<float, true, true>);
    // Strips of 64 channels (or D).  With few of them the blocks at work on one are many, and each
    // waits longer for the state before its tile, so they are halved, and their tiles twice as
    // long, down to rows of 64 bytes, until there are 128 of them (128 channels, bf16: 1 x 131072
    // tokens 155 us with one strip of 128 channels, 86 with two, 54 with four when they were
    // compared, 39 with four now; 64 x 32768 tokens
    // 245 us with two strips a row, 258 with four).  Down to rows of 32 bytes where all of a
    // sequence then is one tile and nobody waits (2 x 777 x 768: 6.3 us against 7.7).
    auto strips_at = [&](int log) { return (long long)a.N * ((a.D + (V << log) - 1) / (V << log)); };
    auto tokens_at = [&](int log) { return (kThreads >> log) * run; };
    while (p.cw_log < kMaxLog && (V << p.cw_log) < a.D) ++p.cw_log;
    while (p.cw_log > 0 && (V << p.cw_log) * es > 64 && a.T > tokens_at(p.cw_log) && strips_at(p.cw_log) < 128)
        --p.cw_log;
    if (p.cw_log > 0 && (V << p.cw_log) * es > 32 && a.T > tokens_at(p.cw_log) &&
        a.T <= tokens_at(p.cw_log - 1) && strips_at(p.cw_log - 1) <= 2 * 152)
        --p.cw_log;
    const int chans = V << p.cw_log;
    p.tokens = tokens_at(p.cw_log);
    p.ntiles = (a.T + p.tokens - 1) / p.tokens;
    if (p.ntiles < 1) p.ntiles = 1;
    p.ncols = (a.D + chans - 1) / chans;
    const size_t strips = (size_t)a.N * p.ncols;
    p.tiles = (unsigned)(strips * p.ntiles);
    size_t off = 0;
    char* w = static_cast<char*>(a.workspace);
    if (p.ntiles > 1) {
        const size_t words = strips * p.ntiles * chans;
        p.counter = reinterpret_cast<unsigned*>(w);
        p.maps = reinterpret_cast<unsigned long long*>(w + 256);
        p.ends = reinterpret_cast<unsigned*>(w + 256 + words * 8);
        p.hints = p.ends + words;
        p.words_bytes = 256 + words * 12 + strips * ((chans + 31) / 32) * p.ntiles * 4;
        off = (p.words_bytes + 255) / 256 * 256;
    }
    if (backward && a.gate_token && p.ncols > 1) {
        p.dg_part = reinterpret_cast<float*>(w + off);
        off += (size_t)p.ncols * a.N * a.T * sizeof(float);
    }
    *bytes = off;
    return p;
}

// Tensor maps where the strides allow it: 16-byte rows and strides below 2^40, the outer one the
// larger and a multiple of the inner one.  Of the tokens and the sequences those come first (`first`: the
// sequences do) that lie closer together.
template <typename E>
bool tile_map(CUtensorMap* m, const TilePlan& p, const GlrArgs& a, const void* ptr, long long seq,
              long long tok, int* first = nullptr) {
    const unsigned long long es = sizeof(E), D = a.D, T = a.T, N = a.N;
    unsigned long long ts = tok * es, ss = seq * es;
    if (a.T == 1) ts = a.N > 1 ? ss : (D * es + 15) / 16 * 16;   // any will do
    if (a.N == 1) ss = ts * T;
    const bool swap = ss < ts;
    const unsigned long long inner = swap ? ss : ts, outer = swap ? ts : ss;
    if (reinterpret_cast<uintptr_t>(ptr) % 16 || inner % 16 || outer % inner || outer >= 1ull << 40) return false;
    if (first) *first = swap;
    const unsigned tokens = (unsigned)min(p.tokens, 256);
    const TmaType type = sizeof(E) == 2 ? TmaType::bf16 : TmaType::f32;
    if (swap) return make_tma_map(m, type, ptr, {D, N, T}, {ss, ts}, {(unsigned)V << p.cw_log, 1u, tokens}, false);
    return make_tma_map(m, type, ptr, {D, T, N}, {ts, ss}, {(unsigned)V << p.cw_log, tokens, 1u}, false);
}

template <typename E, bool kToken, bool kBack>
cudaError_t tile_launch(const GlrArgs& a, TilePlan p, cudaStream_t s) {
    constexpr int tiles = 1 + (kToken ? 0 : 1) + (kBack ? 1 : 0) + (kBack && !kToken ? 2 : 1);
    const int smem = tiles * kTileBytes<E, kToken, kBack> + (int)sizeof(Joints) +
                     (kToken ? 2 * p.tokens * (int)sizeof(float) : 0);
    // The most any call needs, so that calls of two host threads set the same limit
    constexpr int most = tiles * kTileBytes<E, kToken, kBack> + (int)sizeof(Joints) +
                         (kToken ? 2 * kThreads * kRun<E, kToken, kBack> * (int)sizeof(float) : 0);
    auto kernel = glr_tile_kernel<E, kToken, kBack>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    if (p.ntiles > 1) {
        e = cudaMemsetAsync(a.workspace, kEmpty & 0xff, p.words_bytes, s);
        if (e != cudaSuccess) return e;
    }
    CUtensorMap mx{}, mg{}, mh{}, mo{}, mog{};
    p.tma = ((size_t)V << p.cw_log) * sizeof(E) >= 16 &&
            tile_map<E>(&mx, p, a, a.x, a.x_seq, a.x_tok, &p.x_first) &&
            (kToken || tile_map<E>(&mg, p, a, a.g, a.g_seq, a.g_tok, &p.g_first)) &&
            (!kBack || tile_map<E>(&mh, p, a, a.h, (long long)a.T * a.D, a.D));
    p.tma_out = ((size_t)V << p.cw_log) * sizeof(E) >= 16 &&
                tile_map<E>(&mo, p, a, kBack ? a.dx : a.h, (long long)a.T * a.D, a.D) &&
                (!kBack || kToken || tile_map<E>(&mog, p, a, a.dg, (long long)a.T * a.D, a.D));
    kernel<<<min(p.tiles, kResident<kToken, kBack> * 152u), kThreads, smem, s>>>(mx, mg, mh, mo, mog, a, p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t tiles(GlrArgs a, bool back, cudaStream_t s, int* launches) {
    size_t bytes;
    TilePlan p = make_plan(a, back, &bytes);
    const int es = sizeof(E);
    const int srow = (V << p.cw_log) * es;
    p.width_o = min(access_width(nullptr, 0, a.D, es), min(srow, 8));
    if (a.wait_cycles <= 0) a.wait_cycles = kWaitCycles;
    *launches = 1;
    cudaError_t e;
    if (back) e = a.gate_token ? tile_launch<E, true, true>(a, p, s) : tile_launch<E, false, true>(a, p, s);
    else e = a.gate_token ? tile_launch<E, true, false>(a, p, s) : tile_launch<E, false, false>(a, p, s);
    if (e != cudaSuccess || !p.dg_part) return e;
    const size_t n = (size_t)a.N * a.T;
    glr_gate_sum_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p.dg_part, p.ncols, n,
                                                                     static_cast<float*>(a.dg));
    *launches = 2;
    return cudaGetLastError();
}

template <typename E, int W, int B>
cudaError_t serial_launch(const GlrArgs& a, bool back, const float* start, cudaStream_t s) {
    const size_t threads = (size_t)a.N * (a.D / W);
    const unsigned blocks = (unsigned)((threads + 127) / 128);
    if (back) glr_serial_back_kernel<E, W, W == 1 || B == 1 ? B : B / 2><<<blocks, 128, 0, s>>>(a);
    else if (a.gate_token) glr_serial_kernel<E, true, W, B><<<blocks, 128, 0, s>>>(a, start);
    else glr_serial_kernel<E, false, W, B><<<blocks, 128, 0, s>>>(a, start);
    return cudaGetLastError();
}

// One or two tokens one by one: loads past the end cost more than they hide (1228 tokens of 3371
// channels, bf16: 39 us by eight, 20 by one).
template <typename E, int W>
cudaError_t serial_batches(const GlrArgs& a, bool back, const float* start, cudaStream_t s) {
    return a.T <= 2 ? serial_launch<E, W, 1>(a, back, start, s)
                    : serial_launch<E, W, W == 8 ? 4 : 8>(a, back, start, s);
}

template <typename E>
cudaError_t serial(const GlrArgs& a, bool back, const float* start, cudaStream_t s) {
    const int width = thread_width(a);
    if constexpr (sizeof(E) == 2)
        if (width == 8) return serial_batches<E, 8>(a, back, start, s);
    if (width == V) return serial_batches<E, V>(a, back, start, s);
    return serial_batches<E, 1>(a, back, start, s);
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, int backward) {
    size_t bytes = 0;
    if (!by_tokens(a, backward != 0)) make_plan(a, backward, &bytes);
    return bytes;
}

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    if (!by_tokens(a, false))
        return a.bf16 ? tiles<__nv_bfloat16>(a, false, s, launches) : tiles<float>(a, false, s, launches);
    *launches = 1;
    return a.bf16 ? serial<__nv_bfloat16>(a, false, a.h0, s) : serial<float>(a, false, a.h0, s);
}

cudaError_t glr_step_launch(const GlrArgs& a, cudaStream_t s) {
    return a.bf16 ? serial<__nv_bfloat16>(a, false, a.h_last, s) : serial<float>(a, false, a.h_last, s);
}

cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    if (a.T == 0) {   // nothing to go through: dh0 = dh_last
        const size_t bytes = (size_t)a.N * a.D * sizeof(float);
        *launches = 0;
        if (!a.dh0) return cudaSuccess;
        return a.dh_last ? cudaMemcpyAsync(a.dh0, a.dh_last, bytes, cudaMemcpyDeviceToDevice, s)
                         : cudaMemsetAsync(a.dh0, 0, bytes, s);
    }
    if (!by_tokens(a, true))
        return a.bf16 ? tiles<__nv_bfloat16>(a, true, s, launches) : tiles<float>(a, true, s, launches);
    *launches = 1;
    return a.bf16 ? serial<__nv_bfloat16>(a, true, nullptr, s) : serial<float>(a, true, nullptr, s);
}

}  // namespace ttm
