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
// Tile: 256 threads, each 16 bytes of channels (8 bf16 or 4 fp32 values) times R
// consecutive tokens, CW threads side by side over the channels and 256 / CW over
// the tokens.  CW is the smallest power of two that covers D, at most 16: rows of
// 256 bytes keep DRAM pages busy, and a narrower strip gives more, longer tiles
// to a row.  The map of a tile is joined by shuffles inside a warp and through
// shared memory between the eight warps.
//
// Between tiles (look-back): a block publishes its tile's map as soon as it has it,
// then its last warp reads the maps of the tiles before it, 32 flags at a time, back
// to the nearest one whose end state is known, and publishes its own end state.
// Tiles are handed out in order by a counter, so a block only ever waits for blocks
// that are already running.  The waits are bounded: one that runs out sets the
// device status word and the call's outputs are invalid.
#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/ttm.h"
#include "train_ops.h"

namespace ttm {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 8;                       // tokens of one thread in a tile
constexpr int kTileBytes = kThreads * kRun * 16;
constexpr unsigned kMapReady = 1, kEndReady = 2;
constexpr long long kWaitCycles = 4000000000LL;   // default limit, ~2 s at 2 GHz

template <typename E> struct Vec;
template <> struct Vec<float> { static constexpr int n = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int n = 8; };

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float& o, float v) { o = v; }
__device__ __forceinline__ void put(__nv_bfloat16& o, float v) { o = __float2bfloat16(v); }

// 16 bytes of channels as fp32 values and back.
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4], float) {
    f[0] = __uint_as_float(u.x); f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z); f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8], __nv_bfloat16) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4], float) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8], __nv_bfloat16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// exp through the base-2 unit (2 units in the last place); -infinity gives 0.
__device__ __forceinline__ float retention(float g) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(g * 1.44269504088896341f));
    return r;
}

// A c + H for the map (A, H).  A state of exactly zero stays out of the product: a
// growing gate may have taken A to infinity, which must not turn it into NaN.
__device__ __forceinline__ float apply(float A, float H, float c) {
    return c == 0.f ? H : fmaf(A, c, H);
}

// ------------------------------------------------------------ global <-> shared

// Widest access all rows of a view allow, in bytes.
inline int access_width(const void* p, long long seq, long long tok, int es) {
    const unsigned long long m =
        reinterpret_cast<uintptr_t>(p) | (unsigned long long)seq * es | (unsigned long long)tok * es;
    return m % 16 == 0 ? 16 : (m % 4 == 0 ? 4 : es);
}

// Copies rows [0, rows) of `bytes` bytes at `pitch` bytes from global memory into
// shared rows of `srow` bytes, width bytes at a time; rows below `lo` or from `hi` on
// and bytes past the end read as zero (`any`: an address of the tensor that copies of
// no bytes name).  Asynchronous except for 2-byte accesses.
__device__ __forceinline__ void load_rows(unsigned char* dst, int rows, int srow, const char* src,
                                          long long pitch, int lo, int hi, int bytes, int width,
                                          const void* any) {
    const int shift = width == 16 ? 4 : (width == 4 ? 2 : 1);
    const int per = srow >> shift;                    // accesses per row, a power of two
    const int log_per = 31 - __clz(per);
    const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
    for (int i = threadIdx.x; i < rows << log_per; i += kThreads) {
        const int r = i >> log_per, o = (i & (per - 1)) << shift;
        const int n = r >= lo && r < hi ? max(0, min(width, bytes - o)) : 0;
        const char* p = n ? src + r * pitch + o : static_cast<const char*>(any);
        if (width == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + r * srow + o),
                         "l"(p), "r"(n) : "memory");
        else if (width == 4)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(base + r * srow + o),
                         "l"(p), "r"(n) : "memory");
        else
            *reinterpret_cast<unsigned short*>(dst + r * srow + o) =
                n ? *reinterpret_cast<const unsigned short*>(p) : (unsigned short)0;
    }
}

__device__ __forceinline__ void load_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Shared rows back to global memory where a row does not start on 16 bytes:
// neighbouring threads write neighbouring values.
__device__ __forceinline__ void store_rows(char* dst, long long pitch, const unsigned char* src,
                                           int rows, int srow, int bytes, int width) {
    const int shift = width == 4 ? 2 : 1;
    const int per = srow >> shift, log_per = 31 - __clz(per);
    for (int i = threadIdx.x; i < rows << log_per; i += kThreads) {
        const int r = i >> log_per, o = (i & (per - 1)) << shift;
        if (o >= bytes) continue;
        if (width == 4)
            *reinterpret_cast<uint32_t*>(dst + r * pitch + o) =
                *reinterpret_cast<const uint32_t*>(src + r * srow + o);
        else
            *reinterpret_cast<unsigned short*>(dst + r * pitch + o) =
                *reinterpret_cast<const unsigned short*>(src + r * srow + o);
    }
}

// ------------------------------------------------------------------- look-back

struct TilePlan {
    int cw_log;            // log2 of the threads side by side over the channels
    int tokens;            // of a tile
    int ntiles, ncols;     // tiles of a sequence, strips of channels
    unsigned* counter;     // hands out tiles in order; NULL when ntiles == 1
    unsigned* flags;       // [strip][tile] in processing order
    float* maps;           // [strip][tile][A | H | end][channels of a strip]
    int width_x, width_g, width_o;   // access widths of x / dh, g, and the contiguous tensors
    float* dg_part;        // token gate over several strips: [ncols][N T] partial sums
};

__device__ __forceinline__ unsigned load_flag(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void store_flag(unsigned* p, unsigned v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// One warp: the state before processing tile j of a strip.  Lane l holds channels
// 4l .. 4l+3 (chans <= 128).  `first` is the state before tile 0.
__device__ __forceinline__ float4 look_back(const unsigned* flags, const float* maps, int chans,
                                            int j, float4 first, int* status, long long limit) {
    const int lane = threadIdx.x & 31;
    const bool mine = 4 * lane < chans;
    float4 A = make_float4(1.f, 1.f, 1.f, 1.f), H = make_float4(0.f, 0.f, 0.f, 0.f);
    const long long t0 = clock64();
    int next = j - 1;                       // nearest tile not joined yet
    while (true) {
        // flags of tiles next, next - 1, ..: wait until those down to an end state are set
        const int at = next - lane;
        unsigned have, ends;
        while (true) {
            const unsigned f = at >= 0 ? load_flag(flags + at) : kMapReady;
            have = __ballot_sync(0xffffffffu, f != 0);
            ends = __ballot_sync(0xffffffffu, at >= 0 && f == kEndReady);
            const unsigned upto = ends ? (ends & (0u - ends)) : 0u;    // lowest end state
            const unsigned need = ends ? (upto | (upto - 1u)) : 0xffffffffu;
            if ((have & need) == need) break;
            if (__any_sync(0xffffffffu, clock64() - t0 > limit)) {
                if (lane == 0) atomicExch(status, TTM_ERR_TIMEOUT);
                return first;
            }
        }
        __syncwarp();       // the flags' lanes have acquired; now all lanes may read
        const int stop = ends ? __ffs(ends) - 1 : 32;     // maps of tiles next .. next - stop + 1
        const int n = min(stop, next + 1);
        const float* m = maps + (size_t)next * 3 * chans + 4 * lane;
        for (int i = 0; i < n; i += 4) {
            float4 a[4], h[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (mine && i + u < n) {
                    const float* p = m - (size_t)(i + u) * 3 * chans;
                    a[u] = __ldcg(reinterpret_cast<const float4*>(p));
                    h[u] = __ldcg(reinterpret_cast<const float4*>(p + chans));
                } else {
                    a[u] = make_float4(1.f, 1.f, 1.f, 1.f);
                    h[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                H.x = apply(A.x, H.x, h[u].x); H.y = apply(A.y, H.y, h[u].y);
                H.z = apply(A.z, H.z, h[u].z); H.w = apply(A.w, H.w, h[u].w);
                A.x *= a[u].x; A.y *= a[u].y; A.z *= a[u].z; A.w *= a[u].w;
            }
        }
        if (ends) {
            if (mine)
                first = __ldcg(reinterpret_cast<const float4*>(m - (size_t)stop * 3 * chans +
                                                               2 * chans));
            break;
        }
        next -= n;
        if (next < 0) break;
    }
    return make_float4(apply(A.x, H.x, first.x), apply(A.y, H.y, first.y),
                       apply(A.z, H.z, first.z), apply(A.w, H.w, first.w));
}

// Shared memory behind the input tiles.
struct Joints {
    float a[kWarps][128], h[kWarps][128];   // map of each warp's tokens, by channel of the strip
    float carry[128];                       // state before the tile
    unsigned ticket;
};

// ------------------------------------------------------------------ tile kernel

template <typename E, bool kToken, bool kBack>
__global__ void __launch_bounds__(kThreads) glr_tile_kernel(GlrArgs a, TilePlan p) {
    constexpr int V = Vec<E>::n;
    extern __shared__ __align__(16) unsigned char smem[];
    constexpr int kTiles = 1 + (kToken ? 0 : 1) + (kBack ? 1 : 0);
    unsigned char* sx = smem;                                   // x or dh
    unsigned char* sg = smem + (kToken ? 0 : kTileBytes);       // g (gate per channel)
    unsigned char* sh = smem + (kTiles - 1) * kTileBytes;       // gradient: h one token earlier
    Joints& J = *reinterpret_cast<Joints*>(smem + kTiles * kTileBytes);

    const int tid = threadIdx.x, warp = tid >> 5;
    // Which tile: in order of the counter, all strips of tile 0 first
    unsigned ticket = blockIdx.x;
    if (p.counter) {
        if (tid == 0) J.ticket = atomicAdd(p.counter, 1u);
        __syncthreads();
        ticket = J.ticket;
    }
    const unsigned strips = (unsigned)a.N * p.ncols;
    const int j = ticket / strips;                    // place in processing order
    const unsigned strip = ticket % strips;
    const size_t n = strip / p.ncols;
    const int chans = V << p.cw_log, c0 = (strip % p.ncols) * chans;
    const int tile = kBack ? p.ntiles - 1 - j : j;
    const int t0 = tile * p.tokens;
    const int ntok = min(p.tokens, a.T - t0);
    const int srow = 16 << p.cw_log;                  // bytes of a shared row
    const int bytes = min(chans, a.D - c0) * (int)sizeof(E);

    load_rows(sx, p.tokens, srow,
              reinterpret_cast<const char*>(static_cast<const E*>(a.x) + n * a.x_seq +
                                            (long long)t0 * a.x_tok + c0),
              a.x_tok * (long long)sizeof(E), 0, ntok, bytes, p.width_x, a.x);
    if (!kToken)
        load_rows(sg, p.tokens, srow,
                  reinterpret_cast<const char*>(static_cast<const E*>(a.g) + n * a.g_seq +
                                                (long long)t0 * a.g_tok + c0),
                  a.g_tok * (long long)sizeof(E), 0, ntok, bytes, p.width_g, a.g);
    const size_t row0 = n * a.T + t0;                 // row of the contiguous tensors
    if (kBack)   // row r holds h of token t0 + r - 1; token -1 is h0, taken below
        load_rows(sh, p.tokens, srow,
                  reinterpret_cast<const char*>(static_cast<const E*>(a.h) + c0) +
                      ((long long)row0 - 1) * a.D * (long long)sizeof(E),
                  (long long)a.D * sizeof(E), t0 == 0 ? 1 : 0, ntok, bytes, p.width_o, a.h);

    // This thread's channels and run of tokens, in processing order
    const int cw = 1 << p.cw_log, ch = (tid & (cw - 1)) * V;
    const int place = tid >> p.cw_log, runs = kThreads >> p.cw_log;
    const int r0 = (kBack ? runs - 1 - place : place) * kRun;
    const bool live = c0 + ch < a.D;
    float tg[kRun];                                   // retentions of a token gate
    if (kToken) {
        const float* g = static_cast<const float*>(a.g) + n * a.g_seq + (long long)t0 * a.g_tok;
#pragma unroll
        for (int i = 0; i < kRun; ++i)
            tg[i] = r0 + i < ntok ? retention(g[(long long)(r0 + i) * a.g_tok]) : 1.f;
    }
    const float* init = kBack ? a.dh_last : a.h0;
    load_wait();
    __syncthreads();

    const int so = r0 * srow + (tid & (cw - 1)) * 16;
    float A[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) { A[v] = 1.f; H[v] = 0.f; }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int q = kBack ? kRun - 1 - i : i;
        float x[V], g[V];
        unpack(*reinterpret_cast<const uint4*>(sx + so + q * srow), x, E());
        if (!kToken) unpack(*reinterpret_cast<const uint4*>(sg + so + q * srow), g, E());
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float r = kToken ? tg[q] : retention(g[v]);
            H[v] = kBack ? r * (H[v] + x[v]) : fmaf(r, H[v], x[v]);
            A[v] *= r;
        }
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
#pragma unroll
        for (int v = 0; v < V; v += 4) {
            *reinterpret_cast<float4*>(&J.a[warp][ch + v]) = make_float4(A[v], A[v + 1], A[v + 2], A[v + 3]);
            *reinterpret_cast<float4*>(&J.h[warp][ch + v]) = make_float4(H[v], H[v + 1], H[v + 2], H[v + 3]);
        }
    }
    // exclusive of this thread's own run
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = __shfl_up_sync(0xffffffffu, A[v], cw);
        H[v] = __shfl_up_sync(0xffffffffu, H[v], cw);
        if ((tid & 31) < cw) { A[v] = 1.f; H[v] = 0.f; }
    }
    __syncthreads();

    // The last warp takes the tile's map and the state before the tile
    if (warp == kWarps - 1) {
        const int lane = tid & 31, c = 4 * lane;
        float4 first = make_float4(0.f, 0.f, 0.f, 0.f), mA = make_float4(1.f, 1.f, 1.f, 1.f),
               mH = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < chans) {
            const size_t nd = n * a.D + c0 + c;
            const int left = a.D - c0 - c;
            if (j == 0 && init) {
                if (left > 0) first.x = init[nd];
                if (left > 1) first.y = init[nd + 1];
                if (left > 2) first.z = init[nd + 2];
                if (left > 3) first.w = init[nd + 3];
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 wa = *reinterpret_cast<const float4*>(&J.a[w][c]);
                const float4 wh = *reinterpret_cast<const float4*>(&J.h[w][c]);
                mH.x = apply(wa.x, wh.x, mH.x); mH.y = apply(wa.y, wh.y, mH.y);
                mH.z = apply(wa.z, wh.z, mH.z); mH.w = apply(wa.w, wh.w, mH.w);
                mA.x *= wa.x; mA.y *= wa.y; mA.z *= wa.z; mA.w *= wa.w;
            }
        }
        float4 before = first;
        if (p.counter) {
            unsigned* flags = p.flags + (size_t)strip * p.ntiles;
            float* maps = p.maps + (size_t)strip * p.ntiles * 3 * chans;
            float* own = maps + (size_t)j * 3 * chans + c;
            if (j > 0) {
                if (c < chans) {
                    __stcg(reinterpret_cast<float4*>(own), mA);
                    __stcg(reinterpret_cast<float4*>(own + chans), mH);
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) store_flag(flags + j, kMapReady);
                before = look_back(flags, maps, chans, j, first, a.status, a.wait_cycles);
            }
            if (j + 1 < p.ntiles) {
                if (c < chans)
                    __stcg(reinterpret_cast<float4*>(own + 2 * chans),
                           make_float4(apply(mA.x, mH.x, before.x), apply(mA.y, mH.y, before.y),
                                       apply(mA.z, mH.z, before.z), apply(mA.w, mH.w, before.w)));
                __threadfence();
                __syncwarp();
                if (lane == 0) store_flag(flags + j, kEndReady);
            }
        }
        if (c < chans) *reinterpret_cast<float4*>(&J.carry[c]) = before;
    }
    __syncthreads();

    // State before this thread's run: the tile's, through the warps before, then the
    // runs before in this warp
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = J.carry[ch + v];
    for (int w = 0; w < warp; ++w) {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = apply(J.a[w][ch + v], J.h[w][ch + v], s[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = apply(A[v], H[v], s[v]);

    const bool direct = p.width_o == 16;
    E* out = static_cast<E*>(kBack ? a.dx : a.h) + row0 * a.D + c0 + ch;
    E* outg = kBack && !kToken ? static_cast<E*>(a.dg) + row0 * a.D + c0 + ch : nullptr;
    float sum[kRun];                                  // token gate: this thread's share of dg
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int q = kBack ? kRun - 1 - i : i, r = r0 + q;
        float x[V], g[V], o[V];
        unpack(*reinterpret_cast<const uint4*>(sx + so + q * srow), x, E());
        if (!kToken) unpack(*reinterpret_cast<const uint4*>(sg + so + q * srow), g, E());
        if (!kBack) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = fmaf(kToken ? tg[q] : retention(g[v]), s[v], x[v]);
                o[v] = s[v];
            }
        } else {
            float b[V];
            unpack(*reinterpret_cast<const uint4*>(sh + so + q * srow), b, E());
            if (t0 + r == 0 && a.h0 && live) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    b[v] = c0 + ch + v < a.D ? a.h0[n * a.D + c0 + ch + v] : 0.f;
            }
            float acc = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                o[v] = x[v] + s[v];
                s[v] = (kToken ? tg[q] : retention(g[v])) * o[v];
                b[v] *= s[v];
                if (kToken) acc += b[v];
            }
            if (kToken) {
                sum[q] = acc;
            } else {
                const uint4 u = pack(b, E());
                if (!direct) *reinterpret_cast<uint4*>(sh + so + q * srow) = u;
                else if (live && r < ntok) *reinterpret_cast<uint4*>(outg + (size_t)r * a.D) = u;
            }
        }
        const uint4 u = pack(o, E());
        if (!direct) *reinterpret_cast<uint4*>(sx + so + q * srow) = u;
        else if (live && r < ntok) *reinterpret_cast<uint4*>(out + (size_t)r * a.D) = u;
    }

    // End of the strip: the tokens past T leave the state as it is
    float* end = kBack ? a.dh0 : a.h_last;
    if (j == p.ntiles - 1 && place == runs - 1 && end) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c0 + ch + v < a.D) end[n * a.D + c0 + ch + v] = s[v];
    }
    if (kBack && kToken) {
        // over the cw threads of the strip's channels; they are lanes of one warp
#pragma unroll
        for (int q = 0; q < kRun; ++q)
            for (int d = cw >> 1; d; d >>= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], d);
        float* dg = p.ncols > 1 ? p.dg_part + (size_t)(strip % p.ncols) * a.N * a.T
                                : static_cast<float*>(a.dg);
#pragma unroll
        for (int q = 0; q < kRun; ++q)
            if ((tid & (cw - 1)) == (q & (cw - 1)) && r0 + q < ntok) dg[row0 + r0 + q] = sum[q];
    }
    if (!direct) {
        __syncthreads();
        char* o = reinterpret_cast<char*>(static_cast<E*>(kBack ? a.dx : a.h) + row0 * a.D + c0);
        store_rows(o, (long long)a.D * sizeof(E), sx, ntok, srow, bytes, p.width_o);
        if (kBack && !kToken) {
            o = reinterpret_cast<char*>(static_cast<E*>(a.dg) + row0 * a.D + c0);
            store_rows(o, (long long)a.D * sizeof(E), sh, ntok, srow, bytes, p.width_o);
        }
    }
}

// dg of a token gate from the strips' partial sums, in the strips' order.
__global__ void glr_gate_sum_kernel(const float* part, int ncols, size_t n, float* dg) {
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int c = 0; c < ncols; ++c) s += part[c * n + i];
    dg[i] = s;
}

// Token by token for calls of few tokens: one thread per 16 bytes of channels (W = 1:
// per channel, where rows do not start on 16 bytes).  The state stays in registers.
template <typename E, bool kToken, int W>
__global__ void glr_serial_kernel(GlrArgs a, const float* start) {
    const int per = (a.D + W - 1) / W;
    const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= (size_t)a.N * per) return;
    const size_t n = i / per;
    const int d = (int)(i % per) * W;
    const size_t nd = n * a.D + d;
    float s[W];
#pragma unroll
    for (int v = 0; v < W; ++v) s[v] = start ? start[nd + v] : 0.f;
    const E* x = static_cast<const E*>(a.x) + n * a.x_seq + d;
    const E* gc = static_cast<const E*>(a.g) + n * a.g_seq + d;
    const float* gt = static_cast<const float*>(a.g) + n * a.g_seq;
    E* h = static_cast<E*>(a.h) + n * a.T * a.D + d;
#pragma unroll 2
    for (int t = 0; t < a.T; ++t) {
        float xv[W], gv[W];
        if constexpr (W == 1) {
            xv[0] = to_f(x[(long long)t * a.x_tok]);
            if (!kToken) gv[0] = to_f(gc[(long long)t * a.g_tok]);
        } else {
            unpack(*reinterpret_cast<const uint4*>(x + (long long)t * a.x_tok), xv, E());
            if (!kToken) unpack(*reinterpret_cast<const uint4*>(gc + (long long)t * a.g_tok), gv, E());
        }
        const float rt = kToken ? retention(gt[(long long)t * a.g_tok]) : 0.f;
#pragma unroll
        for (int v = 0; v < W; ++v) s[v] = fmaf(kToken ? rt : retention(gv[v]), s[v], xv[v]);
        if constexpr (W == 1) put(h[(size_t)t * a.D], s[0]);
        else *reinterpret_cast<uint4*>(h + (size_t)t * a.D) = pack(s, E());
    }
#pragma unroll
    for (int v = 0; v < W; ++v) a.h_last[nd + v] = s[v];
}

// ------------------------------------------------------------------------- host

// A call of at most this many tokens runs token by token: a tile would be mostly empty.
constexpr int kSerialTokens = 8;

TilePlan make_plan(const GlrArgs& a, int backward, size_t* bytes) {
    TilePlan p{};
    const int es = a.bf16 ? 2 : 4, V = 16 / es;
    while (p.cw_log < 4 && (V << p.cw_log) < a.D) ++p.cw_log;
    const int chans = V << p.cw_log;
    p.tokens = (kThreads >> p.cw_log) * kRun;
    p.ntiles = (a.T + p.tokens - 1) / p.tokens;
    if (p.ntiles < 1) p.ntiles = 1;
    p.ncols = (a.D + chans - 1) / chans;
    const size_t strips = (size_t)a.N * p.ncols;
    size_t off = 0;
    char* w = static_cast<char*>(a.workspace);
    if (p.ntiles > 1) {
        p.counter = reinterpret_cast<unsigned*>(w);
        p.flags = reinterpret_cast<unsigned*>(w + 256);
        off = 256 + (strips * p.ntiles * 4 + 255) / 256 * 256;
        p.maps = reinterpret_cast<float*>(w + off);
        off += strips * p.ntiles * 3 * chans * sizeof(float);
    }
    if (backward && a.gate_token && p.ncols > 1) {
        p.dg_part = reinterpret_cast<float*>(w + off);
        off += (size_t)p.ncols * a.N * a.T * sizeof(float);
    }
    *bytes = off;
    return p;
}

template <typename E, bool kToken, bool kBack>
cudaError_t tile_launch(const GlrArgs& a, const TilePlan& p, cudaStream_t s) {
    constexpr int tiles = 1 + (kToken ? 0 : 1) + (kBack ? 1 : 0);
    constexpr int smem = tiles * kTileBytes + (int)sizeof(Joints);
    auto kernel = glr_tile_kernel<E, kToken, kBack>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (p.ntiles > 1) {
        e = cudaMemsetAsync(a.workspace, 0, 256 + (size_t)a.N * p.ncols * p.ntiles * 4, s);
        if (e != cudaSuccess) return e;
    }
    kernel<<<(unsigned)((size_t)a.N * p.ncols * p.ntiles), kThreads, smem, s>>>(a, p);
    return cudaGetLastError();
}

template <typename E>
cudaError_t tiles(GlrArgs a, bool back, cudaStream_t s, int* launches) {
    size_t bytes;
    TilePlan p = make_plan(a, back, &bytes);
    const int es = sizeof(E);
    p.width_x = access_width(a.x, a.N > 1 ? a.x_seq : 0, a.T > 1 ? a.x_tok : 0, es);
    p.width_g = a.gate_token ? 4 : access_width(a.g, a.N > 1 ? a.g_seq : 0, a.T > 1 ? a.g_tok : 0, es);
    p.width_o = access_width(nullptr, 0, a.D, es);
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

template <typename E>
cudaError_t serial(const GlrArgs& a, const float* start, cudaStream_t s) {
    constexpr int V = Vec<E>::n;
    const int es = sizeof(E);
    bool wide = access_width(a.x, a.N > 1 ? a.x_seq : 0, a.T > 1 ? a.x_tok : 0, es) == 16 &&
                access_width(nullptr, 0, a.D, es) == 16;
    if (!a.gate_token)
        wide = wide && access_width(a.g, a.N > 1 ? a.g_seq : 0, a.T > 1 ? a.g_tok : 0, es) == 16;
    const size_t threads = (size_t)a.N * (wide ? a.D / V : a.D);
    const unsigned blocks = (unsigned)((threads + 127) / 128);
    if (wide && a.gate_token) glr_serial_kernel<E, true, V><<<blocks, 128, 0, s>>>(a, start);
    else if (wide) glr_serial_kernel<E, false, V><<<blocks, 128, 0, s>>>(a, start);
    else if (a.gate_token) glr_serial_kernel<E, true, 1><<<blocks, 128, 0, s>>>(a, start);
    else glr_serial_kernel<E, false, 1><<<blocks, 128, 0, s>>>(a, start);
    return cudaGetLastError();
}

}  // namespace

size_t glr_workspace_bytes(const GlrArgs& a, int backward) {
    size_t bytes = 0;
    if (backward || a.T > kSerialTokens) make_plan(a, backward, &bytes);
    return bytes;
}

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    if (a.T > kSerialTokens)
        return a.bf16 ? tiles<__nv_bfloat16>(a, false, s, launches) : tiles<float>(a, false, s, launches);
    *launches = 1;
    return a.bf16 ? serial<__nv_bfloat16>(a, a.h0, s) : serial<float>(a, a.h0, s);
}

cudaError_t glr_step_launch(const GlrArgs& a, cudaStream_t s) {
    return a.bf16 ? serial<__nv_bfloat16>(a, a.h_last, s) : serial<float>(a, a.h_last, s);
}

cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t s, int* launches) {
    if (a.T == 0) {   // nothing to go through: dh0 = dh_last
        const size_t bytes = (size_t)a.N * a.D * sizeof(float);
        *launches = 0;
        if (!a.dh0) return cudaSuccess;
        return a.dh_last ? cudaMemcpyAsync(a.dh0, a.dh_last, bytes, cudaMemcpyDeviceToDevice, s)
                         : cudaMemsetAsync(a.dh0, 0, bytes, s);
    }
    return a.bf16 ? tiles<__nv_bfloat16>(a, true, s, launches) : tiles<float>(a, true, s, launches);
}

}  // namespace ttm
