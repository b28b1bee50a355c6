// What the kernels on clusters and pairs of blocks share (the operators around the scan): bounded waits,
// cluster and pair instructions, launches that overlap.  Device code only but for the launch; sm_103a.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/ttm.h"
#include "tc_ptx.cuh"

namespace ttm {
namespace tc {

// Bounded wait.  A wait that runs out sets the block's abort flag (every role then
// stops) and the device status word.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* abort, int* status,
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

// The kernels of a call are launched so that one may start while the blocks of the one before
// finish: its set-up runs beside them, and it waits here before it reads what they wrote.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------- two blocks on one tile (PTX)

__device__ __forceinline__ void mbar_arrive_at(uint32_t addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// The same without the wait for this thread's own stores: for hand-offs that pass no memory on.
__device__ __forceinline__ void mbar_arrive_relaxed_at(uint32_t addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
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
// Arrives on `bar` in the blocks of `mask` (both of a cluster of two) once the products issued so far are complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask = 3) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)), "h"(mask)
        : "memory");
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

}  // namespace tc
}  // namespace ttm
