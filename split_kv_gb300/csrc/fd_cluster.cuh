// fd_cluster.cuh -- sums over a CTA and steps of a cluster, shared by the
// kernels that keep page tables.
#pragma once

#include <stdint.h>

#include "fd_device.cuh"

namespace fdk {

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

// Inclusive prefix sum over the CTA of one value per thread; `total` gets the
// sum.  warp_sums: 32 values of shared memory, free again after the call's
// last barrier.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        const long long s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    __syncthreads();
    total = all;
    return x + before;
}

// Address of this CTA's shared-memory place `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote_smem(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t remote_load(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void remote_store(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

}  // namespace fdk
