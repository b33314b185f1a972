// What the kernels that run as clusters of blocks share: a block's place in its
// cluster, barriers over it, and stores to the other blocks' shared memory.
//
// The barriers are of the `.aligned` form, which takes for granted that a warp's
// lanes are there together.  They come behind branches and loops that lanes leave
// at different times, so each brings its warp together first.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {
namespace cluster {

__device__ __forceinline__ uint32_t rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void sync() {
    arrive();
    wait();
}
// Stores to the same shared variable of block `to` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t to) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(to));
    return a;
}
__device__ __forceinline__ void store(float2* p, uint32_t to, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(remote(p, to)), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void store(float4* p, uint32_t to, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(remote(p, to)), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

}  // namespace cluster
}  // namespace gdn
