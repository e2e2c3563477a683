// Helpers of kernels whose thread-block clusters divide one item's tokens and
// merge their results through distributed shared memory.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace dec {

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(v.x), "f"(v.y)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void store2(T *dst, float2 v);
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16 *dst, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(v.x, v.y);
}
template <>
__device__ __forceinline__ void store2<float>(float *dst, float2 v) {
    *reinterpret_cast<float2 *>(dst) = v;
}

// weight of a partial with maximum m under the common maximum M (0 for an
// empty one; also when every partial is empty)
__device__ __forceinline__ float weight(float m, float M) {
    return m == -INFINITY ? 0.f : exp2f(m - M);
}

}  // namespace dec
}  // namespace pa
