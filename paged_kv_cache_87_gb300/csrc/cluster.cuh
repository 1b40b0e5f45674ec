// cluster.cuh -- thread-block clusters: their barrier, and loads of another CTA's shared memory.
#pragma once

#include "common.cuh"

namespace pkv {

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Two or four floats of this CTA's shared memory, in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t place_in(const float* mine, int rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(mine)), "r"(rank));
    return at;
}
__device__ __forceinline__ void load_from(const float* mine, int rank, float& a, float& b) {
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(a), "=f"(b) : "r"(place_in(mine, rank)) : "memory");
}
__device__ __forceinline__ void load_from(const float* mine, int rank, float (&v)[2]) {
    load_from(mine, rank, v[0], v[1]);
}
__device__ __forceinline__ void load_from(const float* mine, int rank, float (&v)[4]) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(place_in(mine, rank)) : "memory");
}

}  // namespace pkv
