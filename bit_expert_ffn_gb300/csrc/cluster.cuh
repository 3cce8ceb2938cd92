// cluster.cuh -- thread-block clusters: rank, barrier and loads from the shared
// memory of another CTA.
#pragma once

#include <stdint.h>

namespace moe {

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Every thread of the cluster (stores before it are seen after it).
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}

// The 32-bit word at the same shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank)
{
    uint32_t v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.u32 %0, [a];\n\t}"
                 : "=r"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}

}  // namespace moe
