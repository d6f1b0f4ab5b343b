// kda_cluster.cuh - clusters: blocks that run at once and reach one another's shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <utility>

namespace kda {

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute *at, unsigned grid, int nc, int threads, size_t smem, cudaStream_t stream)
{
    at->id = cudaLaunchAttributeClusterDimension;
    at->val.clusterDim.x = (unsigned)nc;
    at->val.clusterDim.y = at->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = nc > 1 ? 1 : 0;
    return cfg;
}

// A launch of clusters of nc blocks (nc 1: without).
template <typename... P, typename... A>
inline cudaError_t launch_cluster(void (*kernel)(P...), unsigned grid, int nc, int threads, size_t smem, cudaStream_t stream, A &&...args)
{
    cudaLaunchAttribute at = {};
    const cudaLaunchConfig_t cfg = cluster_config(&at, grid, nc, threads, smem, stream);
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace kda
