// Included ahead of a kernel file of the library whose wait limit is then wl_limit(): the waits of chosen warps
// and lanes give up without a poll, all others after 2^14 polls, so that every path behind a wait that ran out
// can be taken on purpose and ends by itself.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

static __device__ uint32_t wl_warps, wl_lanes;

static __device__ __forceinline__ uint32_t wl_limit()
{
    return (wl_warps >> (threadIdx.x >> 5) & 1) && (wl_lanes >> (threadIdx.x & 31) & 1) ? 0u : 1u << 14;
}

extern "C" int wl_set(uint32_t warps, uint32_t lanes)
{
    const cudaError_t e = cudaMemcpyToSymbol(wl_warps, &warps, sizeof(warps));
    return (int)(e != cudaSuccess ? e : cudaMemcpyToSymbol(wl_lanes, &lanes, sizeof(lanes)));
}
