// kda_wait.cuh - waits and barriers of kernels whose warps do different work.
#pragma once

#include "kda_ptx.cuh"

namespace kda {

// mbar_wait_bounded by a whole warp: true in every lane or in none, so that the warp goes on as one (the limit may
// run out in one lane just before the phase completes for another).
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, uint32_t limit)
{
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, parity, limit));
    __syncwarp();
    return ok;
}

// Arrive at a named barrier (named_bar_sync) without waiting for it; what this thread wrote before is seen by those
// who wait.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t count)
{
    __threadfence_block();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

}  // namespace kda
