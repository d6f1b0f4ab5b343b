// kda_wait.cuh - a wait for kernels whose warps do different work.
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

}  // namespace kda
