// kda_launch.cuh - programmatic dependent launch: a kernel is set up while the one before it in the stream
// is still running, and waits for it on the device.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace kda {

// In the first kernel: the next one, if it was launched by launch_after, may start.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// In the second: wait until the first has finished and its writes are visible.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launch a kernel that calls wait_for_previous() before it touches what the kernel before it in the stream
// writes. That kernel must be an ordinary launch of this library: the second kernel may read what is older.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A &&...args)
{
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

}  // namespace kda
