// kda_launch.cuh - host side of a launch: what is asked of a device once, and programmatic dependent launch
// (a kernel is set up while the one before it in the stream is still running, and waits for it on the device).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

namespace kda {

// The current device and its SM count (asked once per device).
inline cudaError_t current_sms(int *dev, int *sms)
{
    static std::atomic<int> known[64];
    cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess) return e;
    const bool slot = *dev >= 0 && *dev < 64;
    if (slot && (*sms = known[*dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
    if (e == cudaSuccess && slot) known[*dev].store(*sms, std::memory_order_relaxed);
    return e;
}

// Raise a kernel's dynamic shared-memory limit, once per device: `done` is a bit per device, static at the call.
template <typename Fn>
inline cudaError_t raise_smem_on(std::atomic<uint64_t> &done, int dev, Fn *kernel, int bytes)
{
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

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
