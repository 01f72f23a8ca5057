// lisa_launch.cuh -- launches as a programmatic dependent of the kernel before
// it on the stream: the kernel's set-up overlaps that one's tail.  Every kernel
// launched this way calls chain_begin() before it touches memory that another
// kernel may have written (or may still read), so a chain of them orders like
// plain launches.  It pays for the forward (a 56 x 56 pooled call 2 us), not between
// the backward's persistent kernels (14 of 121 us lost): those launch plainly.
#pragma once

#include <mutex>

#include <cuda_runtime.h>

namespace lisa {
namespace attn {
namespace {

__device__ __forceinline__ void chain_begin() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_plain(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
    kernel<<<grid, block, smem, s>>>(static_cast<KArgs>(args)...);
    return cudaGetLastError();
}

template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Raises a kernel's shared-memory limit to what the device allows, once per device.
template <auto kKernel>
cudaError_t allow_smem() {
    static std::mutex mu;
    static bool done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, kKernel);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - (int)a.sharedSizeBytes);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

}  // namespace
}  // namespace attn
}  // namespace lisa
