// decode_launch.h -- launch helpers of the decoding kernels.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace lossk {

// A launch that may begin before the kernel ahead of it in the stream has
// ended (`after`: that kernel is one of the same call); the kernel waits with
// griddepcontrol.wait before it touches memory.
template <typename... P, typename... A>
cudaError_t launch_after(bool after, void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Lets kernel K take `bytes` of dynamic shared memory: set on the current device
// when first needed, or when more is.
template <auto K> cudaError_t raise_smem(size_t bytes)
{
    static std::atomic<size_t> have[64];
    if (bytes <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 64;
    if (known && have[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    // the most a block can have beside a kernel's static arrays, once and for all
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, K);
    if (e != cudaSuccess) return e;
    const size_t most = 227 * 1024 - attr.sharedSizeBytes;
    if (bytes > most) return cudaErrorInvalidValue;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e == cudaSuccess && known) have[dev].store(most, std::memory_order_release);
    return e;
}

} // namespace lossk
