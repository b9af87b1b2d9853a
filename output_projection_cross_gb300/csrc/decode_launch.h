// decode_launch.h -- launch helpers of the decoding kernels.
#pragma once
#include <atomic>
#include <cuda_runtime.h>

namespace lossk {

// What is ahead of a kernel in its stream has ended, and its memory is there to
// see, after this: the first thing that every thread of a kernel does that
// launch() starts.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A launch whose blocks may be set up while the kernel ahead of them in the
// stream, of whatever call, ends.  Between two calls of a few microseconds that
// saves 2 us of each (4 beams over 32000 tokens: 14.1 -> 11.6 us a call).
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args)
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
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Lets kernel K take `bytes` of dynamic shared memory: set on the current device
// when first needed.  (Without it a block has 48 KB in all, its static arrays
// among them: a kernel of 3 KB of those is refused 46 KB beside them.)
template <auto K> cudaError_t raise_smem(size_t bytes)
{
    static std::atomic<size_t> have[64];
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
