// launch_util.h -- launch helpers of the cache operators, and what their kernels need of a launch's form.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "../../include/lka.h"

namespace lka {

// The status of a call whose launches ended with `e`.  The runtime keeps a refused launch's error for whoever asks next:
// it is taken here, so that the next call does not find it after a launch of its own.
inline lka_status_t call_status(cudaError_t e) {
    if (e == cudaSuccess) return LKA_OK;
    cudaGetLastError();
    return LKA_ERR_CUDA;
}

// Test hook, per host thread: the launches by launch_pdl until one is made that the runtime refuses (0: none is).
inline thread_local int t_refused_launch = 0;

// Allows a kernel `bytes` of dynamic shared memory, once per device (always the same bytes for one kernel).
template <auto KERN>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launches the next kernel of one call so that its blocks may start while the kernel before it still runs, from the
// moment all blocks of that one have called pdl_trigger().  Whatever it needs of that kernel it takes after
// pdl_wait(), which returns when the kernel has ended and its writes are visible.
template <auto KERN, class... Args>
cudaError_t launch_pdl(dim3 grid, int block, int smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    if (t_refused_launch > 0 && --t_refused_launch == 0) cfg.blockDim = dim3(4096);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, KERN, args...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
#endif

}  // namespace lka
