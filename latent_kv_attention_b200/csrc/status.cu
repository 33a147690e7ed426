// status.cu -- status words of calls captured into CUDA graphs.
//
// A captured call's scratch belongs to its graph, so its flags have to outlive it in a header that no graph owns: one per
// device, inside the library, zero when the library is loaded and at one address until the process ends.  It is not
// allocated, so that its first use may be inside a capture (memory taken there is the graph's, and so is its zero fill:
// every replay of that graph would clear what other graphs raised).
#include <atomic>

#include "common.cuh"
#include "host_util.h"
#include "launch_util.h"

namespace lka {

static __device__ __align__(256) uint8_t g_captured_header[kWsHeaderBytes];

// The address on each device, looked up once with that device current.
static std::atomic<void*> g_captured_addr[64];

// Atomically: graphs that replay at the same time, and calls that raise flags in the header itself, lose nothing.
__global__ void add_status_kernel(uint32_t* to, const uint32_t* from) {
    if (const uint32_t flags = *from) atomicOr(to, flags);
}

}  // namespace lka

extern "C" void* lka_captured_header(void) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    void* p = lka::g_captured_addr[dev].load(std::memory_order_acquire);
    if (p) return p;
    // the lookup may load this file's code onto the device, which a capture under way on some stream forbids otherwise
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, lka::g_captured_header);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess || !p) return nullptr;
    lka::g_captured_addr[dev].store(p, std::memory_order_release);
    return p;
}

extern "C" lka_status_t lka_add_status(void* to, const void* ws, void* stream) {
    if (!to || !ws || !lka::aligned16(to) || !lka::aligned16(ws)) return LKA_ERR_INVALID_ARG;
    lka::add_status_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(static_cast<uint32_t*>(to), static_cast<const uint32_t*>(ws));
    return lka::call_status(cudaPeekAtLastError());
}
