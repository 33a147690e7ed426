// status.cu -- status words of calls captured into CUDA graphs: a captured call raises its flags in scratch of its
// graph's, from where they are added to a header that outlives it.
#include "common.cuh"
#include "host_util.h"

namespace lka {

// Atomically: graphs that replay at the same time, and calls that raise flags in the header itself, lose nothing.
__global__ void add_status_kernel(uint32_t* to, const uint32_t* from) {
    if (const uint32_t flags = *from) atomicOr(to, flags);
}

}  // namespace lka

extern "C" lka_status_t lka_add_status(void* to, const void* ws, void* stream) {
    if (!to || !ws || !lka::aligned16(to) || !lka::aligned16(ws)) return LKA_ERR_INVALID_ARG;
    lka::add_status_kernel<<<1, 1, 0, (cudaStream_t)stream>>>(static_cast<uint32_t*>(to), static_cast<const uint32_t*>(ws));
    return cudaPeekAtLastError() == cudaSuccess ? LKA_OK : LKA_ERR_CUDA;
}
