// key_weights.h -- parameters of the key-weight kernels.
#pragma once

#include "../../include/lka.h"
#include "common.cuh"

namespace lka {

struct KeyWeightParams {
    const void* q;        // [B, h_q, s, D]
    const void* k;        // [B, h_kv, Lmax, D] or pages [num_pages, h_kv, page_size, D]
    const float* lse;     // [B, h_q, s] natural log
    const int32_t* lens;  // [B]
    const int32_t* table;
    float* w;             // [B, h_kv, Lmax]
    uint32_t* status;
    int B, h_q, h_kv, s, Lmax, causal, accumulate, ratio;
    int page_size, max_pages, num_pages;
    int chunk;            // query rows staged at a time (a multiple of 8)
    int groups;           // tiles of keys per block
    float scale_log2;
};

constexpr float kLog2e = 1.4426950408889634f;

// Queries per head from which the tensor-core kernel runs (bf16): a tile of 128 query rows is half
// full there.
constexpr int kKeyWeightsTcMinQueries = 64;
lka_status_t key_weights_tc(const KeyWeightParams& p, int d, cudaStream_t st);

}  // namespace lka
