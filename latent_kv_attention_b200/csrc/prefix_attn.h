// prefix_attn.h -- parameters of the shared-prefix attention kernels.
#pragma once

#include <math.h>

#include "../../include/lka.h"
#include "common.cuh"

namespace lka {

struct PrefixParams {
    const void* q;               // [B, h_q, s, D]
    const void *kp, *vp;         // prefix: [h_kv, Lp, D], or the page pools
    const void *k, *v;           // suffixes: [B, h_kv, Lmax, D], or the page pools
    const int32_t* prefix_len;   // device [1], or null: Lp
    const int32_t* lens;         // device [B], suffix lengths
    const int32_t *ptable, *table;  // paged: [max_prefix_pages] and [B, max_pages]; null: contiguous
    void* out;                   // [B, h_q, s, D]
    float* lse;                  // [B, h_q, s] natural log, or null
    float *part_o, *part_lse;    // [B * h_q * s][n_slots][D] and [..][n_slots] (log2 domain)
    uint32_t* status;
    int* next_item;              // items handed out beyond the first of every block; 0 between calls
    int B, h_q, h_kv, s, ratio, R, Lp, Lmax, causal;
    int pre_tokens, n_pre, suf_tokens, n_suf, n_slots;
    int do_prefix, do_suffix;    // which items a launch holds
    int page_size, max_pages, num_pages;
    float scale_log2;
};

// Row tiles of the tensor-core prefix kernel: the R rows of `seqs` sequences (R <= 128), or 128 of one sequence's R.
struct PrefixTiles {
    int seqs, per_seq;  // sequences per tile; tiles per sequence
    int rows, n_tiles;  // rows of a tile, tiles per KV head
    int box_rows;       // key rows per TMA box
};
PrefixTiles prefix_tiles(int B, int R);
lka_status_t prefix_tc(const PrefixParams& p, int d, cudaStream_t st);

// The prefix length, clamped into [0, Lp].
__device__ __forceinline__ int prefix_length(const PrefixParams& p, bool report) {
    int P = p.prefix_len ? *p.prefix_len : p.Lp;
    if (P < 0 || P > p.Lp) {
        if (report) atomicOr(p.status, kDevBadLength);
        P = P < 0 ? 0 : p.Lp;
    }
    return P;
}

// A part of a row, from its maximum and the sum of its exponentials: the sum is 0 where no key counts, and NaN (which the
// row's output and normaliser then are, as in gqa_attn) where a score is NaN.
__device__ __forceinline__ float part_inverse(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float part_normaliser(float m, float sum) { return sum == 0.f ? -INFINITY : m + log2f(sum); }

}  // namespace lka
