// key_weights.cu -- the attention weight every cached key received (gqa_key_weights,
// gqa_key_weights_paged): the quantity a cache is cut by.
//
// Operation: for each (sequence, KV head, key j), over the h_q / h_kv heads of the group
// and the s_q queries t that see the key,
//     w_j = sum_{head, t} exp(scale <q_{head,t}, k_j> - lse_{head,t})
// with the log-sum-exp of each query row as gqa_attn returned it: the probabilities are
// recomputed, never stored.
//
// Every key belongs to one warp, which sums its weights over all rows in fp32 and in a
// fixed order: no atomics, the same bits every time.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "host_util.h"
#include "key_weights.h"
#include "launch_util.h"
#include "mma.cuh"

namespace lka {

namespace {

constexpr int kTile = 64;  // keys per block

__device__ __forceinline__ void write_weight(const KeyWeightParams& p, size_t at, float v) {
    p.w[at] = p.accumulate ? p.w[at] + v : v;
}

// The rows of the group an fp32 block walks: flat over (head, query) while a head has few queries; head by head, from
// the first query that sees the tile's first key, when it has many (a prompt's causal half is skipped).
struct RowWalk {
    int segs, len, start;
};
__device__ __forceinline__ RowWalk row_walk(const KeyWeightParams& p, int j0, int L) {
    if (p.s < kTile) return {1, p.ratio * p.s, 0};
    return {p.ratio, p.s, p.causal ? max(0, (j0 - (L - p.s)) & ~7) : 0};
}

// bf16 caches.  S^T = K Q^T: a warp's 16 keys are the MMA's rows and stay in registers, read straight from global
// memory 16 bytes a lane; the query rows pass through shared memory as columns, 8 at a time.  The head dim is
// contracted in an order of its own, the same for both operands: in 32-value group j, lane column t brings values
// 32 j + 8 t .. + 7, the first four to k-step 2j, the last four to 2j + 1.
// A decode step is bound by reading the keys: a warp walks `groups` groups of 16 keys and has the next group's loads
// (4 KB at D = 128) under way while it works on this one.
// Blocks per SM as many as the next tile's keys leave registers for (at d = 128 five: 116.7 us for 64 sequences of
// 1024-8192 keys, caches out of L2; four, which the compiler takes to on its own, 122.9).
template <int D>
__global__ void __launch_bounds__(128, D == 64 ? 8 : D == 128 ? 5 : 3) key_weights_mma_kernel(const KeyWeightParams p) {
    constexpr int NJ = D / 32;
    constexpr int QROW = D * 2 + 64;  // bytes; rows g and g + 1 fall in different halves of the banks
    extern __shared__ __align__(16) uint8_t smem[];
    const int chunk = p.chunk;
    uint8_t* qs = smem;                                                    // [2][chunk][QROW]
    float* ls = reinterpret_cast<float*>(smem + 2 * (size_t)chunk * QROW);  // [2][chunk] log2 normalisers
    const int kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int L = clamp_len(p.lens, b, p.Lmax, p.s, p.causal, p.status, threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0);
    const size_t wrow = ((size_t)b * p.h_kv + kvh) * p.Lmax;
    const int first_tile = blockIdx.x * p.groups, block0 = first_tile * kTile;
    if (!p.accumulate)  // the block's keys past the length
        for (int j = max(block0, L) + threadIdx.x; j < min(block0 + p.groups * kTile, p.Lmax); j += 128) p.w[wrow + j] = 0.f;
    if (block0 >= L) return;
    const int n_tiles = min(p.groups, cdiv(L - block0, kTile));
    const CacheRows rows{p.table ? p.table + (size_t)b * p.max_pages : nullptr, p.page_size, p.num_pages,
                         p.table ? (long long)kvh : ((long long)b * p.h_kv + kvh) * p.Lmax, p.h_kv};
    // this lane's two keys of a tile: rows g and g + 8 of the warp's 16
    auto load_keys = [&](int j0, uint4 (*to)[NJ]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int key = j0 + warp * 16 + g + 8 * h;
            const bool ok = key < L;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.k) + (ok ? cache_row(rows, key, p.status) : 0) * D;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                to[h][j] = ok ? __ldg(reinterpret_cast<const uint4*>(src + 32 * j + 8 * t)) : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 kr[2][NJ], kn[2][NJ];
    load_keys(block0, kr);

    const int n_rows = p.ratio * p.s, n_chunks = cdiv(n_rows, chunk);  // flat over (head, query): a head has few queries
    const size_t row0 = ((size_t)b * p.h_q + (size_t)kvh * p.ratio) * p.s;
    auto stage = [&](int c) {
        const int first = c * chunk, n = min(chunk, n_rows - first), buf = c & 1;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + (row0 + first) * D;
        for (int i = threadIdx.x; i < chunk * (D / 8); i += 128) {
            const int r = i / (D / 8), ch = i % (D / 8);
            cp_async16(smem_u32(qs + ((size_t)buf * chunk + r) * QROW + ch * 16), q + (r < n ? (size_t)r * D + ch * 8 : 0),
                       r < n);
        }
        for (int r = threadIdx.x; r < chunk; r += 128) {
            const float l = r < n ? p.lse[row0 + first + r] : -INFINITY;
            ls[buf * chunk + r] = l == -INFINITY ? INFINITY : l * kLog2e;  // a row without keys gives nothing
        }
        cp_async_commit();
    };
    // Several tiles per block only where all rows are one chunk (kernel launch); otherwise one tile and all chunks.
    stage(0);
    for (int tile = 0; tile < n_tiles; ++tile) {
        const int j0 = block0 + tile * kTile;
        if (tile + 1 < n_tiles) load_keys(j0 + kTile, kn);
        float w[2] = {0.f, 0.f};
        for (int c = 0; c < n_chunks; ++c) {
            if (tile == 0) {
                if (c + 1 < n_chunks) {
                    stage(c + 1);
                    cp_async_wait<1>();
                } else {
                    cp_async_wait<0>();
                }
                __syncthreads();
            }
            const int first = c * chunk, n = min(chunk, n_rows - first);
            const uint8_t* qb = qs + (size_t)(c & 1) * chunk * QROW;
            const float* lb = ls + (c & 1) * chunk;
            // queries that may not see every key of the tile need the mask
            const bool masked = (p.causal && j0 + kTile - 1 > L - p.s) || j0 + kTile > L;
#pragma unroll 2
            for (int r0 = 0; r0 < n; r0 += 8) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const uint8_t* qrow = qb + (r0 + g) * QROW + t * 16;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const uint4 qv = *reinterpret_cast<const uint4*>(qrow + j * 64);
                    const uint32_t a0[4] = {kr[0][j].x, kr[1][j].x, kr[0][j].y, kr[1][j].y};
                    const uint32_t a1[4] = {kr[0][j].z, kr[1][j].z, kr[0][j].w, kr[1][j].w};
                    mma_bf16(acc, a0, qv.x, qv.y);
                    mma_bf16(acc, a1, qv.z, qv.w);
                }
                const float2 l2 = *reinterpret_cast<const float2*>(lb + r0 + 2 * t);
                float e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float l = i & 1 ? l2.y : l2.x;
                    e[i] = l == INFINITY ? 0.f : fast_exp2(fmaf(acc[i], p.scale_log2, -l));  // (an empty row may score NaN)
                }
                if (masked || r0 + 8 > n) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = r0 + 2 * t + (i & 1), key = j0 + warp * 16 + g + 8 * (i / 2);
                        const int last = p.causal ? L - p.s + (first + r) % p.s : L - 1;
                        if (r >= n || key > last) e[i] = 0.f;
                    }
                }
                w[0] += e[0] + e[1];
                w[1] += e[2] + e[3];
            }
            if (n_chunks > 1) __syncthreads();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[h] += __shfl_xor_sync(0xffffffffu, w[h], 1);
            w[h] += __shfl_xor_sync(0xffffffffu, w[h], 2);
            const int key = j0 + warp * 16 + g + 8 * h;
            if (t == 0 && key < L) write_weight(p, wrow + key, w[h]);
#pragma unroll
            for (int j = 0; j < NJ; ++j) kr[h][j] = kn[h][j];
        }
    }
}

// fp32 caches: one key per lane pair (two halves of the rows), the tile and RB query rows at a time in shared memory
// (4 where the group has no more, so that a decode step computes no empty rows).
template <int D, int RB>
__global__ void __launch_bounds__(128) key_weights_f32_kernel(const KeyWeightParams p) {
    constexpr int KROW = D + 4;
    extern __shared__ __align__(16) uint8_t smem[];
    float* ks = reinterpret_cast<float*>(smem);  // [kTile][KROW]
    float* qs = ks + kTile * KROW;               // [RB][D]
    float* ls = qs + RB * D;                     // [RB]
    float* red = ls + RB;                        // [kTile]
    const int j0 = blockIdx.x * kTile, kvh = blockIdx.y, b = blockIdx.z;
    const int L = clamp_len(p.lens, b, p.Lmax, p.s, p.causal, p.status, threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0);
    const size_t wrow = ((size_t)b * p.h_kv + kvh) * p.Lmax;
    const int kk = threadIdx.x % kTile, half = threadIdx.x / kTile, key = j0 + kk;
    if (j0 >= L) {
        if (half == 0 && key < p.Lmax && !p.accumulate) p.w[wrow + key] = 0.f;
        return;
    }
    const CacheRows rows{p.table ? p.table + (size_t)b * p.max_pages : nullptr, p.page_size, p.num_pages,
                         p.table ? (long long)kvh : ((long long)b * p.h_kv + kvh) * p.Lmax, p.h_kv};
    for (int i = threadIdx.x; i < kTile * (D / 4); i += 128) {
        const int r = i / (D / 4), c = i % (D / 4), tok = j0 + r;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tok < L) v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.k) + cache_row(rows, tok, p.status) * D + c * 4);
        *reinterpret_cast<float4*>(ks + r * KROW + c * 4) = v;
    }
    const RowWalk walk = row_walk(p, j0, L);
    const size_t row0 = ((size_t)b * p.h_q + (size_t)kvh * p.ratio) * p.s;
    float w = 0.f;
    for (int seg = 0; seg < walk.segs; ++seg)
        for (int r0 = walk.start; r0 < walk.len; r0 += RB) {
            const int first = seg * walk.len + r0, n = min(RB, walk.len - r0);
            __syncthreads();
            for (int i = threadIdx.x; i < RB * (D / 4); i += 128) {
                const int r = i / (D / 4), c = i % (D / 4);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < n) v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (row0 + first + r) * D + c * 4);
                *reinterpret_cast<float4*>(qs + r * D + c * 4) = v;
            }
            if (threadIdx.x < RB) {
                const float l = threadIdx.x < n ? p.lse[row0 + first + threadIdx.x] : -INFINITY;
                ls[threadIdx.x] = l == -INFINITY ? INFINITY : l * kLog2e;
            }
            __syncthreads();
            float acc[RB / 2] = {};
            const float* kp = ks + kk * KROW;
            const float* qp = qs + half * (RB / 2) * D;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 kv = *reinterpret_cast<const float4*>(kp + c);
#pragma unroll
                for (int r = 0; r < RB / 2; ++r) {
                    const float4 qv = *reinterpret_cast<const float4*>(qp + r * D + c);
                    acc[r] = fmaf(kv.x, qv.x, fmaf(kv.y, qv.y, fmaf(kv.z, qv.z, fmaf(kv.w, qv.w, acc[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < RB / 2; ++r) {
                const int rr = half * (RB / 2) + r;
                const int last = p.causal ? L - p.s + (first + rr) % p.s : L - 1;
                if (rr < n && key <= last && key < L && ls[rr] != INFINITY) w += exp2f(fmaf(acc[r], p.scale_log2, -ls[rr]));
            }
        }
    if (half) red[kk] = w;
    __syncthreads();
    if (!half) {
        if (key < L)
            write_weight(p, wrow + key, w + red[kk]);
        else if (key < p.Lmax && !p.accumulate)
            p.w[wrow + key] = 0.f;
    }
}

template <int D>
cudaError_t launch_mma(KeyWeightParams p, dim3 grid, cudaStream_t st) {
    // whole groups of 8 rows; 64 rows at a time hide the copies of the next ones behind 8 MMA column groups
    p.chunk = std::min(64, cdiv(p.ratio * p.s, 8) * 8);
    const int smem = 2 * p.chunk * (D * 2 + 64 + 4);
    // several tiles of keys per block, for the loads ahead, where the rows are one chunk and the blocks stay many
    p.groups = 1;
    if (p.ratio * p.s <= p.chunk)
        while (p.groups < 8 && (long long)grid.y * grid.z * cdiv(p.Lmax, kTile * p.groups * 2) >= 8LL * sm_count()) p.groups *= 2;
    grid.x = cdiv(p.Lmax, kTile * p.groups);
    const cudaError_t e = allow_smem<key_weights_mma_kernel<D>>(2 * 64 * (D * 2 + 64 + 4));
    if (e != cudaSuccess) return e;
    TimedLaunch timer(st);
    key_weights_mma_kernel<D><<<grid, 128, smem, st>>>(p);
    timer.stop();
    return cudaPeekAtLastError();
}

template <int D, int RB>
cudaError_t launch_f32_rows(const KeyWeightParams& p, const dim3& grid, cudaStream_t st) {
    constexpr int smem = (kTile * (D + 4) + RB * D + RB + kTile) * 4;
    const cudaError_t e = allow_smem<key_weights_f32_kernel<D, RB>>(smem);
    if (e != cudaSuccess) return e;
    TimedLaunch timer(st);
    key_weights_f32_kernel<D, RB><<<grid, 128, smem, st>>>(p);
    timer.stop();
    return cudaPeekAtLastError();
}

template <int D>
cudaError_t launch_f32(const KeyWeightParams& p, const dim3& grid, cudaStream_t st) {
    return p.ratio * p.s <= 4 ? launch_f32_rows<D, 4>(p, grid, st) : launch_f32_rows<D, 16>(p, grid, st);
}

struct KwPages {
    const int32_t* table;
    int page_size, max_pages, num_pages;
};

lka_status_t key_weights_run(const void* q, const void* k, const float* lse, const int32_t* lens, float* w, int B,
                             int h_q, int h_kv, int s, int d, int Lmax, int causal, int accumulate, float scale,
                             lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream, const KwPages* pg) {
    if (B < 0 || h_q < 1 || h_kv < 1 || s < 1 || d < 1 || Lmax < 1 || h_q % h_kv) return LKA_ERR_INVALID_ARG;
    if (dtype != LKA_BF16 && dtype != LKA_FP32) return LKA_ERR_UNSUPPORTED;
    if (!(d == 64 || d == 128 || (d == 256 && dtype == LKA_BF16))) return LKA_ERR_UNSUPPORTED;
    if (B > 65535 || h_kv > 65535 || (long long)h_q * s >= (1ll << 31) || Lmax > (1 << 30)) return LKA_ERR_UNSUPPORTED;
    if (B == 0) return LKA_OK;
    if (!q || !k || !lse || !lens || !w || !aligned16(q) || !aligned16(k) || !aligned16(lse) || !aligned16(lens) ||
        !aligned16(w) || !isfinite(scale))
        return LKA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < kWsHeaderBytes) return LKA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LKA_ERR_INVALID_ARG;
    KeyWeightParams p{};
    p.q = q;
    p.k = k;
    p.lse = lse;
    p.lens = lens;
    p.w = w;
    p.status = static_cast<uint32_t*>(ws);
    p.B = B;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.s = s;
    p.Lmax = Lmax;
    p.causal = causal ? 1 : 0;
    p.accumulate = accumulate ? 1 : 0;
    p.ratio = h_q / h_kv;
    p.scale_log2 = scale * kLog2e;
    if (pg) {
        p.table = pg->table;
        p.page_size = pg->page_size;
        p.max_pages = pg->max_pages;
        p.num_pages = pg->num_pages;
    }
    const dim3 grid(cdiv(Lmax, kTile), h_kv, B);
    const cudaStream_t st = (cudaStream_t)stream;
    if (dtype == LKA_BF16 && s >= kKeyWeightsTcMinQueries) return key_weights_tc(p, d, st);
    cudaError_t e;
    if (dtype == LKA_FP32)
        e = d == 64 ? launch_f32<64>(p, grid, st) : launch_f32<128>(p, grid, st);
    else
        e = d == 64 ? launch_mma<64>(p, grid, st) : d == 128 ? launch_mma<128>(p, grid, st) : launch_mma<256>(p, grid, st);
    return call_status(e);
}

}  // namespace
}  // namespace lka

using namespace lka;

extern "C" {

lka_status_t gqa_key_weights(const void* q, const void* k, const float* lse, const int32_t* cache_lens, float* weights,
                             int B, int h_q, int h_kv, int s_q, int d_h, int Lmax, int causal, int accumulate,
                             float scale, lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream) {
    return key_weights_run(q, k, lse, cache_lens, weights, B, h_q, h_kv, s_q, d_h, Lmax, causal, accumulate, scale,
                           dtype, ws, ws_bytes, stream, nullptr);
}

lka_status_t gqa_key_weights_paged(const void* q, const void* k_pages, const float* lse, const int32_t* block_table,
                                   const int32_t* cache_lens, float* weights, int B, int h_q, int h_kv, int s_q,
                                   int d_h, int page_size, int max_pages, int num_pages, int causal, int accumulate,
                                   float scale, lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream) {
    if (page_size < 8 || (page_size & (page_size - 1)) || max_pages < 1 || num_pages < 1) return LKA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size >= (1ll << 31)) return LKA_ERR_UNSUPPORTED;
    if (B > 0 && (!block_table || (reinterpret_cast<uintptr_t>(block_table) & 3u))) return LKA_ERR_INVALID_ARG;
    const KwPages pg{block_table, page_size, max_pages, num_pages};
    return key_weights_run(q, k_pages, lse, cache_lens, weights, B, h_q, h_kv, s_q, d_h, page_size * max_pages, causal,
                           accumulate, scale, dtype, ws, ws_bytes, stream, &pg);
}

}  // extern "C"
