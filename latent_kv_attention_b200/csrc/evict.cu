// evict.cu -- cutting a KV cache to a budget of keys per KV head by accumulated
// attention weight (gqa_evict, gqa_evict_paged).
//
// Operation, per sequence and KV head with L cached keys and a budget n < L: the first
// `sinks` keys and the last `recent` keys stay, and of the keys between them the
// n - sinks - recent with the largest weights (equal weights: the lowest position first;
// a NaN weight is less than every number).  The kept rows of K, V and the weights move
// to rows 0 .. n - 1 in the order of their positions.  L <= n keeps everything.
//
// Two kernels.  evict_select_kernel finds the positions: one pass over the weights per
// digit of a radix select (three digits of 11, 11 and 10 bits of the weight's order-
// preserving bits), then one that writes the kept positions in order.
// evict_move_kernel moves the rows: bound by HBM, 2 * d * bytes per kept row read and
// written once.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "host_util.h"
#include "launch_util.h"
#include "mma.cuh"

namespace lka {

struct EvictParams {
    const uint8_t *k, *v;   // [B, h_kv, Lmax, row_bytes] or pages [num_pages, h_kv, page_size, row_bytes]
    uint8_t *ko, *vo;       // [B, h_kv, Lout, row_bytes], or the same pages
    const float* w;         // [B, h_kv, Lmax]
    float* wo;              // [B, h_kv, Lout]
    const int32_t* lens;
    const int32_t* table;
    int32_t* new_lens;      // [B]
    int32_t* kept;          // [B, h_kv, budget] ascending positions, -1 behind them
    uint32_t* status;
    int B, h_kv, Lmax, Lout, row_bytes, budget, sinks, recent;
    int page_size, max_pages, num_pages;
};

namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048, kKeep = 8;  // weights per thread that stay in registers
constexpr int kMaxCluster = 8;

__device__ __forceinline__ int2 cluster_load2(uint32_t addr, uint32_t rank) {
    uint32_t a;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// The weight's bits in an order that unsigned comparison follows: -0 as +0, NaN below every number.
__device__ __forceinline__ uint32_t order_bits(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int evict_len(const EvictParams& p, int b, bool report) {
    int L = p.lens[b];
    if (L < 0 || L > p.Lmax) {
        if (report) atomicOr(p.status, kDevBadLength);
        L = L < 0 ? 0 : p.Lmax;
    }
    return L;
}

// One cluster of `cluster` blocks per (KV head, sequence); each block takes a contiguous part of the weights.  The
// blocks add up one another's histograms through distributed shared memory and all come to the same threshold.
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictParams p, const int cluster) {
    __shared__ __align__(16) int hists[3][kBins];  // one per digit: none is cleared while another block may read it
    __shared__ int part[kSelWarps], part_eq[kSelWarps];
    __shared__ __align__(8) int totals[2];  // this block's keys above the threshold, and equal to it
    __shared__ uint32_t s_prefix;
    __shared__ int s_need, s_whole;
    const int rank = cluster > 1 ? (int)cluster_rank() : 0;
    const int h = (int)blockIdx.x / cluster, b = blockIdx.y, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    pdl_trigger();
    const int L = evict_len(p, b, tid == 0 && blockIdx.x == 0);
    const int n_out = min(L, p.budget);
    if (blockIdx.x == 0 && tid == 0) p.new_lens[b] = n_out;
    int32_t* kept = p.kept + ((size_t)b * p.h_kv + h) * p.budget;
    if (L <= p.budget) {  // the whole cluster
        for (int i = rank * kSelThreads + tid; i < p.budget; i += cluster * kSelThreads) kept[i] = i < L ? i : -1;
        return;
    }
    const float* w = p.w + ((size_t)b * p.h_kv + h) * p.Lmax;
    const int sinks = min(p.sinks, p.budget), recent = min(p.recent, p.budget - sinks);
    const int lo = sinks, hi = L - recent;           // the keys that compete
    const int chosen = p.budget - sinks - recent;    // how many of them stay
    // this block's part of them, whole groups of 32 per warp
    const int share = cdiv(hi - lo, cluster);
    const int b0 = lo + min(hi - lo, rank * share), b1 = lo + min(hi - lo, (rank + 1) * share);
    // Every warp owns a contiguous run [w0, w1) of it.  Up to kKeep weights per thread are read once and kept; a
    // longer run is read again by every pass.
    const int n = b1 - b0, per = cdiv(cdiv(n, kSelWarps), 32) * 32;
    const int w0 = b0 + min(n, warp * per), w1 = b0 + min(n, (warp + 1) * per);
    const bool keep = per <= 32 * kKeep;
    uint32_t own[kKeep];
#pragma unroll
    for (int k = 0; k < kKeep; ++k) own[k] = keep && w0 + 32 * k + lane < w1 ? order_bits(w[w0 + 32 * k + lane]) : 0u;
    // f(position, bits, in the run) for this lane's places, in warp order; whole warps call together
    auto for_each = [&](auto f) {
        if (keep) {
#pragma unroll
            for (int k = 0; k < kKeep; ++k)
                if (w0 + 32 * k < w1) f(w0 + 32 * k + lane, own[k], w0 + 32 * k + lane < w1);
        } else {
            for (int i0 = w0; i0 < w1; i0 += 32) f(i0 + lane, i0 + lane < w1 ? order_bits(w[i0 + lane]) : 0u, i0 + lane < w1);
        }
    };
    uint32_t prefix = 0;
    int need = chosen;  // of the keys whose higher digits equal prefix
    if (chosen > 0) {
        constexpr int shift[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
        for (int i = tid; i < 3 * kBins / 4; i += kSelThreads) reinterpret_cast<int4*>(hists)[i] = make_int4(0, 0, 0, 0);
        if (tid == 0) s_whole = 0;
        __syncthreads();
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            int* hist = hists[d];
            const uint32_t mask = (1u << bits[d]) - 1;
            for_each([&](int, uint32_t u, bool in) {
                if (in && (d == 0 || (u >> (shift[d] + bits[d])) == prefix)) atomicAdd(&hist[(u >> shift[d]) & mask], 1);
            });
            if (cluster > 1)
                cluster_sync();
            else
                __syncthreads();
            // the largest digit with at least `need` keys at or above it: thread tid sums two bins, from the top
            const int nb = 1 << bits[d];
            int c0 = 0, c1 = 0;
            const int top = nb - 1 - 2 * tid;
            if (top >= 1) {
                if (cluster > 1) {
                    int2 two[kMaxCluster];  // all on their way before the first is used
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r)
                        two[r] = r < cluster ? cluster_load2(smem_u32(&hist[top - 1]), r) : make_int2(0, 0);
#pragma unroll
                    for (int r = 0; r < kMaxCluster; ++r) {
                        c0 += two[r].y;
                        c1 += two[r].x;
                    }
                } else {
                    const int2 two = *reinterpret_cast<const int2*>(&hist[top - 1]);
                    c0 = two.y;
                    c1 = two.x;
                }
            }
            int sum = c0 + c1;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (lane == 31) part[warp] = sum;
            __syncthreads();
            int before = lane < warp ? part[lane] : 0;
            before = __reduce_add_sync(0xffffffffu, before) + sum - c0 - c1;
            if (top >= 1 && before < need && before + c0 + c1 >= need) {
                const bool second = before + c0 < need;
                s_prefix = (prefix << bits[d]) | (uint32_t)(second ? top - 1 : top);
                s_need = need - before - (second ? c0 : 0);
                s_whole = s_need == (second ? c1 : c0) && s_prefix > 0;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
            if (s_whole) {  // the digit's keys all stay: no need to tell them apart (mostly so after two digits)
                prefix = (prefix << shift[d]) - 1;
                need = 0;
                break;
            }
        }
    }
    // Count, then write in order.  Keys above the threshold all stay, of those equal to it the first `need`.
    int gt = 0, eq = 0;
    for_each([&](int, uint32_t u, bool in) {
        gt += in && u > prefix;
        eq += in && u == prefix;
    });
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        part[warp] = gt;
        part_eq[warp] = eq;
    }
    for (int i = rank * kSelThreads + tid; i < sinks; i += cluster * kSelThreads) kept[i] = i;
    for (int i = rank * kSelThreads + tid; i < recent; i += cluster * kSelThreads) kept[p.budget - recent + i] = hi + i;
    __syncthreads();
    int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? part[lane] : 0);
    int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? part_eq[lane] : 0);
    if (cluster > 1) {
        if (warp == 0) {
            const int g = __reduce_add_sync(0xffffffffu, part[lane]), e = __reduce_add_sync(0xffffffffu, part_eq[lane]);
            if (lane == 0) {
                totals[0] = g;
                totals[1] = e;
            }
        }
        cluster_sync();
        const int2 two = lane < rank ? cluster_load2(smem_u32(totals), lane) : make_int2(0, 0);
        gt_before += __reduce_add_sync(0xffffffffu, two.x);
        eq_before += __reduce_add_sync(0xffffffffu, two.y);
    }
    if (chosen > 0) {
        int at = sinks + gt_before + min(eq_before, need);
        const uint32_t below = (1u << lane) - 1;
        for_each([&](int i, uint32_t u, bool in) {
            const uint32_t is_eq = __ballot_sync(0xffffffffu, in && u == prefix);
            const bool take = in && (u > prefix || (u == prefix && eq_before + __popc(is_eq & below) < need));
            const uint32_t taken = __ballot_sync(0xffffffffu, take);
            if (take) kept[at + __popc(taken & below)] = i;
            at += __popc(taken);
            eq_before += __popc(is_eq);
        });
    }
    if (cluster > 1) cluster_sync();  // a block's shared memory outlives its readers
}

// Moves the kept rows.  blockIdx.y: KV head, .z: sequence; blockIdx.x: a matrix (K, V, the weights), a slice of its
// row and, when source and destination are different buffers, a range of rows.
// In place, one block owns a slice of all rows and walks them in order, `kRows` at a time: row i's source is at or
// behind row i, so the rows that a step writes are not the source of any later step, and the block loads a whole
// step (and the next one) before it writes.
constexpr int kMoveThreads = 256, kMoveUnroll = 4;

constexpr int kCopyUnroll = 4;  // rows a thread has in flight where nothing orders them

template <typename V, bool IN_PLACE>
__device__ __forceinline__ void move_rows(const EvictParams& p, const uint8_t* src, uint8_t* dst, int64_t src_row0,
                                          int64_t dst_row0, const CacheRows* paged, int row_bytes, int col, int lanes,
                                          const int32_t* kept, int r0, int r1) {
    // `lanes` threads of V bytes carry one row's slice at byte `col`
    const int sub = threadIdx.x % lanes, first = threadIdx.x / lanes, step = kMoveThreads / lanes;
    const bool on = first < step;  // lanes need not divide the block
    const int64_t off = col + (int64_t)sub * sizeof(V);
    if constexpr (!IN_PLACE) {
        for (int base = r0 + first; base < r1; base += kCopyUnroll * step) {
            int from[kCopyUnroll];
            V x[kCopyUnroll];
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u) from[u] = on && base + u * step < r1 ? kept[base + u * step] : -1;
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (from[u] >= 0) x[u] = *reinterpret_cast<const V*>(src + (src_row0 + from[u]) * row_bytes + off);
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u)
                if (from[u] >= 0) *reinterpret_cast<V*>(dst + (dst_row0 + base + u * step) * row_bytes + off) = x[u];
        }
    } else {
        V buf[kMoveUnroll], nxt[kMoveUnroll];
        auto load = [&](int base, V* to) {
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u) {
                const int r = base + u * step + first;
                if (on && r < r1) {
                    const int from = kept[r];
                    const int64_t row = paged ? cache_row(*paged, from, p.status) : src_row0 + from;
                    to[u] = *reinterpret_cast<const V*>(src + row * row_bytes + off);
                }
            }
        };
        load(r0, buf);
        for (int base = r0; base < r1; base += kMoveUnroll * step) {
            load(base + kMoveUnroll * step, nxt);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kMoveUnroll; ++u) {
                const int r = base + u * step + first;
                if (on && r < r1) {
                    const int64_t row = paged ? cache_row_or_none(*paged, r, p.status) : dst_row0 + r;
                    if (row >= 0) *reinterpret_cast<V*>(dst + row * row_bytes + off) = buf[u];
                }
                buf[u] = nxt[u];
            }
            __syncthreads();
        }
    }
}

struct MovePlan {
    int slice;    // bytes of a K / V row per block
    int slices;   // of one row
    int ranges;   // of rows (1 in place)
};

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, IN_PLACE ? 4 : 7) evict_move_kernel(const EvictParams p, const MovePlan m) {
    const int h = blockIdx.y, b = blockIdx.z;
    const int range = blockIdx.x % m.ranges, what = blockIdx.x / m.ranges;
    const int32_t* kept = p.kept + ((size_t)b * p.h_kv + h) * p.budget;
    const int64_t bh = (int64_t)b * p.h_kv + h;
    pdl_wait();
    if (what == 2 * m.slices) {  // the weights; the places behind the kept keys start from nothing
        const int n = min(evict_len(p, b, false), p.budget);
        const int per = cdiv(n, m.ranges), r0 = min(n, range * per), r1 = min(n, r0 + per);
        move_rows<float, IN_PLACE>(p, reinterpret_cast<const uint8_t*>(p.w), reinterpret_cast<uint8_t*>(p.wo), bh * p.Lmax,
                                   bh * p.Lout, nullptr, 4, 0, 1, kept, r0, r1);
        const int z = p.Lout - n, zper = cdiv(z, m.ranges);
        for (int i = n + range * zper + threadIdx.x; i < min(p.Lout, n + (range + 1) * zper); i += kMoveThreads)
            p.wo[bh * p.Lout + i] = 0.f;
        return;
    }
    const bool is_v = what >= m.slices;
    const int col = (what - (is_v ? m.slices : 0)) * m.slice;
    const int bytes = min(m.slice, p.row_bytes - col);
    if constexpr (IN_PLACE) {
        const int L = evict_len(p, b, false);
        if (L <= p.budget) return;  // nothing leaves
        const CacheRows rows{p.table ? p.table + (size_t)b * p.max_pages : nullptr, p.page_size, p.num_pages, h, p.h_kv};
        move_rows<uint4, true>(p, is_v ? p.v : p.k, is_v ? p.vo : p.ko, bh * p.Lmax, bh * p.Lout, p.table ? &rows : nullptr,
                               p.row_bytes, col, bytes / 16, kept, 0, p.budget);
    } else {
        // the list itself says where the kept rows end
        const int per = cdiv(p.budget, m.ranges), r0 = min(p.budget, range * per);
        move_rows<uint4, false>(p, is_v ? p.v : p.k, is_v ? p.vo : p.ko, bh * p.Lmax, bh * p.Lout, nullptr, p.row_bytes, col,
                                bytes / 16, kept, r0, min(p.budget, r0 + per));
    }
}

lka_status_t evict_run(EvictParams& p, int d, lka_dtype_t dtype, size_t ws_bytes, void* ws, void* stream) {
    if (p.B < 0 || p.h_kv < 1 || d < 1 || p.Lmax < 1 || p.Lout < 1 || p.budget < 1 || p.sinks < 0 || p.recent < 0)
        return LKA_ERR_INVALID_ARG;
    if (p.budget > p.Lout) return LKA_ERR_INVALID_ARG;
    if (dtype != LKA_BF16 && dtype != LKA_FP32 && dtype != LKA_E4M3) return LKA_ERR_UNSUPPORTED;
    const int eb = dtype == LKA_BF16 ? 2 : dtype == LKA_FP32 ? 4 : 1;
    if (d > 65536 || (d * eb) % 16 || p.B > 65535 || p.h_kv > 65535 || p.Lmax > (1 << 30) || p.Lout > (1 << 30))
        return LKA_ERR_UNSUPPORTED;
    p.row_bytes = d * eb;
    if (p.B == 0) return LKA_OK;
    const void* ptrs[] = {p.k, p.v, p.ko, p.vo, p.w, p.wo, p.lens, p.new_lens, p.kept};
    for (const void* x : ptrs)
        if (!x || !aligned16(x)) return LKA_ERR_INVALID_ARG;
    if (p.new_lens == p.lens) return LKA_ERR_INVALID_ARG;
    const bool in_place = p.k == p.ko;
    if (p.table) {
        const size_t pool = (size_t)p.num_pages * p.h_kv * p.page_size * p.row_bytes;
        if (overlap(p.ko, pool, p.vo, pool)) return LKA_ERR_INVALID_ARG;
    } else {
        const size_t rows_in = (size_t)p.B * p.h_kv * p.Lmax, rows_out = (size_t)p.B * p.h_kv * p.Lout;
        if (overlap(p.ko, rows_out * p.row_bytes, p.vo, rows_out * p.row_bytes)) return LKA_ERR_INVALID_ARG;
        if (in_place) {
            if (p.v != p.vo || p.w != p.wo || p.Lmax != p.Lout) return LKA_ERR_INVALID_ARG;
        } else if (overlap(p.k, rows_in * p.row_bytes, p.ko, rows_out * p.row_bytes) ||
                   overlap(p.v, rows_in * p.row_bytes, p.vo, rows_out * p.row_bytes) ||
                   overlap(p.k, rows_in * p.row_bytes, p.vo, rows_out * p.row_bytes) ||
                   overlap(p.v, rows_in * p.row_bytes, p.ko, rows_out * p.row_bytes) ||
                   overlap(p.w, rows_in * 4, p.wo, rows_out * 4)) {
            return LKA_ERR_INVALID_ARG;
        }
    }
    if (!ws || ws_bytes < kWsHeaderBytes) return LKA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LKA_ERR_INVALID_ARG;
    p.status = static_cast<uint32_t*>(ws);
    const cudaStream_t st = (cudaStream_t)stream;
    // Up to 8192 weights a row fits one block's registers.  A longer row is shared by a cluster while all clusters run
    // at once (both kernels: 32 rows of 17,600 weights 25 us alone, 20 in fours; 8 of 65,536: 82, 33 in fours, 21 in
    // eights), but clusters of eight blocks of 1024 threads find few places (32 rows: 45 us), nor do fours past the
    // number of SMs (56 rows of 17,600: 29 us alone, 34 in fours).
    const long long rows = (long long)p.B * p.h_kv;
    int cluster = 1;
    if (p.Lmax > 4 * kKeep * kSelThreads && rows <= 8)
        cluster = 8;
    else if (p.Lmax > kKeep * kSelThreads && rows * 4 <= sm_count())
        cluster = 4;
    else if (p.Lmax > 4 * kKeep * kSelThreads && rows * 2 <= sm_count())
        cluster = 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.h_kv * cluster, p.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    TimedLaunch timer(st);  // of both kernels: which is the longer depends on the shape
    cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, cluster);
    if (e != cudaSuccess) return call_status(e);
    MovePlan m;
    if (in_place) {
        // one block walks all rows of its slice: slices of 64 bytes (two sectors) give the parallelism
        m.slice = std::min(p.row_bytes, 64);
        m.ranges = 1;
    } else {
        // whole rows, kCopyUnroll per thread and block: short blocks, all of whose reads are in flight at once
        m.slice = std::min(p.row_bytes, 16 * kMoveThreads);
        m.ranges = std::min(cdiv(p.budget, kCopyUnroll * (kMoveThreads / (m.slice / 16))), 32768);
    }
    m.slices = cdiv(p.row_bytes, m.slice);
    const dim3 grid((2 * m.slices + 1) * m.ranges, p.h_kv, p.B);
    e = in_place ? launch_pdl<evict_move_kernel<true>>(grid, kMoveThreads, 0, st, p, m)
                 : launch_pdl<evict_move_kernel<false>>(grid, kMoveThreads, 0, st, p, m);
    timer.stop();
    return call_status(e);
}

}  // namespace
}  // namespace lka

using namespace lka;

extern "C" {

lka_status_t gqa_evict(const void* k, const void* v, const float* weights, const int32_t* cache_lens, void* k_out,
                       void* v_out, float* weights_out, int32_t* new_lens, int32_t* kept, int B, int h_kv, int d_h,
                       int Lmax, int Lout, int budget, int sinks, int recent, lka_dtype_t dtype, void* ws,
                       size_t ws_bytes, void* stream) {
    EvictParams p{};
    p.k = static_cast<const uint8_t*>(k);
    p.v = static_cast<const uint8_t*>(v);
    p.ko = static_cast<uint8_t*>(k_out);
    p.vo = static_cast<uint8_t*>(v_out);
    p.w = weights;
    p.wo = weights_out;
    p.lens = cache_lens;
    p.new_lens = new_lens;
    p.kept = kept;
    p.B = B;
    p.h_kv = h_kv;
    p.Lmax = Lmax;
    p.Lout = Lout;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    return evict_run(p, d_h, dtype, ws_bytes, ws, stream);
}

lka_status_t gqa_evict_paged(void* k_pages, void* v_pages, float* weights, const int32_t* block_table,
                             const int32_t* cache_lens, int32_t* new_lens, int32_t* kept, int B, int h_kv, int d_h,
                             int page_size, int max_pages, int num_pages, int budget, int sinks, int recent,
                             lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream) {
    if (page_size < 8 || (page_size & (page_size - 1)) || max_pages < 1 || num_pages < 1) return LKA_ERR_INVALID_ARG;
    if ((long long)max_pages * page_size > (1 << 30)) return LKA_ERR_UNSUPPORTED;
    if (B > 0 && (!block_table || (reinterpret_cast<uintptr_t>(block_table) & 3u))) return LKA_ERR_INVALID_ARG;
    EvictParams p{};
    p.k = p.ko = static_cast<uint8_t*>(k_pages);
    p.v = p.vo = static_cast<uint8_t*>(v_pages);
    p.w = p.wo = weights;
    p.lens = cache_lens;
    p.table = block_table;
    p.new_lens = new_lens;
    p.kept = kept;
    p.B = B;
    p.h_kv = h_kv;
    p.Lmax = p.Lout = page_size * max_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    return evict_run(p, d_h, dtype, ws_bytes, ws, stream);
}

}  // extern "C"
