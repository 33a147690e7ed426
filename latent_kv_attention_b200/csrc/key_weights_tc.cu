// key_weights_tc.cu -- the attention weight every key received from a prompt's queries,
// on the 5th-generation tensor cores (bf16, many queries per head).
//
// S^T = K Q^T: one CTA keeps a tile of 128 keys (the MMA's rows, one per tensor-memory
// lane) and streams tiles of 128 query rows of the group's heads (the columns) through a TMA
// ring.  A key's weight is a sum along its own lane, so nothing crosses lanes and no P is
// written back: per score one multiply-add with the row's normaliser, one exponential, one
// addition.  Warp 8 loads, warp 9 issues the MMAs into two score buffers of tensor memory, two
// groups of four warps take the score tiles in turn; two CTAs per SM (one at d = 256) cover
// each other's starts and waits.  With few key tiles, the query tiles of one key tile are dealt to the CTAs of a
// cluster, whose sums rank 0 adds in order.
//
// Bound: 16,384 exponentials per tile are 1024 cycles of the special-function unit (16 per
// cycle and SM) against 520 of the tensor pipe at d = 128.  Measured after a causal prompt of
// 4096 tokens, 32 / 8 heads of 128 (16,896 tiles): 106-107 us among other calls (97 at best), the
// unit about 0.7 busy.  Beside the best figure: one CTA per SM with four groups and one issuing
// thread 101 us (that thread's 1400 cycles per tile), with three issuing threads 102-106; a quarter
// or three eighths of the exponentials as polynomials on the FMA pipe 100-112 in every layout.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "host_util.h"
#include "key_weights.h"
#include "launch_util.h"
#include "tc.cuh"

namespace lka {

namespace kwt {
constexpr int TK = 128, TQ = 128, NBUF = 2;
constexpr int NG = 2, W_LOAD = 4 * NG, W_MMA = W_LOAD + 1, NT = 32 * (W_MMA + 1);  // groups of four warps, one per buffer
template <int D>
struct Cfg {
    static constexpr int NB = D / 64, BOX = 128 * 128, TILE = NB * BOX;
    static constexpr int NS = D == 64 ? 4 : 2;       // query tiles in flight
    static constexpr int CTAS = D == 256 ? 1 : 2;    // per SM
    static constexpr int OFF_Q = TILE, OFF_LSE = OFF_Q + NS * TILE;
    static constexpr int OFF_SUM = OFF_LSE + 2 * 4 * NG * TQ * 4;  // [softmax warp][2 parities][TQ]
    static constexpr int OFF_BAR = OFF_SUM + NG * TK * 4;      // [NG][TK]
    static constexpr int SMEM = 1024 + OFF_BAR + 256;
    static_assert(CTAS * (SMEM + 1024) <= 233472, "shared memory");
};
}  // namespace kwt

__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

template <int D>
__global__ void __launch_bounds__(kwt::NT, kwt::Cfg<D>::CTAS)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const KeyWeightParams p, const int cluster, const int box_rows) {
    using namespace kwt;
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_full = bars;
    uint64_t* full = bars + 1;
    uint64_t* empty = full + C::NS;
    uint64_t* s_ready = empty + C::NS;  // [NBUF]
    uint64_t* s_free = s_ready + NBUF;  // [NBUF]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_free + NBUF);
    __shared__ int s_abort;

    const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
    // key tiles are the slowest grid dimension: the causal half makes the first ones the longest, and they start first
    const int j0 = (int)blockIdx.z * TK, kvh = (int)blockIdx.x / cluster, b = blockIdx.y;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int L = clamp_len(p.lens, b, p.Lmax, p.s, p.causal, p.status, threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0);
    const size_t wrow = ((size_t)b * p.h_kv + kvh) * p.Lmax;
    if (j0 >= L) {  // the whole cluster: one key tile
        const int j = j0 + threadIdx.x;
        if (rank == 0 && threadIdx.x < TK && j < p.Lmax && !p.accumulate) p.w[wrow + j] = 0.f;
        return;
    }
    // the queries that see the tile's first key, head by head; this CTA's tiles are n = rank, rank + cluster, ...
    const int start = p.causal ? max(0, j0 - (L - p.s)) : 0;
    const int per = cdiv(p.s - start, TQ), total = p.ratio * per;
    const int n_mine = total > (int)rank ? (total - (int)rank + cluster - 1) / cluster : 0;

    if (threadIdx.x == 0) {
        s_abort = 0;
        mbar_init(smem_u32(k_full), 1);
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int i = 0; i < NBUF; ++i) {
            mbar_init(smem_u32(&s_ready[i]), 1);
            mbar_init(smem_u32(&s_free[i]), 4);
        }
        fence_barrier_init();
    }
    if (warp == W_LOAD) {
        tmem_alloc(tmem_slot, NBUF * TQ);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == W_LOAD) {
        if (lane == 0) {
            const uint32_t kb = smem_u32(k_full);
            mbar_arrive_expect_tx(kb, C::TILE);
            for (int r = 0; r < TK; r += box_rows) {
                const int tok = j0 + r;
                int y = tok, z = b * p.h_kv + kvh;
                if (p.table) {
                    int page = tok < L ? p.table[(size_t)b * p.max_pages + tok / p.page_size] : 0;
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(p.status, kDevBadPage);
                        page = 0;
                    }
                    y = tok % p.page_size;
                    z = page * p.h_kv + kvh;
                }
#pragma unroll
                for (int x = 0; x < C::NB; ++x)
                    tma_load_3d(smem_u32(smem + x * C::BOX + r * 128), &tm_k, x * 64, y, z, kb);
            }
            int issued = 0;
            bool ok = true;
            for (int i = 0; i < n_mine; ++i) {
                const int s = i % C::NS;
                if (*(volatile int*)&s_abort) break;
                if (i >= C::NS && !mbar_wait(smem_u32(&empty[s]), (i / C::NS - 1) & 1, p.status)) {
                    ok = false;
                    break;
                }
                const int n = (int)rank + i * cluster, head = n / per, t0 = start + n % per * TQ;
                const uint32_t fb = smem_u32(&full[s]);
                mbar_arrive_expect_tx(fb, C::TILE);
#pragma unroll
                for (int x = 0; x < C::NB; ++x)
                    tma_load_3d(smem_u32(smem + C::OFF_Q + s * C::TILE + x * C::BOX), &tm_q, x * 64, t0,
                                b * p.h_q + kvh * p.ratio + head, fb);
                ++issued;
            }
            if (!ok) s_abort = 1;
            for (int i = issued - 1; i >= 0 && i >= issued - C::NS; --i)
                mbar_wait(smem_u32(&full[i % C::NS]), (i / C::NS) & 1, p.status);
            mbar_wait(kb, 0, p.status);
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
            constexpr int B4 = C::BOX >> 4;
            const uint64_t kd = smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + C::OFF_Q), 16, 1024);
            bool ok = mbar_wait(smem_u32(k_full), 0, p.status);
            for (int i = 0; ok && i < n_mine; ++i) {
                const int s = i % C::NS, buf = i % NBUF;
                ok = mbar_wait(smem_u32(&full[s]), (i / C::NS) & 1, p.status);
                if (ok && i >= NBUF) ok = mbar_wait(smem_u32(&s_free[buf]), (i / NBUF - 1) & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t qd = q_desc + (uint64_t)(s * (C::TILE >> 4));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_ss(tmem + buf * 128, kd + (k / 4) * B4 + (k % 4) * 2, qd + (k / 4) * B4 + (k % 4) * 2, idesc, k != 0);
                umma_commit(smem_u32(&s_ready[buf]));
                // only where the loader waits for it: an arrival that nobody waits for may find the CTA's shared memory
                // in other hands
                if (i + C::NS < n_mine) umma_commit(smem_u32(&empty[s]));
            }
            if (!ok) s_abort = 1;
        }
    } else {
        const int grp = warp / 4, r = threadIdx.x % 128;  // the key's tensor-memory lane
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        float* ls = reinterpret_cast<float*>(smem + C::OFF_LSE) + warp * 2 * TQ;
        const size_t row0 = ((size_t)b * p.h_q + (size_t)kvh * p.ratio) * p.s;
        const int key = j0 + r;
        // Every warp stages the negated log2 normalisers of a tile's rows for itself, a tile ahead (one copy per group
        // needed a barrier per tile, whose skew cost a quarter of the time): -inf (nothing is added) past the head's
        // queries and for rows that saw no key.
        float next[TQ / 32];
        auto fetch = [&](int i) {
            const int n = (int)rank + i * cluster, head = n / per, t0 = start + (n - head * per) * TQ;
#pragma unroll
            for (int k = 0; k < TQ / 32; ++k) {
                const int t = t0 + 32 * k + lane;
                next[k] = INFINITY;
                if (i < n_mine && t < p.s) next[k] = p.lse[row0 + (size_t)head * p.s + t];
            }
        };
        fetch(grp);
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 sc = make_float2(p.scale_log2, p.scale_log2);
        // one score tile, 16 columns at a time; MASK: rows before `first` do not see the key, and rows without keys, whose
        // queries may be NaN, give nothing (elsewhere finite scores less the infinite normaliser do that)
        auto tile = [&](auto mask, uint32_t ts, const float* lb, int first, uint32_t release) {
            constexpr bool MASK = decltype(mask)::value;
            uint32_t sr[2][16];
            tmem_ld16(ts, sr[0]);
#pragma unroll
            for (int q = 0; q < TQ / 16; ++q) {
                tmem_ld_wait();
                if (q + 1 < TQ / 16) {
                    tmem_ld16(ts + 16 * (q + 1), sr[(q + 1) & 1]);
                } else {  // the last read of the buffer
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(release);
                }
                const uint32_t* x = sr[q & 1];
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const float4 l4 = *reinterpret_cast<const float4*>(lb + 16 * q + c);
                    const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc,
                                                 make_float2(l4.x, l4.y));
                    const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc,
                                                 make_float2(l4.z, l4.w));
                    float2 e0 = make_float2(fast_exp2(x0.x), fast_exp2(x0.y));
                    float2 e1 = make_float2(fast_exp2(x1.x), fast_exp2(x1.y));
                    if constexpr (MASK) {
                        if (16 * q + c < first || l4.x == -INFINITY) e0.x = 0.f;
                        if (16 * q + c + 1 < first || l4.y == -INFINITY) e0.y = 0.f;
                        if (16 * q + c + 2 < first || l4.z == -INFINITY) e1.x = 0.f;
                        if (16 * q + c + 3 < first || l4.w == -INFINITY) e1.y = 0.f;
                    }
                    acc[0] = __fadd2_rn(acc[0], e0);
                    acc[1] = __fadd2_rn(acc[1], e1);
                }
            }
        };
        bool ok = true;
        for (int i = grp, turn = 0; i < n_mine; i += NG, ++turn) {
            float* lb = ls + (turn & 1) * TQ;
#pragma unroll
            for (int k = 0; k < TQ / 32; ++k) lb[32 * k + lane] = next[k] == -INFINITY ? -INFINITY : -next[k] * kLog2e;
            const bool empty = __any_sync(0xffffffffu, fminf(fminf(next[0], next[1]), fminf(next[2], next[3])) == -INFINITY);
            static_assert(TQ / 32 == 4, "the rows above");
            fetch(i + NG);
            const int buf = i % NBUF;
            if (ok) ok = mbar_wait(smem_u32(&s_ready[buf]), (i / NBUF) & 1, p.status);
            tc_fence_after();
            const int n = (int)rank + i * cluster, t0 = start + n % per * TQ;
            const uint32_t ts = tmem + lanes + buf * 128, release = smem_u32(&s_free[buf]);
            // query t sees key j when j <= L - s + t: a tile whose first query sees the last key needs no mask
            if (empty || (p.causal && j0 + TK - 1 > L - p.s + t0))
                tile(std::true_type{}, ts, lb, p.causal ? key - (L - p.s) - t0 : 0, release);
            else
                tile(std::false_type{}, ts, lb, 0, release);
        }
        if (!ok) s_abort = 1;
        reinterpret_cast<float*>(smem + C::OFF_SUM)[grp * TK + r] = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_LOAD) tmem_dealloc(tmem, NBUF * TQ);
    if (cluster > 1) cluster_sync();
    if (rank == 0 && threadIdx.x < TK) {
        const int key = j0 + threadIdx.x;
        const uint32_t at = smem_u32(smem + C::OFF_SUM) + threadIdx.x * 4;
        float w = 0.f;
        for (int c = 0; c < cluster; ++c)
#pragma unroll
            for (int g = 0; g < NG; ++g)
                w += cluster > 1 ? cluster_load(at + g * TK * 4, c)
                                 : reinterpret_cast<const float*>(smem + C::OFF_SUM)[g * TK + threadIdx.x];
        if (key < L)
            p.w[wrow + key] = p.accumulate ? p.w[wrow + key] + w : w;
        else if (key < p.Lmax && !p.accumulate)
            p.w[wrow + key] = 0.f;
    }
    if (cluster > 1) cluster_sync();  // a CTA's shared memory outlives its readers
}

template <int D>
static lka_status_t key_weights_tc_run(const KeyWeightParams& p, cudaStream_t st) {
    using C = kwt::Cfg<D>;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tq, tk;
    const uint64_t row = D * 2;
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)p.s, (uint64_t)p.B * p.h_q}, qs[2] = {row, row * p.s};
    const uint32_t qb[3] = {64, kwt::TQ, 1};
    const int box_rows = p.table ? std::min(kwt::TK, p.page_size) : kwt::TK;
    const uint64_t rows = p.table ? p.page_size : p.Lmax;
    const uint64_t slabs = (uint64_t)(p.table ? p.num_pages : p.B) * p.h_kv;
    const uint64_t kd[3] = {(uint64_t)D, rows, slabs}, ks[2] = {row, row * rows};
    const uint32_t kb[3] = {64, (uint32_t)box_rows, 1};
    if (!make_tmap_nd(&tq, BF, p.q, 3, qd, qs, qb) || !make_tmap_nd(&tk, BF, p.k, 3, kd, ks, kb)) return LKA_ERR_CUDA;
    cudaError_t e = allow_smem<key_weights_tc_kernel<D>>(C::SMEM);
    if (e != cudaSuccess) return call_status(e);
    const int key_tiles = cdiv(p.Lmax, kwt::TK);
    if (key_tiles > 65535) return LKA_ERR_UNSUPPORTED;
    // clusters share a key tile's queries while the key tiles alone leave SMs idle, and while every CTA keeps at
    // least two query tiles
    const long long units = (long long)key_tiles * p.h_kv * p.B;
    const int q_tiles = p.ratio * cdiv(p.s, kwt::TQ);
    int cluster = 1;
    while (cluster < 8 && units * cluster * 2 <= 4LL * sm_count() && q_tiles >= 4 * cluster) cluster *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(p.h_kv * cluster, p.B, key_tiles);
    cfg.blockDim = dim3(kwt::NT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    TimedLaunch timer(st);
    e = cudaLaunchKernelEx(&cfg, key_weights_tc_kernel<D>, tq, tk, p, cluster, box_rows);
    timer.stop();
    return call_status(e);
}

lka_status_t key_weights_tc(const KeyWeightParams& p, int d, cudaStream_t st) {
    return d == 64 ? key_weights_tc_run<64>(p, st) : d == 128 ? key_weights_tc_run<128>(p, st) : key_weights_tc_run<256>(p, st);
}

}  // namespace lka
