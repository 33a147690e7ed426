// prefix_tc.cu -- the shared prefix of gqa_attn_shared_prefix on the 5th-generation
// tensor cores (bf16, d = 64 and 128): flash attention whose rows are the query rows of
// all sequences that use one KV head.
//
// One CTA takes two tiles of up to 128 query rows of one KV head and a range of the
// prefix's keys, in tiles of 128 keys; the two row tiles share every K and V tile.  Warp 8
// streams K and V with TMA through one ring; warp 9 issues the MMAs, per key tile j and row
// tile i: O_i += P_i(j) V_j, then S_i(j + 1) = Q_i K_{j+1}^T; warps 0-3 and 4-7 are the
// softmax of row tile 0 and 1, one thread per row.  While one row tile is in its softmax,
// the tensor pipe works for the other.  P_i overwrites S_i in tensor memory: the MMAs run in
// the order they are issued, so S_i(j + 1) follows the P V product that reads P_i(j), and
// s_ready(j + 1) also tells that O_i holds tile j, which makes rescaling O_i safe then.  P is
// handed over in quarters of 32 keys, so that P V starts on the first while the next is
// still in its exponentials.
//
// Bound: 2 x 128 x 128 x 4 d FLOPs per key tile pair at d = 128 are 2080 tensor cycles; its
// 32,768 exponentials are 2048 cycles of the special-function unit (16 per cycle and SM), so
// both pipes are full together.  Below about 256 rows per KV head the prefix's bytes bound.
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "launch_util.h"
#include "prefix_attn.h"
#include "tc.cuh"

namespace lka {

namespace ptc {
constexpr int TK = 128, NT = 320;
template <int D>
struct Cfg {
    static constexpr int NB = D / 64;            // 64-column boxes of a row
    static constexpr int BOX = 128 * 128;        // 128 rows of 128 bytes
    static constexpr int TILE = NB * BOX;
    static constexpr int NS = D == 128 ? 5 : 8;  // ring stages, each a K or a V tile
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_BAR = OFF_RING + NS * TILE;
    static constexpr int SMEM = 1024 + OFF_BAR + 256;
    static constexpr uint32_t T_O = 0, T_S = 2 * D;  // tensor memory columns: O_0, O_1, then S_0, S_1 (128 each)
    static constexpr uint32_t T_COLS = 512;
    static_assert(2 * D + 256 <= 512 && SMEM <= 232448, "budgets");
};
}  // namespace ptc

template <int D>
__global__ void __launch_bounds__(ptc::NT, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PrefixParams p, const PrefixTiles g) {
    using namespace ptc;
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* q_full = bars;
    uint64_t* full = bars + 1;
    uint64_t* empty = full + C::NS;
    uint64_t* s_ready = empty + C::NS;  // [2]
    uint64_t* p_ready = s_ready + 2;    // [2][4]: row tile, quarter of the keys
    uint64_t* o_done = p_ready + 8;     // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_done + 2);
    __shared__ int s_abort;

    const int pairs = cdiv(g.n_tiles, 2);
    const int pair = blockIdx.x % pairs, split = (blockIdx.x / pairs) % p.n_pre, kvh = blockIdx.x / (pairs * p.n_pre);
    const int n_qt = min(2, g.n_tiles - 2 * pair);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int P = prefix_length(p, threadIdx.x == 0 && blockIdx.x == 0);
    const int kbeg = split * p.pre_tokens, kend = min(P, kbeg + p.pre_tokens);
    if (kend <= kbeg) return;
    const int n_kt = cdiv(kend - kbeg, TK);

    if (threadIdx.x == 0) {
        s_abort = 0;
        mbar_init(smem_u32(q_full), 1);
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s_ready[i]), 1);
            for (int h = 0; h < 4; ++h) mbar_init(smem_u32(&p_ready[4 * i + h]), 4);
            mbar_init(smem_u32(&o_done[i]), 1);
        }
        fence_barrier_init();
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, C::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 8) {
        // ------------------------------ producer: Q, then K_0, V_0, K_1, V_1, ... ------------------------------
        if (lane == 0) {
            const uint32_t qb = smem_u32(q_full);
            mbar_arrive_expect_tx(qb, n_qt * C::NB * g.rows * 128);
            for (int i = 0; i < n_qt; ++i) {
                const int t = 2 * pair + i;
                const int b0 = g.per_seq > 1 ? t / g.per_seq : t * g.seqs, g0 = g.per_seq > 1 ? t % g.per_seq * g.rows : 0;
#pragma unroll
                for (int x = 0; x < C::NB; ++x)
                    tma_load_4d(smem_u32(smem + i * C::TILE + x * C::BOX), &tm_q, x * 64, g0, kvh, b0, qb);
            }
            bool ok = true;
            int issued = 0;
            for (int n = 0; n < 2 * n_kt; ++n) {
                const int s = n % C::NS;
                if (*(volatile int*)&s_abort) break;
                if (n >= C::NS && !mbar_wait(smem_u32(&empty[s]), (n / C::NS - 1) & 1, p.status)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + C::OFF_RING + s * C::TILE);
                mbar_arrive_expect_tx(fb, C::TILE);
                const CUtensorMap* map = n & 1 ? &tm_v : &tm_k;
                for (int r = 0; r < TK; r += g.box_rows) {
                    const int tok = kbeg + n / 2 * TK + r;
                    int y = tok, z = kvh;
                    if (p.ptable) {
                        // pages [num_pages][h_kv][page_size]; rows past the keys of this split are not looked up
                        int page = tok < kend ? p.ptable[tok / p.page_size] : 0;
                        if (page < 0 || page >= p.num_pages) {
                            atomicOr(p.status, kDevBadPage);
                            page = 0;
                        }
                        y = tok % p.page_size;
                        z = page * p.h_kv + kvh;
                    }
#pragma unroll
                    for (int x = 0; x < C::NB; ++x) tma_load_3d(dst + x * C::BOX + r * 128, map, x * 64, y, z, fb);
                }
                ++issued;
            }
            if (!ok) s_abort = 1;
            // every issued copy lands before the CTA may end
            for (int n = issued - 1; n >= 0 && n >= issued - C::NS; --n)
                mbar_wait(smem_u32(&full[n % C::NS]), (n / C::NS) & 1, p.status);
            mbar_wait(qb, 0, p.status);
        }
    } else if (warp == 9) {
        // ------------------------------ MMA issuer ------------------------------
        constexpr uint32_t id_qk = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_pv = idesc_bf16_f32(128, D, false, true);
        bool ok = mbar_wait(smem_u32(q_full), 0, p.status);
        auto stage = [&](int n) { return smem + C::OFF_RING + (n % C::NS) * C::TILE; };
        auto wait_full = [&](int n) { return mbar_wait(smem_u32(&full[n % C::NS]), (n / C::NS) & 1, p.status); };
        auto scores = [&](int i, int j) {  // S_i(j)
            if (lane == 0) {
                const uint32_t qa = smem_u32(smem + i * C::TILE), ka = smem_u32(stage(2 * j));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_ss(tmem + C::T_S + i * 128, smem_desc_sw128(qa + (k / 4) * C::BOX + (k % 4) * 32, 16, 1024),
                            smem_desc_sw128(ka + (k / 4) * C::BOX + (k % 4) * 32, 16, 1024), id_qk, k != 0);
                umma_commit(smem_u32(&s_ready[i]));
                if (i == n_qt - 1) umma_commit(smem_u32(&empty[(2 * j) % C::NS]));
            }
            __syncwarp();
        };
        if (ok) ok = wait_full(0);
        if (ok) {
            tc_fence_after();
            for (int i = 0; i < n_qt; ++i) scores(i, 0);
        }
        for (int j = 0; ok && j < n_kt; ++j) {
            ok = wait_full(2 * j + 1);
            if (!ok) break;
            const int valid = kend - (kbeg + j * TK);
            if (valid < TK) {
                // value rows past the keys may hold anything; 0 x NaN would reach every row
                uint8_t* v = stage(2 * j + 1);
                const int rows = TK - valid;
                for (int x = lane; x < C::NB * rows * 8; x += 32)
                    *reinterpret_cast<uint4*>(v + x / (rows * 8) * C::BOX + (valid + x / 8 % rows) * 128 + x % 8 * 16) =
                        make_uint4(0, 0, 0, 0);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            for (int i = 0; ok && i < n_qt; ++i) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    if (!mbar_wait(smem_u32(&p_ready[4 * i + h]), j & 1, p.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t va = smem_u32(stage(2 * j + 1));
#pragma unroll
                        for (int k = 2 * h; k < 2 * h + 2; ++k)
                            umma_ts(tmem + C::T_O + i * D, tmem + C::T_S + i * 128 + k * 8,
                                    smem_desc_sw128(va + k * 2048, C::BOX, 1024), id_pv, (j | k) != 0);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) {
                    if (i == n_qt - 1) umma_commit(smem_u32(&empty[(2 * j + 1) % C::NS]));
                    if (j == n_kt - 1) umma_commit(smem_u32(&o_done[i]));
                }
                __syncwarp();
                if (j + 1 < n_kt) {
                    if (i == 0 && !wait_full(2 * (j + 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    scores(i, j + 1);
                }
            }
        }
        if (!ok) s_abort = 1;
    } else if (warp / 4 < n_qt) {
        // ------------------------------ softmax: one thread per query row ------------------------------
        const int i = warp / 4, r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t ts = tmem + lanes + C::T_S + i * 128, to = tmem + lanes + C::T_O + i * D;
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        bool ok = true;
        for (int j = 0; j < n_kt; ++j) {
            if (ok) ok = mbar_wait(smem_u32(&s_ready[i]), j & 1, p.status);
            tc_fence_after();
            uint32_t sr[TK];
#pragma unroll
            for (int c = 0; c < TK; c += 16) tmem_ld16(ts + c, sr + c);
            tmem_ld_wait();
            float* f = reinterpret_cast<float*>(sr);
            float mul = p.scale_log2;
            const int valid = kend - (kbeg + j * TK);
            if (valid < TK) {
#pragma unroll
                for (int c = 0; c < TK; ++c) f[c] = c < valid ? f[c] * mul : -INFINITY;
                mul = 1.f;
            }
            const float2 mul2 = make_float2(mul, mul);
            // a quarter of the row: 32 probabilities against the reference maximum `ref`, as bf16 pairs, and their sum
            uint32_t pk[16];
            float2 part;
            auto quarter = [&](int c0, float ref) {
                const float2 neg2 = make_float2(-ref, -ref);
                float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 x = __ffma2_rn(make_float2(f[c0 + c], f[c0 + c + 1]), mul2, neg2);
                    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    s2[(c / 2) & 1] = __fadd2_rn(s2[(c / 2) & 1], e);
                    pk[c / 2] = pack_bf16x2(e.x, e.y);
                }
                part = __fadd2_rn(s2[0], s2[1]);
            };
            // The reference moves only when a score exceeds it by 2^8, which is rare after the first tile: the first
            // quarter is computed against the old one while the maximum is still being found.
            quarter(0, m == -INFINITY ? 0.f : m);
            float mx;
            if (mul >= 0.f) {
                float a[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) a[c] = f[c];
#pragma unroll
                for (int c = 4; c < TK; ++c) a[c % 4] = fmaxf(a[c % 4], f[c]);
                mx = tree_max<4>(a) * mul;
            } else {
                float a = f[0];
#pragma unroll
                for (int c = 1; c < TK; ++c) a = fminf(a, f[c]);
                mx = a * mul;
            }
            const bool grow = m == -INFINITY || mx > m + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
                const float to_m = grow ? mx : m;
                const float alpha = m == -INFINITY || to_m == m ? 1.f : fast_exp2(m - to_m);
                m = to_m;
                l2.x *= alpha;
                l2.y *= alpha;
                if (j > 0) {  // s_ready also says that O holds the tiles before this one
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(to + c, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(to + c, o);
                    }
                }
                quarter(0, m == -INFINITY ? 0.f : m);
            }
            const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (h) quarter(32 * h, ms);
                l2 = __fadd2_rn(l2, part);
                tmem_st16(ts + 16 * h, pk);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&p_ready[4 * i + h]));
            }
        }
        if (ok) ok = mbar_wait(smem_u32(&o_done[i]), 0, p.status);
        if (!ok) s_abort = 1;
        tc_fence_after();
        const int t = 2 * pair + i;
        const int b = g.per_seq > 1 ? t / g.per_seq : t * g.seqs + r / p.R, gr = g.per_seq > 1 ? t % g.per_seq * g.rows + r : r % p.R;
        const bool mine = ok && r < g.rows && b < p.B && gr < p.R;
        const size_t at = mine ? (((size_t)b * p.h_kv + kvh) * p.R + gr) * p.n_slots + split : 0;
        const float l = l2.x + l2.y, inv = l > 0.f ? 1.f / l : 0.f;
        float* po = p.part_o + at * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_ld_wait();
            if (mine) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4*>(po + c + e) =
                        make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                                    __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
            }
        }
        if (mine) p.part_lse[at] = l > 0.f ? m + log2f(l) : -INFINITY;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) tmem_dealloc(tmem, C::T_COLS);
}

PrefixTiles prefix_tiles(int B, int R) {
    PrefixTiles g{};
    g.seqs = std::max(1, 128 / R);
    g.per_seq = cdiv(R, 128);
    g.rows = g.per_seq > 1 ? 128 : g.seqs * R;
    g.n_tiles = g.per_seq > 1 ? B * g.per_seq : cdiv(B, g.seqs);
    return g;
}

template <int D>
static lka_status_t prefix_tc_run(const PrefixParams& p, cudaStream_t st) {
    using C = ptc::Cfg<D>;
    PrefixTiles g = prefix_tiles(p.B, p.R);
    g.box_rows = p.ptable ? std::min(ptc::TK, p.page_size) : ptc::TK;
    const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tq, tk, tv;
    const uint64_t row = D * 2;
    const uint64_t qd[4] = {(uint64_t)D, (uint64_t)p.R, (uint64_t)p.h_kv, (uint64_t)p.B};
    const uint64_t qs[3] = {row, row * p.R, row * p.R * p.h_kv};
    const uint32_t qb[4] = {64, (uint32_t)std::min(p.R, 128), 1, (uint32_t)(g.per_seq > 1 ? 1 : g.seqs)};
    // contiguous: [h_kv][Lp][D]; pages: [num_pages * h_kv][page_size][D]
    const uint64_t rows = p.ptable ? p.page_size : p.Lp, slabs = p.ptable ? (uint64_t)p.num_pages * p.h_kv : p.h_kv;
    const uint64_t kd[3] = {(uint64_t)D, rows, slabs};
    const uint64_t ks[2] = {row, row * rows};
    const uint32_t kb[3] = {64, (uint32_t)g.box_rows, 1};
    if (!make_tmap_nd(&tq, BF, p.q, 4, qd, qs, qb) || !make_tmap_nd(&tk, BF, p.kp, 3, kd, ks, kb) ||
        !make_tmap_nd(&tv, BF, p.vp, 3, kd, ks, kb))
        return LKA_ERR_CUDA;
    if (allow_smem<prefix_tc_kernel<D>>(C::SMEM) != cudaSuccess) return LKA_ERR_CUDA;
    const long long n = (long long)cdiv(g.n_tiles, 2) * p.n_pre * p.h_kv;
    if (n >= (1ll << 31)) return LKA_ERR_UNSUPPORTED;
    TimedLaunch timer(st);
    prefix_tc_kernel<D><<<(unsigned)n, ptc::NT, C::SMEM, st>>>(tq, tk, tv, p, g);
    timer.stop();
    return cudaPeekAtLastError() == cudaSuccess ? LKA_OK : LKA_ERR_CUDA;
}

lka_status_t prefix_tc(const PrefixParams& p, int d, cudaStream_t st) {
    return d == 64 ? prefix_tc_run<64>(p, st) : prefix_tc_run<128>(p, st);
}

}  // namespace lka
