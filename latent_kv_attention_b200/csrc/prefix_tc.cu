// prefix_tc.cu -- the shared prefix of gqa_attn_shared_prefix on the 5th-generation
// tensor cores (bf16, d = 64 and 128): flash attention whose rows are the query rows of
// all sequences that use one KV head.
//
// One CTA takes two tiles of up to 128 query rows of one KV head and a range of the
// prefix's keys; the two row tiles share every K and V tile of 128 keys, which warp 8 streams
// with TMA through one ring.  Scores are made 64 keys at a time into two buffers per row tile:
// warps 0-3 and 4-7 are the softmax of row tile 0 and 1, one thread per row, and find the next
// block of scores made while they work on this one.  P_i(n), in bf16, overwrites S_i(n) in
// tensor memory.  Four threads issue the MMAs, two per row tile (scores; values), each waiting
// only for what its product needs, so that one's waits (about 200 cycles each) pass under the
// others' MMAs; the tensor core's reads of P_i(n) and writes of S_i(n + 2) are ordered by a commit.
//
// Bound: per 128 keys the 2 x 128 x 128 x 4 d FLOPs take 2640 tensor cycles at d = 128 (2080
// at the full rate; an N = 64 MMA costs 50 cycles, not 32) and 32,768 exponentials 2048 cycles
// of the special-function unit (16 per cycle and SM).  Measured on 256 sequences of 2 queries,
// 32 / 8 heads of 128, a paged prefix of 16,384 keys (137 GFLOP): 121-132 us, 0.61-0.66 of the
// measured dense rate.  Steps to it: one score buffer of 128 keys per row tile and one issuing
// thread 193 us (score product, softmax, value product in series); 64-key blocks 171; four issuing
// threads 176 but ordered; the row tiles taking turns at the exponentials 175; one lane per TMA
// box with its page looked up early 132 (one lane alone took 1500 cycles per tile); loads before
// the block meets and outputs through shared memory 121 at best.
//
// Rounding: P goes to bf16, the type of V, because both operands of one product have the same type
// (the sums are of the fp32 values).  That alone is 0.0016 of a result's size, as much as the
// result's own rounding to bf16: 0.0023 together against 0.0017 with an fp32 P (64 sequences over
// 8192 keys), the same in every bit from call to call.
#include <math.h>

#include <algorithm>

#include "host_util.h"
#include "launch_util.h"
#include "prefix_attn.h"
#include "tc.cuh"

namespace lka {

namespace ptc {
constexpr int TK = 128, TB = 64;  // keys per K / V tile, per block of scores
constexpr int W_LOAD = 8, W_MMA = 9, NT = 416;  // warps 0-3 and 4-7: softmax; 8: loads; 9 + 2i, 10 + 2i: scores, values
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

__device__ __forceinline__ void named_barrier_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

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
    uint64_t* s_ready = empty + C::NS;  // [2][2]: row tile, score buffer
    uint64_t* p_ready = s_ready + 4;    // [2][2]
    uint64_t* o_ready = p_ready + 4;    // [2][2]: the block of that buffer is in O
    uint64_t* o_done = o_ready + 4;     // [2]
    uint64_t* v_tail = o_done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_tail + 1);
    __shared__ int s_abort;

    const int pairs = cdiv(g.n_tiles, 2);
    const int pair = blockIdx.x % pairs, split = (blockIdx.x / pairs) % p.n_pre, kvh = blockIdx.x / (pairs * p.n_pre);
    const int n_qt = min(2, g.n_tiles - 2 * pair);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int P = prefix_length(p, threadIdx.x == 0 && blockIdx.x == 0);
    pdl_trigger();  // the suffix kernel needs nothing of this one
    const int kbeg = split * p.pre_tokens, kend = min(P, kbeg + p.pre_tokens);
    if (kend <= kbeg) return;
    const int n_kt = cdiv(kend - kbeg, TK), nb = cdiv(kend - kbeg, TB);  // tiles of keys, blocks of scores

    // The loader sets up the barriers and issues what needs no waiting before the block meets: Q, then K_0, V_0, K_1, ...
    // as far as the ring goes.  One lane per box of a tile (a tile is one box, or one per page piece); the rows of tile
    // j + 1 are looked up while its ring stage is still in use, once for its keys and values.
    const uint32_t qb = smem_u32(q_full);
    const int box_r = lane * g.box_rows;
    int y = 0, z = kvh, issued = 0;
    auto look_up = [&](int j) {
        const int tok = kbeg + j * TK + box_r;
        if (box_r >= TK) return;
        y = tok;
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
    };
    auto issue_tile = [&]() {
        const int s = issued % C::NS;
        const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + C::OFF_RING + s * C::TILE) + box_r * 128;
        if (lane == 0) mbar_arrive_expect_tx(fb, C::TILE);
        __syncwarp();
        if (box_r < TK) {
            const CUtensorMap* map = issued & 1 ? &tm_v : &tm_k;
#pragma unroll
            for (int x = 0; x < C::NB; ++x) tma_load_3d(dst + x * C::BOX, map, x * 64, y, z, fb);
        }
        if (issued & 1) look_up(issued / 2 + 1);
        ++issued;
    };
    if (warp == W_LOAD) {
        if (lane == 0) {
            s_abort = 0;
            mbar_init(smem_u32(q_full), 1);
            for (int s = 0; s < C::NS; ++s) {
                mbar_init(smem_u32(&full[s]), 1);
                mbar_init(smem_u32(&empty[s]), n_qt);
            }
            for (int i = 0; i < 2; ++i) {
                for (int h = 0; h < 2; ++h) {
                    mbar_init(smem_u32(&s_ready[2 * i + h]), 1);
                    mbar_init(smem_u32(&p_ready[2 * i + h]), 4);
                    mbar_init(smem_u32(&o_ready[2 * i + h]), 1);
                }
                mbar_init(smem_u32(&o_done[i]), 1);
            }
            mbar_init(smem_u32(v_tail), 1);
            fence_barrier_init();
            mbar_arrive_expect_tx(qb, n_qt * C::NB * g.rows * 128);
            for (int i = 0; i < n_qt; ++i) {
                const int t = 2 * pair + i;
                const int b0 = g.per_seq > 1 ? t / g.per_seq : t * g.seqs, g0 = g.per_seq > 1 ? t % g.per_seq * g.rows : 0;
#pragma unroll
                for (int x = 0; x < C::NB; ++x)
                    tma_load_4d(smem_u32(smem + i * C::TILE + x * C::BOX), &tm_q, x * 64, g0, kvh, b0, qb);
            }
        }
        __syncwarp();
        look_up(0);
        while (issued < min(C::NS, 2 * n_kt)) issue_tile();
    } else if (warp == W_MMA) {
        tmem_alloc(tmem_slot, C::T_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == W_LOAD) {
        // ------------------------------ loader ------------------------------
        bool ok = true;
        while (issued < 2 * n_kt) {
            ok = mbar_wait(smem_u32(&empty[issued % C::NS]), (issued / C::NS - 1) & 1, p.status);
            if (!__all_sync(0xffffffffu, ok && !*(volatile int*)&s_abort)) break;
            issue_tile();
        }
        if (!ok) s_abort = 1;
        // every issued copy lands before the CTA may end
        for (int n = issued - 1; n >= 0 && n >= issued - C::NS; --n)
            mbar_wait(smem_u32(&full[n % C::NS]), (n / C::NS) & 1, p.status);
        mbar_wait(qb, 0, p.status);
        const int n = 2 * n_kt - 1, valid = kend - (kbeg + n / 2 * TK);
        if (valid < TK && issued == 2 * n_kt) {
            // the last tile's value rows past the keys may hold anything, and 0 x NaN would reach every row: zeros
            uint8_t* v = smem + C::OFF_RING + n % C::NS * C::TILE;
            const int rows = TK - valid;
            for (int x = lane; x < C::NB * rows * 8; x += 32)
                *reinterpret_cast<uint4*>(v + x / (rows * 8) * C::BOX + (valid + x / 8 % rows) * 128 + x % 8 * 16) =
                    make_uint4(0, 0, 0, 0);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(v_tail));
        }
    } else if (warp >= W_MMA && warp < W_MMA + 2 * n_qt) {
        // ------------------------------ MMA issuers ------------------------------
        // Every commit's arrival is waited for before the CTA ends (one that nobody waits for may find its shared memory
        // in other hands): stages are released only where the loader fills them again, the last product is o_done's.
        const int i = (warp - W_MMA) / 2;
        constexpr int B4 = C::BOX >> 4, T4 = C::TILE >> 4, H4 = TB * 128 >> 4;
        const uint32_t ts = tmem + C::T_S + 2 * i * TB, to = tmem + C::T_O + i * D;
        if (lane == 0 && (warp - W_MMA) % 2 == 0) {  // S_i(n) = Q_i K_n^T
            constexpr uint32_t idesc = idesc_bf16_f32(128, TB, false, false);
            const uint64_t qd = smem_desc_sw128(smem_u32(smem + i * C::TILE), 16, 1024);
            const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + C::OFF_RING), 16, 1024);
            bool ok = mbar_wait(smem_u32(q_full), 0, p.status);
            for (int n = 0, st = 0, ph = 0; ok && n < nb; ++n) {
                if (!(n & 1)) ok = mbar_wait(smem_u32(&full[st]), ph, p.status);
                // the buffer's P has been read
                if (ok && n >= 2) ok = mbar_wait(smem_u32(&o_ready[2 * i + (n & 1)]), ((n >> 1) - 1) & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kd = k_desc + (uint64_t)(st * T4 + (n & 1) * H4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_ss(ts + (n & 1) * TB, qd + (k / 4) * B4 + (k % 4) * 2, kd + (k / 4) * B4 + (k % 4) * 2, idesc,
                            k != 0);
                umma_commit(smem_u32(&s_ready[2 * i + (n & 1)]));
                if ((n & 1) || n == nb - 1) {
                    // (K tile n / 2 is copy 2 (n / 2) of the ring)
                    if ((n & ~1) + C::NS < 2 * n_kt) umma_commit(smem_u32(&empty[st]));
                    st += 2;
                    if (st >= C::NS) {
                        st -= C::NS;
                        ph ^= 1;
                    }
                }
            }
            // the last product but one, for which no later block waits
            if (ok && nb > 1) ok = mbar_wait(smem_u32(&o_ready[2 * i + (nb & 1)]), ((nb - 2) >> 1) & 1, p.status);
            if (!ok) s_abort = 1;
        } else if (lane == 0) {  // O_i += P_i(n) V_n
            constexpr uint32_t idesc = idesc_bf16_f32(128, D, false, true);
            const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + C::OFF_RING), C::BOX, 1024);
            bool ok = true;
            for (int n = 0, st = 1, ph = 0; ok && n < nb; ++n) {
                if (!(n & 1)) {
                    ok = mbar_wait(smem_u32(&full[st]), ph, p.status);
                    if (ok && kend - (kbeg + n * TB) < TK) ok = mbar_wait(smem_u32(v_tail), 0, p.status);
                }
                if (ok) ok = mbar_wait(smem_u32(&p_ready[2 * i + (n & 1)]), (n >> 1) & 1, p.status);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = v_desc + (uint64_t)(st * T4 + (n & 1) * H4);
#pragma unroll
                for (int k = 0; k < TB / 16; ++k)
                    umma_ts(to, ts + (n & 1) * TB + k * 8, vd + k * (2048 >> 4), idesc, (n | k) != 0);
                umma_commit(smem_u32(n == nb - 1 ? &o_done[i] : &o_ready[2 * i + (n & 1)]));
                if ((n & 1) || n == nb - 1) {
                    if ((n & ~1) + 1 + C::NS < 2 * n_kt) umma_commit(smem_u32(&empty[st]));
                    st += 2;
                    if (st >= C::NS) {
                        st -= C::NS;
                        ph ^= 1;
                    }
                }
            }
            if (!ok) s_abort = 1;
        }
    } else if (warp / 4 < n_qt) {
        // ------------------------------ softmax: one thread per query row ------------------------------
        const int i = warp / 4, r = (warp % 4) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
        const uint32_t to = tmem + lanes + C::T_O + i * D;
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        bool ok = true;
        // The two warps of an SM sub-partition (one of each row tile) take turns at the exponentials: left alone they
        // fall into step, contend for the special-function unit and then leave it idle together.
        const int bar_mine = 1 + 2 * (warp % 4) + i, bar_other = 1 + 2 * (warp % 4) + (i ^ 1);
        if (n_qt == 2 && i == 1) named_barrier_arrive(bar_other, 64);  // row tile 0 goes first
        for (int n = 0; n < nb; ++n) {
            const uint32_t ts = tmem + lanes + C::T_S + (2 * i + (n & 1)) * TB;
            if (ok) ok = mbar_wait(smem_u32(&s_ready[2 * i + (n & 1)]), (n >> 1) & 1, p.status);
            tc_fence_after();
            uint32_t sr[TB];
#pragma unroll
            for (int c = 0; c < TB; c += 16) tmem_ld16(ts + c, sr + c);
            tmem_ld_wait();
            float* f = reinterpret_cast<float*>(sr);
            float mul = p.scale_log2;
            const int valid = kend - (kbeg + n * TB);
            if (valid < TB) {
#pragma unroll
                for (int c = 0; c < TB; ++c) f[c] = c < valid ? f[c] * mul : -INFINITY;
                mul = 1.f;
            }
            float mx;
            if (mul >= 0.f) {
                float a[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) a[c] = f[c];
#pragma unroll
                for (int c = 4; c < TB; ++c) a[c % 4] = fmaxf(a[c % 4], f[c]);
                mx = tree_max<4>(a) * mul;
            } else {
                float a = f[0];
#pragma unroll
                for (int c = 1; c < TB; ++c) a = fminf(a, f[c]);
                mx = a * mul;
            }
            // the reference maximum moves only when a score exceeds it by 2^8: rarely after the first block
            const bool grow = m == -INFINITY || mx > m + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
                const float to_m = grow ? mx : m;
                const float alpha = m == -INFINITY || to_m == m ? 1.f : fast_exp2(m - to_m);
                m = to_m;
                l2.x *= alpha;
                l2.y *= alpha;
                if (n > 0) {
                    // O has to hold block n - 1 (block n waits for this warp, and n - 2 was in before S(n))
                    if (ok) ok = mbar_wait(smem_u32(&o_ready[2 * i + ((n - 1) & 1)]), ((n - 1) >> 1) & 1, p.status);
                    tc_fence_after();
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
            }
            if (n_qt == 2) named_barrier(bar_mine, 64);
            const float ms = m == -INFINITY ? 0.f : m;
            const float2 mul2 = make_float2(mul, mul), neg2 = make_float2(-ms, -ms);
            float2 part[2] = {l2, make_float2(0.f, 0.f)};
#pragma unroll
            for (int h = 0; h < TB / 32; ++h) {
                uint32_t pk[16];
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 x = __ffma2_rn(make_float2(f[32 * h + c], f[32 * h + c + 1]), mul2, neg2);
                    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    part[(c / 2) & 1] = __fadd2_rn(part[(c / 2) & 1], e);
                    pk[c / 2] = pack_bf16x2(e.x, e.y);
                }
                tmem_st16(ts + 16 * h, pk);
            }
            l2 = __fadd2_rn(part[0], part[1]);
            if (n_qt == 2 && (i == 0 || n + 1 < nb)) named_barrier_arrive(bar_other, 64);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&p_ready[2 * i + (n & 1)]));
        }
        if (ok) ok = mbar_wait(smem_u32(&o_done[i]), 0, p.status);
        if (!ok) s_abort = 1;
        tc_fence_after();
        const int t = 2 * pair + i;
        const int b = g.per_seq > 1 ? t / g.per_seq : t * g.seqs + r / p.R, gr = g.per_seq > 1 ? t % g.per_seq * g.rows + r : r % p.R;
        const bool mine = ok && r < g.rows && b < p.B && gr < p.R;
        const long long at = mine ? (long long)((((size_t)b * p.h_kv + kvh) * p.R + gr) * p.n_slots + split) : -1;
        const float l = l2.x + l2.y, inv = part_inverse(l);
        if (mine) p.part_lse[at] = part_normaliser(m, l);
        // O leaves through this warp's quarter of the row tile's query buffer (its products are done), half of the
        // columns at a time: rows written by their lanes in 16-byte chunks, permuted over the banks, and read back row
        // by row (a lane writing its own row of the result touches 32 rows per instruction: 12,000 cycles per CTA)
        constexpr int NC = D / 8;  // chunks of half a row
        uint8_t* buf = smem + i * C::TILE + (warp % 4) * (32 * NC * 16);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t o[16];
                tmem_ld16(to + half * (D / 2) + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float4*>(buf + lane * (NC * 16) + (((c / 4 + e) ^ (lane % NC)) * 16)) =
                        make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                    __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
            }
            __syncwarp();
#pragma unroll 4
            for (int r0 = 0; r0 < 32; r0 += 32 / NC) {
                const int rr = r0 + lane / NC, c = lane % NC;
                const long long to_row = __shfl_sync(0xffffffffu, at, rr);
                const float4 v = *reinterpret_cast<const float4*>(buf + rr * (NC * 16) + ((c ^ (rr % NC)) * 16));
                if (to_row >= 0) *reinterpret_cast<float4*>(p.part_o + to_row * D + half * (D / 2) + c * 4) = v;
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) tmem_dealloc(tmem, C::T_COLS);
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
    const cudaError_t e = allow_smem<prefix_tc_kernel<D>>(C::SMEM);
    if (e != cudaSuccess) return call_status(e);
    const long long n = (long long)cdiv(g.n_tiles, 2) * p.n_pre * p.h_kv;
    if (n >= (1ll << 31)) return LKA_ERR_UNSUPPORTED;
    TimedLaunch timer(st);
    prefix_tc_kernel<D><<<(unsigned)n, ptc::NT, C::SMEM, st>>>(tq, tk, tv, p, g);
    timer.stop();
    return call_status(cudaPeekAtLastError());
}

lka_status_t prefix_tc(const PrefixParams& p, int d, cudaStream_t st) {
    return d == 64 ? prefix_tc_run<64>(p, st) : prefix_tc_run<128>(p, st);
}

}  // namespace lka
