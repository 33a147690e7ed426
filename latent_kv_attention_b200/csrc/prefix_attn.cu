// prefix_attn.cu -- grouped-query attention of a batch that shares one cached prefix
// (gqa_attn_shared_prefix, gqa_attn_shared_prefix_paged).
//
// Operation: every sequence attends over the keys of one prefix (length P, held once) and
// over its own suffix (bottom-right causal, as gqa_attn).  Softmax over the union splits:
//     out = sum_i 2^(m_i - m) l_i o_i / sum_i 2^(m_i - m) l_i
// over parts i of the keys, with each part's maximum m_i, sum l_i and normalised o_i.  The
// prefix parts are computed once for the whole batch: the query rows of all sequences that
// use one KV head are the rows of one matrix product, so the prefix is read once per 16 to
// 128 rows instead of once per sequence.
//
// Every part writes a normalised fp32 output and a log2-domain lse per row;
// prefix_merge_kernel joins them and rounds once.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "host_util.h"
#include "launch_util.h"
#include "mma.cuh"
#include "prefix_attn.h"
#include "tc.cuh"

namespace lka {

namespace {

constexpr int kMaxSplits = 64, kMaxSlots = 2 * kMaxSplits;  // splits of the prefix and of a suffix at most, and both

// ---- what a block works on ---------------------------------------------------------------------------------
// Prefix: rows are the B * R query rows of a KV head (row i: sequence i / R, row i % R of its group).
// Suffix: rows are the R rows of one sequence's group.  R = (h_q / h_kv) * s_q, row g is query g % s_q.
struct Work {
    bool prefix;
    int kvh, b;        // b: the sequence of a suffix item
    int row0, nrows;   // rows of the item (its row numbering), at most the block's rows
    int kbeg, kend;    // keys
    int slot;          // of the partial results
    int L;             // length of the key sequence
};

// Items of a launch, and item `idx` of them; false: nothing to do.
__host__ __device__ inline long long count_work(const PrefixParams& p, int rows_per_block) {
    return (p.do_prefix ? (long long)cdiv(p.B * p.R, rows_per_block) * p.h_kv * p.n_pre : 0) +
           (p.do_suffix ? (long long)p.B * p.h_kv * cdiv(p.R, rows_per_block) * p.n_suf : 0);
}
__device__ __forceinline__ bool find_work(const PrefixParams& p, int rows_per_block, int idx, Work& w, bool report) {
    const int rb_pre = cdiv(p.B * p.R, rows_per_block), n_pre_items = p.do_prefix ? rb_pre * p.h_kv * p.n_pre : 0;
    if (idx < n_pre_items) {
        // row blocks of one (head, split) are neighbours: they read the same keys
        const int rb = idx % rb_pre, split = (idx / rb_pre) % p.n_pre;
        w.kvh = idx / (rb_pre * p.n_pre);
        w.prefix = true;
        w.b = 0;
        w.row0 = rb * rows_per_block;
        w.nrows = min(rows_per_block, p.B * p.R - w.row0);
        w.L = prefix_length(p, report && idx == 0);
        w.kbeg = split * p.pre_tokens;
        w.kend = min(w.L, w.kbeg + p.pre_tokens);
        w.slot = split;
    } else {
        idx -= n_pre_items;
        const int rb_suf = cdiv(p.R, rows_per_block);
        const int split = idx % p.n_suf, rb = (idx / p.n_suf) % rb_suf;
        const int bh = idx / (p.n_suf * rb_suf);
        w.kvh = bh % p.h_kv;
        w.b = bh / p.h_kv;
        w.prefix = false;
        w.row0 = rb * rows_per_block;
        w.nrows = min(rows_per_block, p.R - w.row0);
        w.L = clamp_len(p.lens, w.b, p.Lmax, p.s, p.causal, p.status, report && w.kvh == 0 && rb == 0 && split == 0);
        w.kbeg = split * p.suf_tokens;
        w.kend = min(w.L, w.kbeg + p.suf_tokens);
        w.slot = p.n_pre + split;
    }
    return w.kend > w.kbeg;
}

// Row `r` of the item in [B, h_q, s_q].
__device__ __forceinline__ size_t global_row(const PrefixParams& p, const Work& w, int r) {
    const int i = w.row0 + r;
    const int b = w.prefix ? i / p.R : w.b, g = w.prefix ? i % p.R : i;
    return ((size_t)b * p.h_kv + w.kvh) * p.R + g;
}

// Keys below this are visible to row `r`.
__device__ __forceinline__ int visible_end(const PrefixParams& p, const Work& w, int r) {
    if (w.prefix || !p.causal) return w.L;
    return w.L - p.s + (w.row0 + r) % p.s + 1;
}

__device__ __forceinline__ CacheRows rows_of(const PrefixParams& p, const Work& w) {
    CacheRows c;
    c.page_size = p.page_size;
    c.num_pages = p.num_pages;
    c.heads = p.h_kv;
    if (p.table) {
        c.table = w.prefix ? p.ptable : p.table + (size_t)w.b * p.max_pages;
        c.head_rows = w.kvh;
    } else {
        c.table = nullptr;
        c.head_rows = w.prefix ? (long long)w.kvh * p.Lp : ((long long)w.b * p.h_kv + w.kvh) * p.Lmax;
    }
    return c;
}

// ---- bf16: warp-level MMAs ------------------------------------------------------------------------------------
// What both kernels do with 16 query rows and KG groups of 16 keys: scores, online softmax, values.  A warp's lane
// (g, t) holds rows g and g + 8.
template <int D>
struct RowState {
    float o[D / 8][4];
    float m[2], l[2];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    // the row sums over the four lanes of a row
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
    }
};

// q(ks, regs): A fragments of k-step ks; k_at / v_at (row, 16-byte chunk): shared addresses of the tile; the warp's
// keys are rows key_w .. of the tile, key k0 + j the j-th of them; keys below vis[h] are visible to row g + 8 h.
template <int D, int KG, class Q, class KA, class VA>
__device__ __forceinline__ void attend_tile(RowState<D>& st, const Q& q, const KA& k_at, const VA& v_at, int key_w, int k0,
                                            const int* vis, int vis_all, float scale_log2) {
    const int lane = threadIdx.x % 32, t = lane % 4;
    float s[KG][2][4];
#pragma unroll
    for (int kg = 0; kg < KG; ++kg)
#pragma unroll
        for (int n = 0; n < 2; ++n) s[kg][n][0] = s[kg][n][1] = s[kg][n][2] = s[kg][n][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t qa[4];
        q(ks, qa);
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
            uint32_t kf[4];  // matrices: (keys 0-7, k 0-7), (keys 0-7, k 8-15), (keys 8-15, ..) x 2
            ldmatrix4(kf, k_at(key_w + kg * 16 + (lane / 16) * 8 + lane % 8, 2 * ks + (lane / 8) % 2));
            mma_bf16(s[kg][0], qa, kf[0], kf[1]);
            mma_bf16(s[kg][1], qa, kf[2], kf[3]);
        }
    }
    float mx[2] = {-INFINITY, -INFINITY};
    const bool whole = k0 + 16 * KG <= vis_all;
#pragma unroll
    for (int kg = 0; kg < KG; ++kg)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = s[kg][n][e] * scale_log2;
                if (!whole && k0 + kg * 16 + n * 8 + 2 * t + (e & 1) >= vis[e / 2]) x = -INFINITY;
                s[kg][n][e] = x;
                mx[e / 2] = fmaxf(mx[e / 2], x);
            }
    // the reference maximum moves only when a score exceeds it by 2^8; a row's lanes agree on it only then
    const bool grow = mx[0] > st.m[0] + 8.f || mx[1] > st.m[1] + 8.f || (st.m[0] == -INFINITY && mx[0] > -INFINITY) ||
                      (st.m[1] == -INFINITY && mx[1] > -INFINITY);
    if (__any_sync(0xffffffffu, grow)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            // by its own row alone: what other rows (or rows past the item) hold changes nothing
            const bool move = mx[h] > st.m[h] + 8.f || (st.m[h] == -INFINITY && mx[h] > -INFINITY);
            al[h] = move ? fast_exp2(st.m[h] - mx[h]) : 1.f;
            if (move) st.m[h] = mx[h];
            st.l[h] *= al[h];
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            st.o[i][0] *= al[0];
            st.o[i][1] *= al[0];
            st.o[i][2] *= al[1];
            st.o[i][3] *= al[1];
        }
    }
    const float ms[2] = {st.m[0] == -INFINITY ? 0.f : st.m[0], st.m[1] == -INFINITY ? 0.f : st.m[1]};
    // P in the A layout of the value product (rounded to bf16 as everywhere in the library; the sums are of the fp32
    // values)
#pragma unroll
    for (int kg = 0; kg < KG; ++kg) {
        uint32_t pa[4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = fast_exp2(s[kg][n][i] - ms[i / 2]);
            st.l[0] += e[0] + e[1];
            st.l[1] += e[2] + e[3];
            pa[2 * n] = pack_bf16x2(e[0], e[1]);
            pa[2 * n + 1] = pack_bf16x2(e[2], e[3]);
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t vf[4];  // transposed: (keys 0-7, 8-15) of value columns 16 i .. + 7, then .. + 15
            ldmatrix4_t(vf, v_at(key_w + kg * 16 + lane % 16, 2 * i + lane / 16));
            mma_bf16(st.o[2 * i], pa, vf[0], vf[1]);
            mma_bf16(st.o[2 * i + 1], pa, vf[2], vf[3]);
        }
    }
}

// Few rows: 16 query rows per item, the four consumer warps take 16 keys each of a 64-key tile and join their states
// at the end of the item.  Bound by reading K and V (a suffix's are read once), so the blocks are persistent: warp 4
// streams the tiles of one item after another with TMA through one ring, which never drains between items, and hands
// the consumers each item's description with its query rows.
template <int D>
struct StreamCfg {
    static constexpr int TK = 64, ROWS = 16, NB = D / 64;
    static constexpr int BOX = TK * 128, MAT = NB * BOX, STAGE = 2 * MAT;  // a box: 64 rows of 64 values
    static constexpr int NS = D == 64 ? 4 : 3;
    static constexpr int BLOCKS = D == 64 ? 3 : D == 128 ? 2 : 1;          // per SM
    static constexpr int QROW = D * 2 + 16;                                // padded: ldmatrix without bank conflicts
    static constexpr int OROW = D + 8;                                     // fp32 values, padded likewise
    static constexpr int OFF_Q = NS * STAGE, OFF_O = OFF_Q + ROWS * QROW;  // O: [16][OROW], the join
    static constexpr int OFF_ML = OFF_O + ROWS * OROW * 4;                 // [4][16] maxima, then sums
    static constexpr int OFF_BAR = OFF_ML + 2 * 4 * ROWS * 4;
    static constexpr int SMEM = 1024 + OFF_BAR + 128;
    static_assert((SMEM + 1024) * BLOCKS <= 233472, "shared memory");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// Whether `pred` holds in any of the 128 consumer threads (named barrier 1 with an OR reduction).
__device__ __forceinline__ bool any_consumer(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.aligned.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred)
        : "memory");
    return r != 0;
}

template <int D>
__global__ void __launch_bounds__(160, StreamCfg<D>::BLOCKS)
    prefix_stream_kernel(const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ CUtensorMap tm_vp,
                         const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const PrefixParams p, const int n_items, const int box_rows) {
    using C = StreamCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(smem_raw), 1024));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::NS;
    uint64_t* q_full = empty + C::NS;
    uint64_t* q_empty = q_full + 1;
    __shared__ Work s_work;
    __shared__ int s_more, s_abort;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 4);
        }
        mbar_init(smem_u32(q_full), 1);
        mbar_init(smem_u32(q_empty), 4);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_trigger();

    if (warp == 4) {
        // ------------------------------ producer: one lane per box of a tile ------------------------------
        const int r = lane * box_rows;
        int n = 0, item = 0;  // tiles and items issued
        bool ok = true;
        auto next_item = [&](const Work* w) {  // hands over an item, or the end
            if (item > 0) ok = mbar_wait(smem_u32(q_empty), (item - 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            const uint32_t qb = smem_u32(q_full);
            if (lane == 0) {
                s_more = w && ok;
                if (w) s_work = *w;
                __threadfence_block();
                if (w && ok)
                    mbar_arrive_expect_tx(qb, w->nrows * D * 2);
                else
                    mbar_arrive(qb);
            }
            __syncwarp();
            if (w && ok && lane < w->nrows)
                bulk_load(smem_u32(smem + C::OFF_Q) + lane * C::QROW,
                          static_cast<const __nv_bfloat16*>(p.q) + global_row(p, *w, lane) * D, D * 2, qb);
            ++item;
        };
        // Items are handed out as blocks get to them (their lengths differ); the next number is asked for an item ahead.
        auto ask = [&]() { return lane == 0 ? (int)gridDim.x + atomicAdd(p.next_item, 1) : 0; };
        int asked = ask();
        for (int idx = blockIdx.x, next; ok && idx < n_items; idx = next) {
            Work w;
            const bool some = find_work(p, C::ROWS, idx, w, lane == 0);
            next = __shfl_sync(0xffffffffu, asked, 0);
            if (next < n_items) asked = ask();
            if (!some) continue;
            next_item(&w);
            const CUtensorMap* mk = w.prefix ? &tm_kp : &tm_k;
            const CUtensorMap* mv = w.prefix ? &tm_vp : &tm_v;
            const int32_t* table = p.table ? (w.prefix ? p.ptable : p.table + (size_t)w.b * p.max_pages) : nullptr;
            int y = 0, z = w.prefix ? w.kvh : w.b * p.h_kv + w.kvh;
            auto look_up = [&](int tile) {
                const int tok = w.kbeg + tile * C::TK + r;
                y = tok;
                if (table) {
                    int page = r < C::TK && tok < w.kend ? table[tok / p.page_size] : 0;
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(p.status, kDevBadPage);
                        page = 0;
                    }
                    y = tok % p.page_size;
                    z = page * p.h_kv + w.kvh;
                }
            };
            look_up(0);
            const int n_tiles = cdiv(w.kend - w.kbeg, C::TK);
            for (int j = 0; ok && j < n_tiles; ++j, ++n) {
                const int s = n % C::NS;
                if (n >= C::NS) ok = mbar_wait(smem_u32(&empty[s]), (n / C::NS - 1) & 1, p.status);
                ok = __all_sync(0xffffffffu, ok && !*(volatile int*)&s_abort);
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[s]), dst = smem_u32(smem + s * C::STAGE) + r * 128;
                if (lane == 0) mbar_arrive_expect_tx(fb, C::STAGE);
                __syncwarp();
                if (r < C::TK) {
#pragma unroll
                    for (int x = 0; x < C::NB; ++x) {
                        tma_load_3d(dst + x * C::BOX, mk, x * 64, y, z, fb);
                        tma_load_3d(dst + C::MAT + x * C::BOX, mv, x * 64, y, z, fb);
                    }
                }
                if (j + 1 < n_tiles) look_up(j + 1);
            }
        }
        next_item(nullptr);
        // every issued copy lands before the CTA may end
        for (int i = n - 1; i >= 0 && i >= n - C::NS; --i)
            mbar_wait(smem_u32(&full[i % C::NS]), (i / C::NS) & 1, p.status);
        return;
    }

    const int g = lane / 4, t = lane % 4, key_w = warp * 16;
    float* om = reinterpret_cast<float*>(smem + C::OFF_O);
    float* ml = reinterpret_cast<float*>(smem + C::OFF_ML);
    const uint32_t sq = smem_u32(smem + C::OFF_Q);
    RowState<D> st;
    int n = 0;
    for (int item = 0;; ++item) {
        bool ok = mbar_wait(smem_u32(q_full), item & 1, p.status);
        if (!ok) s_abort = 1;
        if (any_consumer(!ok || !s_more)) break;  // all or none: they meet again at the join
        const Work w = s_work;
        constexpr bool QREG = D <= 128;  // the query fragments stay in registers; otherwise they are read again per tile
        uint32_t qf[QREG ? D / 16 : 1][4];
        auto q_at = [&](int ks, uint32_t* to) { ldmatrix4(to, sq + (lane % 16) * C::QROW + (2 * ks + lane / 16) * 16); };
        if constexpr (QREG) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) q_at(ks, qf[ks]);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(q_empty));
        }
        int vis[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            vis[h] = r < w.nrows ? min(visible_end(p, w, r), w.kend) : 0;
        }
        // keys below are visible to every row of the item (rows past it do not count)
        const int vis_all = __reduce_min_sync(0xffffffffu, min(g < w.nrows ? vis[0] : w.kend, g + 8 < w.nrows ? vis[1] : w.kend));
        st.clear();
        const int n_tiles = cdiv(w.kend - w.kbeg, C::TK);
        for (int j = 0; j < n_tiles; ++j, ++n) {
            const int s = n % C::NS;
            if (ok) ok = mbar_wait(smem_u32(&full[s]), (n / C::NS) & 1, p.status);
            const int k0 = w.kbeg + j * C::TK + key_w;
            if (ok && k0 < w.kend) {
                uint8_t* kt = smem + s * C::STAGE;
                const uint32_t kb = smem_u32(kt), vb = kb + C::MAT;
                auto at = [](uint32_t base, int r, int c) { return base + (c / 8) * C::BOX + r * 128 + (((c % 8) ^ (r & 7)) * 16); };
                if (k0 + 16 > w.kend) {
                    // value rows past the keys may hold anything, and 0 x NaN would reach every row: zeros
                    const int first = w.kend - k0;
                    for (int x = lane; x < (16 - first) * (D / 8); x += 32) {
                        const int r = key_w + first + x / (D / 8), c = x % (D / 8);
                        *reinterpret_cast<uint4*>(kt + C::MAT + (c / 8) * C::BOX + r * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy into the stage
                    __syncwarp();
                }
                auto q_regs = [&](int ks, uint32_t* to) {
                    if constexpr (QREG) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) to[e] = qf[ks][e];
                    } else {
                        q_at(ks, to);
                    }
                };
                attend_tile<D, 1>(st, q_regs, [&](int r, int c) { return at(kb, r, c); }, [&](int r, int c) { return at(vb, r, c); },
                                  key_w, k0, vis, vis_all, p.scale_log2);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
        }
        if constexpr (!QREG) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(q_empty));
        }
        // join the four warps' states, one after the other into one buffer
        st.finish();
        if (t == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ml[warp * 16 + g + 8 * h] = st.m[h];
                ml[64 + warp * 16 + g + 8 * h] = st.l[h];
            }
        }
        named_barrier(1, 128);
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            const float M = fmaxf(fmaxf(ml[r], ml[16 + r]), fmaxf(ml[32 + r], ml[48 + r]));
            f[h] = M == -INFINITY ? 0.f : fast_exp2(st.m[h] - M);
        }
        for (int k = 0; k < 4; ++k) {
            if (k == warp) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = g + 8 * h;
                    if (r >= w.nrows) continue;
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        float2* x = reinterpret_cast<float2*>(om + r * C::OROW + i * 8 + 2 * t);
                        float2 v = make_float2(st.o[i][2 * h] * f[h], st.o[i][2 * h + 1] * f[h]);
                        if (k) v = __fadd2_rn(v, *x);
                        *x = v;
                    }
                }
            }
            named_barrier(1, 128);
        }
        for (int i = threadIdx.x; i < w.nrows * (D / 4); i += 128) {
            const int r = i / (D / 4), c = i % (D / 4);
            float M = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) M = fmaxf(M, ml[k * 16 + r]);
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += fast_exp2(ml[k * 16 + r] - (M == -INFINITY ? 0.f : M)) * ml[64 + k * 16 + r];
            const float inv = part_inverse(sum);
            const float4 x = *reinterpret_cast<const float4*>(om + r * C::OROW + c * 4);
            const size_t to = global_row(p, w, r) * p.n_slots + w.slot;
            *reinterpret_cast<float4*>(p.part_o + to * D + c * 4) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            if (c == 0) p.part_lse[to] = part_normaliser(M, sum);
        }
        named_barrier(1, 128);  // the buffers are free for the next item
        if (!ok) s_abort = 1;
    }
    // the merge waits for this kernel alone: it ends only after the prefix kernel before it
    if (threadIdx.x == 0) pdl_wait();
}

// Many rows at d = 256 (whose accumulators do not fit prefix_tc_kernel's tensor memory twice): 64 query rows, 16 per
// warp, every warp takes whole tiles of 64 keys, copied row by row.
template <int D>
struct Rows64Cfg {
    static constexpr int TK = 64, ROWS = 64, STAGES = 3;
    static constexpr int MAT = TK * D * 2, STAGE = 2 * MAT, QB = ROWS * D * 2;
    static constexpr int SMEM = QB + STAGES * STAGE;
    static_assert(SMEM <= 232448, "shared memory");
};

// Byte offset of 16-byte chunk c of row r: rows of D bf16 values, chunks permuted so that the 8 rows an ldmatrix
// phase reads at one chunk lie in different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return (uint32_t)(r * D * 2 + ((c ^ (r & 7)) * 16));
}

template <int D>
__global__ void __launch_bounds__(128) prefix_rows64_kernel(const PrefixParams p) {
    using C = Rows64Cfg<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    Work w;
    pdl_trigger();
    if (!find_work(p, C::ROWS, blockIdx.x, w, tid == 0)) return;
    const CacheRows rows = rows_of(p, w);
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(w.prefix ? p.kp : p.k);
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(w.prefix ? p.vp : p.v);
    const uint32_t sq = smem_u32(smem), st0 = sq + C::QB;
    for (int i = tid; i < C::ROWS * (D / 8); i += 128) {
        const int r = i / (D / 8), c = i % (D / 8);
        const bool ok = r < w.nrows;
        cp_async16(sq + swz<D>(r, c), static_cast<const __nv_bfloat16*>(p.q) + (ok ? global_row(p, w, r) * D + c * 8 : 0), ok);
    }
    // keys and values of one tile; rows past the item's keys are zeros
    auto load_tile = [&](int tile, int stage) {
        const uint32_t dst = st0 + stage * C::STAGE;
        const int k0 = w.kbeg + tile * C::TK;
        constexpr int RPI = 128 / (D / 8);  // rows per pass of the block
        const int c = tid % (D / 8);
#pragma unroll
        for (int r = tid / (D / 8); r < C::TK; r += RPI) {
            const bool ok = k0 + r < w.kend;
            const long long at = (ok ? cache_row(rows, k0 + r, p.status) : 0) * D + c * 8;
            cp_async16(dst + swz<D>(r, c), kb + at, ok);
            cp_async16(dst + C::MAT + swz<D>(r, c), vb + at, ok);
        }
    };
    const int n_tiles = cdiv(w.kend - w.kbeg, C::TK);
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
        if (s < n_tiles) load_tile(s, s);
        cp_async_commit();
    }
    const int row_w = warp * 16;
    int vis[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row_w + g + 8 * h;
        vis[h] = r < w.nrows ? min(visible_end(p, w, r), w.kend) : 0;
    }
    const int vis_all = __reduce_min_sync(0xffffffffu, min(vis[0], vis[1]));
    RowState<D> st;
    st.clear();
    for (int j = 0; j < n_tiles; ++j) {
        cp_async_wait<C::STAGES - 2>();
        __syncthreads();
        if (j + C::STAGES - 1 < n_tiles) load_tile(j + C::STAGES - 1, (j + C::STAGES - 1) % C::STAGES);
        cp_async_commit();
        const uint32_t kt = st0 + (j % C::STAGES) * C::STAGE, vt = kt + C::MAT;
        attend_tile<D, 4>(st, [&](int ks, uint32_t* to) { ldmatrix4(to, sq + swz<D>(row_w + lane % 16, 2 * ks + lane / 16)); },
                          [&](int r, int c) { return kt + swz<D>(r, c); }, [&](int r, int c) { return vt + swz<D>(r, c); }, 0,
                          w.kbeg + j * C::TK, vis, vis_all, p.scale_log2);
    }
    cp_async_wait<0>();
    st.finish();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = row_w + g + 8 * h;
        if (r >= w.nrows) continue;
        const size_t at = global_row(p, w, r) * p.n_slots + w.slot;
        const float inv = part_inverse(st.l[h]);
        float* po = p.part_o + at * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(po + i * 8 + 2 * t) = make_float2(st.o[i][2 * h] * inv, st.o[i][2 * h + 1] * inv);
        if (t == 0) p.part_lse[at] = part_normaliser(st.m[h], st.l[h]);
    }
}

// ---- fp32: CUDA cores ------------------------------------------------------------------------------------------
// Bound by the issue of instructions and shared-memory reads around the multiply-adds (no fp32 tensor product exists).
// Eight warps share a tile of 64 keys; a warp takes RPW rows and 64 / KG of the keys, so that a key vector feeds RPW
// multiply-adds and a query vector one per key lane.  32 rows: eight rows and half the keys a warp; 16 rows: a quarter,
// two lanes a key; up to 4 rows: every warp all of them on an eighth, four lanes a key.  The key groups of a row keep
// sums of their own, joined once at the end.  64 x 4 rows of 8 heads of 128 over 4096 keys: 247 us (four warps of four
// rows on 32 keys: 324); one sequence of 4 rows: 18 us (26).
template <int D, int RPW, int KG>
struct F32Cfg {
    static constexpr int TK = 64, KPW = TK / KG, LPK = 32 / KPW;  // keys per warp, lanes per key
    static constexpr int WARPS = 8, THREADS = 32 * WARPS, BLOCKS = D == 64 ? 3 : 2;  // blocks per SM
    static constexpr int ROWS = RPW * (WARPS / KG);
    // 16 bytes behind each lane's part of a key or query, 16 behind the key: the reads of 8 lanes hit all banks
    static constexpr int PART = D / LPK, KROW = D + 4 * LPK, QROW = D + 4 * LPK;
    static constexpr int SMEM = (ROWS * QROW + TK * KROW + TK * D + WARPS * RPW * KPW) * 4;
    static_assert(WARPS * RPW * (D + 2) <= TK * KROW, "the join fits the key tile");
};

template <int D, int RPW, int KG>
__global__ void __launch_bounds__(256, (F32Cfg<D, RPW, KG>::BLOCKS)) prefix_f32_kernel(const PrefixParams p) {
    using C = F32Cfg<D, RPW, KG>;
    constexpr int VPL = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    float* qs = reinterpret_cast<float*>(smem);
    float* ks = qs + C::ROWS * C::QROW;
    float* vs = ks + C::TK * C::KROW;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int row_w = warp / KG * RPW, key_w = warp % KG * C::KPW;  // the warp's first row and key
    const int key = key_w + lane / C::LPK, sub = lane % C::LPK;     // the lane's key and its part of the head dim
    float* ps = vs + C::TK * D + warp * RPW * C::KPW;
    Work w;
    pdl_trigger();
    if (!find_work(p, C::ROWS, blockIdx.x, w, tid == 0)) {
        pdl_wait();
        return;
    }
    const CacheRows rows = rows_of(p, w);
    const float* kb = static_cast<const float*>(w.prefix ? p.kp : p.k);
    const float* vb = static_cast<const float*>(w.prefix ? p.vp : p.v);
    for (int i = tid; i < C::ROWS * (D / 4); i += C::THREADS) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < w.nrows) x = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + global_row(p, w, r) * D + c);
        *reinterpret_cast<float4*>(qs + r * C::QROW + c + c / C::PART * 4) = x;
    }
    int vis[RPW];
    float m[RPW], l[RPW], o[RPW][VPL];
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        vis[r] = row_w + r < w.nrows ? min(visible_end(p, w, row_w + r), w.kend) : 0;
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) o[r][i] = 0.f;
    }
    for (int k0 = w.kbeg; k0 < w.kend; k0 += C::TK) {
        __syncthreads();
        for (int i = tid; i < C::TK * (D / 4); i += C::THREADS) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            const bool ok = k0 + r < w.kend;
            const long long at = ok ? cache_row(rows, k0 + r, p.status) * D + c : 0;
            cp_async16(smem_u32(ks + r * C::KROW + c + c / C::PART * 4), kb + at, ok);
            cp_async16(smem_u32(vs + r * D + c), vb + at, ok);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        if (row_w >= w.nrows || k0 + key_w >= w.kend) continue;  // a warp without rows or keys only loads
        float s[RPW] = {};
        const float* kp = ks + key * C::KROW + sub * (C::PART + 4);
        const float* qp = qs + row_w * C::QROW + sub * (C::PART + 4);
#pragma unroll 4
        for (int c = 0; c < C::PART; c += 4) {
            const float4 kv = *reinterpret_cast<const float4*>(kp + c);
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const float4 qv = *reinterpret_cast<const float4*>(qp + r * C::QROW + c);
                s[r] = fmaf(kv.x, qv.x, fmaf(kv.y, qv.y, fmaf(kv.z, qv.z, fmaf(kv.w, qv.w, s[r]))));
            }
        }
#pragma unroll
        for (int r = 0; r < RPW; ++r) {
#pragma unroll
            for (int d = 1; d < C::LPK; d *= 2) s[r] += __shfl_xor_sync(0xffffffffu, s[r], d);
            const float x = k0 + key < vis[r] ? s[r] * p.scale_log2 : -INFINITY;
            float mx = x;
#pragma unroll
            for (int d = 16; d >= C::LPK; d /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[r], mx);
            const float al = mn == -INFINITY ? 1.f : exp2f(m[r] - mn);
            const float e = x == -INFINITY ? 0.f : exp2f(mn == -INFINITY ? x : x - mn);  // (a NaN score moves no maximum)
            m[r] = mn;
            l[r] = l[r] * al + e;
            if (sub == 0) ps[r * C::KPW + lane / C::LPK] = e;
#pragma unroll
            for (int i = 0; i < VPL; ++i) o[r][i] *= al;
        }
        __syncwarp();
        const float* vp = vs + key_w * D + lane * VPL;  // lane: value columns VPL * lane ..
#pragma unroll 2
        for (int k = 0; k < C::KPW; k += 4) {
            float v[4][VPL];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (VPL == 4)
                    *reinterpret_cast<float4*>(v[e]) = *reinterpret_cast<const float4*>(vp + (k + e) * D);
                else
                    *reinterpret_cast<float2*>(v[e]) = *reinterpret_cast<const float2*>(vp + (k + e) * D);
            }
#pragma unroll
            for (int r = 0; r < RPW; ++r) {
                const float4 e = *reinterpret_cast<const float4*>(ps + r * C::KPW + k);
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    o[r][i] = fmaf(e.w, v[3][i], fmaf(e.z, v[2][i], fmaf(e.y, v[1][i], fmaf(e.x, v[0][i], o[r][i]))));
            }
        }
        __syncwarp();
    }
    // every warp's rows side by side, then row by row the sum of its key groups
    __syncthreads();
    float* join = ks;  // [WARPS][RPW][D + 2]: values, maximum, sum
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
        float sum = l[r];
#pragma unroll
        for (int d = 16; d >= C::LPK; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        float* at = join + (warp * RPW + r) * (D + 2);
#pragma unroll
        for (int i = 0; i < VPL; ++i) at[lane * VPL + i] = o[r][i];
        if (lane == 0) {
            at[D] = m[r];
            at[D + 1] = sum;
        }
    }
    __syncthreads();
    for (int r = warp; r < min(C::ROWS, w.nrows); r += C::WARPS) {
        const float* at = join + (r / RPW * KG * RPW + r % RPW) * (D + 2);  // key group g: RPW rows on
        float mx = -INFINITY, sum = 0.f, acc[VPL] = {};
#pragma unroll
        for (int g = 0; g < KG; ++g) mx = fmaxf(mx, at[g * RPW * (D + 2) + D]);
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            const float* part = at + g * RPW * (D + 2);
            const float f = part[D] == -INFINITY ? 0.f : exp2f(part[D] - mx);
            sum += f * part[D + 1];
#pragma unroll
            for (int i = 0; i < VPL; ++i) acc[i] += f * part[lane * VPL + i];
        }
        const size_t to = global_row(p, w, r) * p.n_slots + w.slot;
        const float inv = part_inverse(sum);
#pragma unroll
        for (int i = 0; i < VPL; ++i) p.part_o[to * D + lane * VPL + i] = acc[i] * inv;
        if (lane == 0) p.part_lse[to] = part_normaliser(mx, sum);
    }
    pdl_wait();  // the prefix's launch, before this one counts as done
}

// ---- the merge ---------------------------------------------------------------------------------------------------
// WPR warps per row (four where there are few rows and many parts to a row, one otherwise).  A row's parts are the
// prefix splits its length reaches and the suffix splits with a key that the row sees; the lanes fetch their lse
// together, then every warp joins its share of the parts, every lane D / 32 values, eight parts in flight.
template <typename T, int D, int WPR>
__global__ void __launch_bounds__(128) prefix_merge_kernel(const PrefixParams p) {
    constexpr int VPL = D / 32;
    __shared__ float fs[4][kMaxSlots];
    __shared__ __align__(16) float others[WPR > 1 ? 3 : 1][WPR > 1 ? D : 4];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, share = warp % WPR;
    const size_t row = (size_t)blockIdx.x * (4 / WPR) + warp / WPR;
    if (row >= (size_t)p.B * p.h_q * p.s) return;
    const int b = (int)(row / ((size_t)p.h_q * p.s)), t = (int)(row % p.s);
    const int P = prefix_length(p, false);
    const int L = clamp_len(p.lens, b, p.Lmax, p.s, p.causal, p.status, false);
    const int seen = p.causal ? L - p.s + t + 1 : L;
    const int np = cdiv(P, p.pre_tokens), n = np + cdiv(seen, p.suf_tokens), gap = p.n_pre - np;
    pdl_wait();
    if (row == 0 && threadIdx.x == 0) *p.next_item = 0;  // for the next call
    const float* pl = p.part_lse + row * p.n_slots;
    float x[kMaxSlots / 32], M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kMaxSlots / 32; ++k) {
        const int i = k * 32 + lane;
        x[k] = i < n ? pl[i < np ? i : i + gap] : -INFINITY;
        M = fmaxf(M, x[k]);
    }
#pragma unroll
    for (int o = 16; o; o /= 2) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxSlots / 32; ++k) {
        const float f = x[k] == -INFINITY ? 0.f : exp2f(x[k] - M);
        fs[warp][k * 32 + lane] = f;
        sum += f;
    }
#pragma unroll
    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    const float* po = p.part_o + row * p.n_slots * D + lane * VPL;
    float a[VPL] = {};
#pragma unroll 8
    for (int i = share; i < n; i += WPR) {
        const float f = fs[warp][i];
        const float* src = po + (size_t)(i < np ? i : i + gap) * D;
        float y[VPL];
        if constexpr (VPL == 2) {
            *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(src);
        } else {
#pragma unroll
            for (int e = 0; e < VPL; e += 4) *reinterpret_cast<float4*>(y + e) = *reinterpret_cast<const float4*>(src + e);
        }
#pragma unroll
        for (int e = 0; e < VPL; ++e) a[e] = fmaf(f, y[e], a[e]);
    }
    if constexpr (WPR > 1) {
        if (share > 0) {
#pragma unroll
            for (int e = 0; e < VPL; ++e) others[share - 1][lane * VPL + e] = a[e];
        }
        __syncthreads();
        if (share > 0) return;
#pragma unroll
        for (int k = 0; k < WPR - 1; ++k)
#pragma unroll
            for (int e = 0; e < VPL; ++e) a[e] += others[k][lane * VPL + e];
    }
    const float inv = part_inverse(sum);
    T* out = static_cast<T*>(p.out) + row * D + lane * VPL;
    if constexpr (sizeof(T) == 2) {
        uint32_t u[VPL / 2];
#pragma unroll
        for (int e = 0; e < VPL / 2; ++e) u[e] = pack_bf16x2(a[2 * e] * inv, a[2 * e + 1] * inv);
        if constexpr (VPL == 2) *reinterpret_cast<uint32_t*>(out) = u[0];
        if constexpr (VPL == 4) *reinterpret_cast<uint2*>(out) = make_uint2(u[0], u[1]);
        if constexpr (VPL == 8) *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int e = 0; e < VPL; e += 2) *reinterpret_cast<float2*>(out + e) = make_float2(a[e] * inv, a[e + 1] * inv);
    }
    if (p.lse && lane == 0) p.lse[row] = part_normaliser(M, sum) * 0.69314718055994530942f;
}

template <typename T, int D>
cudaError_t launch_merge(const PrefixParams& p, cudaStream_t st) {
    const size_t rows = (size_t)p.B * p.h_q * p.s;
    if (p.n_slots > 8 && rows <= 4u * sm_count())
        return launch_pdl<prefix_merge_kernel<T, D, 4>>(dim3((unsigned)rows), 128, 0, st, p);
    return launch_pdl<prefix_merge_kernel<T, D, 1>>(dim3((unsigned)((rows + 3) / 4)), 128, 0, st, p);
}

// ---- planning ------------------------------------------------------------------------------------------------------
struct PrefixPlan {
    bool tc;                 // the prefix runs on prefix_tc_kernel
    int rows_pre, rows_suf;  // query rows per block of the prefix and the suffix kernel
    int pre_tokens, n_pre, suf_tokens, n_suf;
    size_t off_lse, off_o, ws_bytes;
};

// Keys per split of `units` row blocks over L keys: the split count n <= 64 that minimises waves x (tiles per split
// + 2), the 2 for a block's start and end, where the waves of w = units n / slots cost max(ceil(w), w + 1/4).
int split_keys(double units, double slots, int L, int tile) {
    const int lt = cdiv(std::max(L, 1), tile);
    int best = 1;
    double best_cost = -1.0;
    for (int n = 1; n <= lt && n <= kMaxSplits; ++n) {
        const double w = units * n / slots;
        const double cost = fmax(ceil(w - 1e-9), w + 0.25) * (cdiv(lt, n) + 2);
        if (best_cost < 0.0 || cost < best_cost - 1e-9) {
            best_cost = cost;
            best = n;
        }
    }
    return cdiv(lt, best) * tile;
}

// The same for persistent blocks, which run on from item to item: the work of a block (half a tile per item for its
// start and join) and half an item's length as the tail.
int stream_keys(double units, double slots, int L, int tile) {
    const int lt = cdiv(std::max(L, 1), tile);
    int best = 1;
    double best_cost = -1.0;
    for (int n = 1; n <= lt && n <= kMaxSplits; ++n) {
        const int t = cdiv(lt, n);
        const double cost = fmax(units * n / slots, 1.0) * (t + 0.5) + 0.5 * t;
        if (best_cost < 0.0 || cost < best_cost - 1e-9) {
            best_cost = cost;
            best = n;
        }
    }
    return cdiv(lt, best) * tile;
}

// Keys per split of the tensor-core prefix kernel, planned with the suffix kernel that shares the SMs with it: blocks of
// the suffix kernel run where prefix blocks leave an SM free, and everywhere once they are done.  In units of a key
// tile's time in a prefix block (1.85 us): a block costs its tiles + 2.7, a 64-key suffix tile 0.4 d / 128 of an SM, a
// suffix block 2 to start; suffixes count at half their capacity.  (64 sequences over a prefix of 8192: 8 splits, half
// the SMs, instead of 16.)
int tc_keys(int pairs_heads, int Lp, double suffix_tiles, int d) {
    const int lt = cdiv(std::max(Lp, 1), 128), sms = sm_count();
    const double suffix = 0.5 * suffix_tiles * 0.4 * d / 128;
    int best = 1;
    double best_cost = -1.0;
    for (int n = 1; n <= lt && n <= kMaxSplits; ++n) {
        const double blocks = (double)pairs_heads * n, waves = ceil(blocks / sms), t = waves * (cdiv(lt, n) + 2.7);
        const double free_sms = sms - blocks / waves, left = suffix - free_sms * fmax(t - 2.0, 0.0);
        const double cost = t + (left > 0.0 ? 2.0 + left / sms : 0.0);
        if (best_cost < 0.0 || cost < best_cost - 1e-9) {
            best_cost = cost;
            best = n;
        }
    }
    return cdiv(lt, best) * 128;
}

// Query rows of a block of prefix_f32_kernel where there are `rows`.
int f32_rows(int rows) { return rows <= 4 ? 4 : rows <= 16 ? 16 : 32; }

lka_status_t prefix_plan(int B, int h_q, int h_kv, int s, int d, int Lp, int Lmax, lka_dtype_t dtype, PrefixPlan* pl) {
    if (B < 0 || h_q < 1 || h_kv < 1 || s < 1 || d < 1 || Lp < 0 || Lmax < 1 || h_q % h_kv) return LKA_ERR_INVALID_ARG;
    if (dtype != LKA_BF16 && dtype != LKA_FP32) return LKA_ERR_UNSUPPORTED;
    if (!(d == 64 || d == 128 || (d == 256 && dtype == LKA_BF16))) return LKA_ERR_UNSUPPORTED;
    if ((long long)B * h_q * s >= (1ll << 28) || Lp > (1 << 30) || Lmax > (1 << 30)) return LKA_ERR_UNSUPPORTED;
    const int R = h_q / h_kv * s, Bn = std::max(B, 1);
    const bool f32 = dtype == LKA_FP32;
    // Up to 16 query rows per KV head in all: prefix_stream_kernel, whose warps split the keys.  More, and the head dim
    // fits prefix_tc_kernel's tensor memory: that one.  d = 256: prefix_rows64_kernel, the prefix read once per 64 rows.
    pl->tc = !f32 && Bn * R > 16 && d <= 128;
    const int tile = 64;
    const double slots = (double)sm_count() * (f32 ? (d == 128 ? 2 : 3) : d == 256 ? 1 : d == 128 ? 2 : 3);
    pl->rows_pre = Bn * R <= 16 ? 16 : 64;
    pl->rows_suf = 16;
    if (f32) {
        // blocks of 32 rows for a prefix that keeps the SMs busy for a while (64 x 4 rows of 8 heads over 4096 keys: 247 us,
        // 295 in 16s), of 16, and with suffixes of as many in one launch, for a short one (7 x 12 rows over 1001 keys:
        // 15.3 us, 17.3 in 32s)
        pl->rows_suf = f32_rows(R);
        const bool own = (double)h_kv * cdiv(Bn * R, 16) * cdiv(Lp, tile) >= 4 * slots;
        pl->rows_pre = own ? f32_rows(Bn * R) : std::max(pl->rows_suf, std::min(16, f32_rows(Bn * R)));
    }
    const bool rows64 = !f32 && !pl->tc && Bn * R > 16;
    // the split knob, where it leaves at most kMaxSplits splits
    const int knob = split_tokens_knob();
    auto by_knob = [knob](int L, int unit) { return cdiv(std::max(knob, cdiv(L, kMaxSplits)), unit) * unit; };
    if (pl->tc)
        pl->pre_tokens = knob > 0 ? by_knob(Lp, 128)
                                  : tc_keys(h_kv * cdiv(prefix_tiles(Bn, R).n_tiles, 2), Lp,
                                            (double)Bn * h_kv * cdiv(R, 16) * cdiv(Lmax, 64), d);
    else
        pl->pre_tokens = knob > 0 ? by_knob(Lp, tile)
                                  : f32 || rows64 ? split_keys((double)h_kv * cdiv(Bn * R, pl->rows_pre), slots, Lp, tile)
                                                  : stream_keys((double)h_kv, slots, Lp, tile);
    pl->suf_tokens = knob > 0 ? by_knob(Lmax, tile)
                              : f32 ? split_keys((double)h_kv * Bn * cdiv(R, pl->rows_suf), slots, Lmax, tile)
                                    : stream_keys((double)h_kv * Bn * cdiv(R, pl->rows_suf), slots, Lmax, tile);
    pl->n_pre = cdiv(Lp, pl->pre_tokens);
    pl->n_suf = cdiv(Lmax, pl->suf_tokens);
    WsCarve c;
    const size_t rows = (size_t)B * h_q * s, slots_n = (size_t)pl->n_pre + pl->n_suf;
    pl->off_lse = c.take(rows * slots_n * sizeof(float));
    pl->off_o = c.take(rows * slots_n * d * sizeof(float));
    pl->ws_bytes = c.off;
    return LKA_OK;
}

template <auto KERN>
cudaError_t launch_items(int smem, const PrefixParams& p, int rows, cudaStream_t st) {
    const cudaError_t e = allow_smem<KERN>(smem);
    if (e != cudaSuccess) return e;
    const long long n = count_work(p, rows);
    if (n == 0) return cudaSuccess;
    if (n >= (1ll << 31)) return cudaErrorInvalidValue;
    KERN<<<(unsigned)n, 128, smem, st>>>(p);
    return cudaPeekAtLastError();
}

// A K or V cache as boxes of 64 values x box_rows tokens: [slabs][rows][D].
template <int D>
bool cache_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t slabs, int box_rows) {
    const uint64_t dims[3] = {(uint64_t)D, rows, slabs}, strides[2] = {D * 2ull, rows * D * 2};
    const uint32_t box[3] = {64, (uint32_t)box_rows, 1};
    return make_tmap_nd(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, dims, strides, box);
}

template <int D>
cudaError_t launch_stream(const PrefixParams& p, cudaStream_t st) {
    using C = StreamCfg<D>;
    const long long n = count_work(p, C::ROWS);
    if (n == 0) return cudaSuccess;
    if (n >= (1ll << 30)) return cudaErrorInvalidValue;
    CUtensorMap kp, vp, k, v;
    const int box_rows = p.table ? std::min(C::TK, p.page_size) : C::TK;
    const uint64_t rows = p.table ? p.page_size : p.Lmax, slabs = (uint64_t)(p.table ? p.num_pages : p.B) * p.h_kv;
    bool ok = cache_map<D>(&k, p.k, rows, slabs, box_rows) && cache_map<D>(&v, p.v, rows, slabs, box_rows);
    if (p.table || p.Lp == 0) {
        kp = k;
        vp = v;
    } else {
        ok = ok && cache_map<D>(&kp, p.kp, p.Lp, p.h_kv, box_rows) && cache_map<D>(&vp, p.vp, p.Lp, p.h_kv, box_rows);
    }
    if (!ok) return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem<prefix_stream_kernel<D>>(C::SMEM);
    if (e != cudaSuccess) return e;
    const int blocks = (int)std::min<long long>(n, (long long)sm_count() * C::BLOCKS);
    if (p.do_prefix) {  // the call's first kernel
        TimedLaunch timer(st);
        prefix_stream_kernel<D><<<blocks, 160, C::SMEM, st>>>(kp, vp, k, v, p, (int)n, box_rows);
        timer.stop();
        return cudaPeekAtLastError();
    }
    return launch_pdl<prefix_stream_kernel<D>>(dim3(blocks), 160, C::SMEM, st, kp, vp, k, v, p, (int)n, box_rows);
}

template <int D>
cudaError_t run_bf16(PrefixParams p, const PrefixPlan& pl, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.n_pre == 0) {
        // no prefix: the suffix kernel is the first
    } else if (pl.tc) {
        if (prefix_tc(p, D, st) != LKA_OK) return cudaErrorLaunchFailure;
        p.do_prefix = 0;
    } else if (pl.rows_pre > 16) {
        if constexpr (D == 256) {
            TimedLaunch timer(st);
            p.do_suffix = 0;
            e = launch_items<prefix_rows64_kernel<D>>(Rows64Cfg<D>::SMEM, p, 64, st);
            p.do_suffix = 1;
            p.do_prefix = 0;
            timer.stop();
        }
    }
    if (e == cudaSuccess) e = launch_stream<D>(p, st);
    if (e != cudaSuccess) return e;
    return launch_merge<__nv_bfloat16, D>(p, st);
}

template <int D, int RPW, int KG>
cudaError_t launch_f32(const PrefixParams& p, bool second, cudaStream_t st) {
    using C = F32Cfg<D, RPW, KG>;
    const cudaError_t e = allow_smem<prefix_f32_kernel<D, RPW, KG>>(C::SMEM);
    const long long n = count_work(p, C::ROWS);
    if (e != cudaSuccess || n == 0) return e;
    if (n >= (1ll << 31)) return cudaErrorInvalidValue;
    if (second) return launch_pdl<prefix_f32_kernel<D, RPW, KG>>(dim3((unsigned)n), C::THREADS, C::SMEM, st, p);
    prefix_f32_kernel<D, RPW, KG><<<(unsigned)n, C::THREADS, C::SMEM, st>>>(p);
    return cudaPeekAtLastError();
}

template <int D>
cudaError_t launch_f32_rows(const PrefixParams& p, int rows, bool second, cudaStream_t st) {
    return rows == 4    ? launch_f32<D, 4, 8>(p, second, st)
           : rows == 16 ? launch_f32<D, 8, 4>(p, second, st)
                        : launch_f32<D, 8, 2>(p, second, st);
}

// Prefix and suffixes in one launch where their blocks have as many rows, else in two beside each other.
template <int D>
cudaError_t run_f32(PrefixParams p, const PrefixPlan& pl, cudaStream_t st) {
    TimedLaunch timer(st);
    cudaError_t e = cudaSuccess;
    const bool two = pl.rows_pre != pl.rows_suf && p.n_pre > 0;
    if (two) {
        p.do_suffix = 0;
        e = launch_f32_rows<D>(p, pl.rows_pre, false, st);
        p.do_prefix = 0;
        p.do_suffix = 1;
    }
    if (e == cudaSuccess) e = launch_f32_rows<D>(p, pl.rows_suf, two, st);
    timer.stop();
    if (e != cudaSuccess) return e;
    return launch_merge<float, D>(p, st);
}

lka_status_t prefix_run(PrefixParams& p, int d, float scale, lka_dtype_t dtype, void* ws, size_t ws_bytes,
                        void* stream) {
    PrefixPlan pl;
    lka_status_t r = prefix_plan(p.B, p.h_q, p.h_kv, p.s, d, p.Lp, p.Lmax, dtype, &pl);
    if (r != LKA_OK) return r;
    if (p.B == 0) return LKA_OK;
    const void* ptrs[] = {p.q, p.k, p.v, p.out, p.lens};
    for (const void* x : ptrs)
        if (!x || !aligned16(x)) return LKA_ERR_INVALID_ARG;
    if (p.Lp > 0 && (!p.kp || !p.vp || !aligned16(p.kp) || !aligned16(p.vp))) return LKA_ERR_INVALID_ARG;
    if (p.prefix_len && (reinterpret_cast<uintptr_t>(p.prefix_len) & 3u)) return LKA_ERR_INVALID_ARG;
    if (p.lse && (reinterpret_cast<uintptr_t>(p.lse) & 3u)) return LKA_ERR_INVALID_ARG;
    if (!isfinite(scale)) return LKA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < pl.ws_bytes) return LKA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LKA_ERR_INVALID_ARG;
    uint8_t* w = static_cast<uint8_t*>(ws);
    p.status = reinterpret_cast<uint32_t*>(w);
    p.next_item = reinterpret_cast<int*>(w + 64);  // in the status header, which is 0 when the workspace is new
    p.part_lse = reinterpret_cast<float*>(w + pl.off_lse);
    p.part_o = reinterpret_cast<float*>(w + pl.off_o);
    p.ratio = p.h_q / p.h_kv;
    p.R = p.ratio * p.s;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.pre_tokens = pl.pre_tokens;
    p.n_pre = pl.n_pre;
    p.suf_tokens = pl.suf_tokens;
    p.n_suf = pl.n_suf;
    p.n_slots = pl.n_pre + pl.n_suf;
    p.do_prefix = p.do_suffix = 1;
    const cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == LKA_FP32)
        e = d == 64 ? run_f32<64>(p, pl, st) : run_f32<128>(p, pl, st);
    else
        e = d == 64 ? run_bf16<64>(p, pl, st) : d == 128 ? run_bf16<128>(p, pl, st) : run_bf16<256>(p, pl, st);
    const lka_status_t done = call_status(e);
    // without a merge the suffix kernel's items stay counted, and a later call would skip as many
    if (done != LKA_OK && cudaMemsetAsync(p.next_item, 0, sizeof(int), st) != cudaSuccess) cudaGetLastError();
    return done;
}

bool prefix_pages_ok(int page_size, int max_prefix_pages, int max_pages, int num_pages) {
    return page_size >= 8 && (page_size & (page_size - 1)) == 0 && max_prefix_pages >= 0 && max_pages >= 1 &&
           num_pages >= 1 && (long long)max_pages * page_size <= (1 << 30) &&
           (long long)max_prefix_pages * page_size <= (1 << 30);
}

}  // namespace
}  // namespace lka

using namespace lka;

extern "C" {

size_t gqa_attn_shared_prefix_workspace_size(int B, int h_q, int h_kv, int s_q, int d_h, int Lp, int Lmax,
                                             lka_dtype_t dtype) {
    PrefixPlan pl;
    return prefix_plan(B, h_q, h_kv, s_q, d_h, Lp, Lmax, dtype, &pl) == LKA_OK ? pl.ws_bytes : 0;
}

lka_status_t gqa_attn_shared_prefix(const void* q, const void* k_prefix, const void* v_prefix,
                                    const int32_t* prefix_len, const void* k, const void* v, const int32_t* cache_lens,
                                    void* out, float* lse, int B, int h_q, int h_kv, int s_q, int d_h, int Lp,
                                    int Lmax, int causal, float scale, lka_dtype_t dtype, void* ws, size_t ws_bytes,
                                    void* stream) {
    PrefixParams p{};
    p.q = q;
    p.kp = k_prefix;
    p.vp = v_prefix;
    p.prefix_len = prefix_len;
    p.k = k;
    p.v = v;
    p.lens = cache_lens;
    p.out = out;
    p.lse = lse;
    p.B = B;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.s = s_q;
    p.Lp = Lp;
    p.Lmax = Lmax;
    p.causal = causal ? 1 : 0;
    return prefix_run(p, d_h, scale, dtype, ws, ws_bytes, stream);
}

size_t gqa_attn_shared_prefix_paged_workspace_size(int B, int h_q, int h_kv, int s_q, int d_h, int page_size,
                                                   int max_prefix_pages, int max_pages, lka_dtype_t dtype) {
    if (!prefix_pages_ok(page_size, max_prefix_pages, max_pages, 1)) return 0;
    return gqa_attn_shared_prefix_workspace_size(B, h_q, h_kv, s_q, d_h, page_size * max_prefix_pages,
                                                 page_size * max_pages, dtype);
}

lka_status_t gqa_attn_shared_prefix_paged(const void* q, const void* k_pages, const void* v_pages,
                                          const int32_t* prefix_table, const int32_t* prefix_len,
                                          const int32_t* block_table, const int32_t* cache_lens, void* out, float* lse,
                                          int B, int h_q, int h_kv, int s_q, int d_h, int page_size,
                                          int max_prefix_pages, int max_pages, int num_pages, int causal, float scale,
                                          lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream) {
    if (!prefix_pages_ok(page_size, max_prefix_pages, max_pages, num_pages)) return LKA_ERR_INVALID_ARG;
    if (B > 0 && (!block_table || (reinterpret_cast<uintptr_t>(block_table) & 3u))) return LKA_ERR_INVALID_ARG;
    if (B > 0 && max_prefix_pages > 0 && (!prefix_table || (reinterpret_cast<uintptr_t>(prefix_table) & 3u)))
        return LKA_ERR_INVALID_ARG;
    PrefixParams p{};
    p.q = q;
    p.kp = p.k = k_pages;
    p.vp = p.v = v_pages;
    p.ptable = prefix_table;
    p.prefix_len = prefix_len;
    p.table = block_table;
    p.lens = cache_lens;
    p.out = out;
    p.lse = lse;
    p.B = B;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.s = s_q;
    p.Lp = page_size * max_prefix_pages;
    p.Lmax = page_size * max_pages;
    p.causal = causal ? 1 : 0;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.num_pages = num_pages;
    return prefix_run(p, d_h, scale, dtype, ws, ws_bytes, stream);
}

}  // extern "C"
