// rope.cu -- rotary positions, alone (rope_apply) and fused with the write of
// a step's new keys and values into the cache (gqa_rope_append*, latent_rope_append*).
//
// Operation: pair i (0 <= i < n) of a head at position p is turned by the angle
// p * inv_freq[i] and scaled by `amplitude` a:
//     y0 = a (x0 cos - x1 sin),  y1 = a (x1 cos + x0 sin)
// with (x0, x1) = (x[i], x[i + n]) (half layout) or (x[2i], x[2i + 1])
// (interleaved); values from 2n on pass through.  The rotation is orthogonal, so
// its backward pass is the same with sin negated (the transpose of a R(p) is a R(-p)).
//
// Angles of far positions lose their fraction of a turn in fp32 (p = 10^6 leaves
// 2^-4 rad), so the turn count p * inv_freq / 2 pi is formed in fp64, reduced to
// [-1/2, 1/2] there, and only the reduced turn goes to fp32 (sincospi): two fp64
// operations per (token, pair), shared by every head of the token.
//
// Bound: HBM (about 0.75 operations per byte moved), or launch latency for a decode step.
// A CTA takes a few consecutive tokens: their cos / sin tables are made once, in shared
// memory, for all heads; then every thread keeps to one unit of a head -- VE pairs, two
// 16-byte vectors -- and carries it through all tokens, two in flight, so that what depends
// on the head (which tensor, addresses, scale) is worked out once per head and what depends on
// the token comes from shared memory.  While there are few tokens, the heads of one token are
// spread over several CTAs instead.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "host_util.h"
#include "launch_util.h"

namespace lka {

struct RopeStrides {
    int64_t b, h, s;  // in elements; the head dim is contiguous
};

struct RopeParams {
    const void *q, *k, *v;  // [B, heads, s, d] through strides; k, v null for rope_apply
    void* q_out;
    RopeStrides qs, ks, vs, os;
    void *kc, *vc;                          // cache bases (k already offset to its column)
    int64_t slab, k_head, v_head, row;      // cache strides in elements: sequence or page, head, token row
    const float *k_scale, *v_scale;         // e4m3 caches: per head (scale_by_head) or one value
    int scale_by_head;
    const int32_t* lens;       // null for rope_apply
    const int32_t* positions;  // [B, s] or null: the token's cache row
    const double* inv_freq;    // [n] radians per token
    const int32_t* table;      // paged: [B, max_pages]
    uint32_t* status;
    int B, s, h_q, h_kv, d, dv, n, Lmax, page_size, max_pages, num_pages;
    float amplitude;
    float sign;  // +1, or -1 for the backward pass
    int width;          // units a head is walked in: the block is `lanes` heads x width units
    int lanes, vheads, vsub;  // virtual heads in all, and per value head
    int heads_per_cta;
    int tokens_per_cta;       // 1 where the heads are spread over several CTAs
};

namespace {

// Two units in flight per thread and as many blocks as the registers then allow: 2 x 4096 tokens of 32 + 8 heads of 128
// take 38.3 us (39.2 with four units and six blocks, 40.4 with eight and four), their e4m3 chunk 21.5 (25.0, 30.1).
constexpr int kRopeThreads = 128, kRopeBatch = 2;
template <typename C>
constexpr int rope_blocks() { return sizeof(C) == 1 ? 8 : 9; }  // per SM
constexpr int kRopeMaxPairs = 256;
constexpr int kRopeMaxTokens = 16, kRopeTable = 512;  // tokens per CTA, (cos, sin) pairs of its tables

template <typename T, int VE>
struct VecOf;
template <>
struct VecOf<__nv_bfloat16, 8> { using V = uint4; };
template <>
struct VecOf<float, 4> { using V = uint4; };
template <>
struct VecOf<__nv_bfloat16, 1> { using V = uint16_t; };
template <>
struct VecOf<float, 1> { using V = uint32_t; };

template <typename T, int VE>
__device__ __forceinline__ void unpack(const typename VecOf<T, VE>::V& u, float* f) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VE; ++i) f[i] = to_f32<T>(e[i]);
}

// VE values to the destination type, in one store.
template <typename C, int VE>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float* f) {
    typename VecOf<C, VE>::V u;
    C* e = reinterpret_cast<C*>(&u);
#pragma unroll
    for (int i = 0; i < VE; ++i) e[i] = from_f32<C>(f[i]);
    *reinterpret_cast<typename VecOf<C, VE>::V*>(static_cast<C*>(base) + at) = u;
}

// A per-head scale of an e4m3 cache and how to divide by it.  For scales of ordinary size x / s is the product with the
// rounded reciprocal r and one correction, q + (x - q s) r: the correctly rounded quotient (Markstein's theorem) in
// three operations; for others, and for infinite quotients, the division itself, out of line (inlined for every value
// it pushed the loop out of the instruction cache).
struct Scale {
    float s, r;
    bool plain;
};
__device__ __forceinline__ Scale make_scale(float s) {
    return {s, __frcp_rn(s), fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f};
}
__device__ __noinline__ float divide(float x, float s) { return __fdiv_rn(x, s); }
// VE values as e4m3 of value / scale, rounded to nearest even and saturated.
template <int VE>
__device__ __forceinline__ void store_e4m3(void* base, int64_t at, const float* f, const Scale& c) {
    uint8_t* p = static_cast<uint8_t*>(base) + at;
    float q[VE], most = 0.f;
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        q[i] = __fmul_rn(f[i], c.r);
        most = fmaxf(most, fabsf(q[i]));
    }
    if (c.plain && most < 0x1p100f) {
#pragma unroll
        for (int i = 0; i < VE; ++i) q[i] = __fmaf_rn(__fmaf_rn(-q[i], c.s, f[i]), c.r, q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) q[i] = divide(f[i], c.s);
    }
    if constexpr (VE == 1) {
        *p = (uint8_t)__nv_cvt_float_to_fp8(q[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint16_t b[VE / 2];
#pragma unroll
        for (int i = 0; i < VE; i += 2)
            b[i / 2] = __nv_cvt_float2_to_fp8x2(make_float2(q[i], q[i + 1]), __NV_SATFINITE, __NV_E4M3);
        if constexpr (VE == 8)
            *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(b);
        else
            *reinterpret_cast<uint32_t*>(p) = *reinterpret_cast<uint32_t*>(b);
    }
}

// Units of one head of d values: the n pairs in groups of VE, then the values past 2n in groups of 2 VE.
__host__ __device__ inline int rot_units(int n, int ve) { return (n + ve - 1) / ve; }
__host__ __device__ inline int copy_units(int values, int ve) { return (values + 2 * ve - 1) / (2 * ve); }

// Place of pair i in a token's table of n: two pairs side by side, then the same two of the next unit, so that the
// threads of consecutive units read consecutive 16 bytes (in the order of the pairs they would meet in the same banks).
template <int VE>
__device__ __forceinline__ int table_at(int i, int n) {
    return VE == 1 ? i : ((i % VE / 2) * (n / VE) + i / VE) * 2 + (i & 1);
}

// Where the CTA's tokens lie, in elements.
struct RopeTokens {
    int64_t q[kRopeMaxTokens], k[kRopeMaxTokens], v[kRopeMaxTokens], out[kRopeMaxTokens], cache[kRopeMaxTokens];
    double pos[kRopeMaxTokens];
    int live[kRopeMaxTokens], store[kRopeMaxTokens];  // a padding token is not live: its queries are 0; store: its cache row is written
};

enum RopeKind { kRotateQuery, kRotateKey, kCopyValue };

// T: element of q, k, v and q_out; C: element of the cache; VE: values per vector (1: no alignment needed).
template <typename T, typename C, int VE, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks<C>()) rope_kernel(const RopeParams p) {
    using V = typename VecOf<T, VE>::V;
    __shared__ __align__(16) float2 cs[kRopeTable];
    __shared__ RopeTokens at;
    const int tok0 = blockIdx.x * p.tokens_per_cta, n_tok = min(p.tokens_per_cta, p.B * p.s - tok0);
    if (threadIdx.x < n_tok) {
        const int i = threadIdx.x, tok = tok0 + i, b = tok / p.s, t = tok % p.s;
        int row = t, slab = b;
        bool live = true;
        if (p.lens) {
            const int L = p.lens[b];
            const bool bad = L < 0 || L > p.Lmax;
            if (bad && t == 0 && blockIdx.y == 0) atomicOr(p.status, kDevBadLength);
            row = L - p.s + t;
            live = !bad && row >= 0;
        }
        bool store = live;
        int in_slab = row;
        if (p.table && live) {
            const int page = p.table[(size_t)b * p.max_pages + row / p.page_size];
            if (page < 0 || page >= p.num_pages) {
                if (blockIdx.y == 0) atomicOr(p.status, kDevBadPage);
                store = false;
            }
            slab = page;
            in_slab = row % p.page_size;
        }
        at.q[i] = b * p.qs.b + t * p.qs.s;
        at.k[i] = b * p.ks.b + t * p.ks.s;
        at.v[i] = b * p.vs.b + t * p.vs.s;
        at.out[i] = b * p.os.b + t * p.os.s;
        at.cache[i] = slab * p.slab + in_slab * p.row;
        at.pos[i] = p.positions ? (double)p.positions[tok] : (double)row;
        at.live[i] = live;
        at.store[i] = store;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * p.n; i += kRopeThreads) {
        const int k = i / p.n;
        const double turns = at.pos[k] * (p.inv_freq[i - k * p.n] * 0.15915494309189533577);
        float sn, cn;
        sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
        cs[k * p.n + table_at<VE>(i - k * p.n, p.n)] = make_float2(cn * p.amplitude, sn * p.amplitude * p.sign);
    }
    __syncthreads();

    const int nrot = rot_units(p.n, VE), upq = nrot + copy_units(p.d - 2 * p.n, VE), upv = copy_units(p.dv, VE);
    const int lane_h = threadIdx.x / p.width;
    if (lane_h >= p.lanes) return;
    const int first_k = p.h_q, first_v = p.h_q + p.h_kv;
    const int h0 = blockIdx.y * p.heads_per_cta, h_end = min(p.vheads, h0 + p.heads_per_cta);

    // One unit of one head over all tokens of the CTA: src + from[token] -> dst + to[token]; the unit's second vector
    // lies `delta` after the first (two: it exists), in both.
    auto walk = [&](auto kind_c, const T* src, const int64_t* from, const int64_t* to, int64_t dst, int delta, bool two,
                    bool turn, int w, Scale sc) {
        constexpr RopeKind kind = decltype(kind_c)::value;
        constexpr bool E4M3 = sizeof(C) == 1 && kind != kRotateQuery;
        for (int t0 = 0; t0 < n_tok; t0 += kRopeBatch) {
            V x[kRopeBatch][2];
#pragma unroll
            for (int j = 0; j < kRopeBatch; ++j) {
                x[j][0] = V{};
                x[j][1] = V{};
                if (t0 + j < n_tok && at.live[t0 + j]) {
                    const T* a = src + from[t0 + j];
                    x[j][0] = *reinterpret_cast<const V*>(a);
                    if (two) x[j][1] = *reinterpret_cast<const V*>(a + delta);
                }
            }
#pragma unroll
            for (int j = 0; j < kRopeBatch; ++j) {
                const int k = t0 + j;
                if (k >= n_tok || (kind != kRotateQuery && !at.store[k])) continue;
                const int64_t o = to[k] + dst;
                if constexpr (kind == kCopyValue && !E4M3) {  // the same type: the bits
                    *reinterpret_cast<V*>(static_cast<C*>(p.vc) + o) = x[j][0];
                    if (two) *reinterpret_cast<V*>(static_cast<C*>(p.vc) + o + delta) = x[j][1];
                    continue;
                }
                float a[VE], c[VE];
                unpack<T, VE>(x[j][0], a);
                unpack<T, VE>(x[j][1], c);
                if (kind != kCopyValue && turn && (kind == kRotateKey || at.live[k])) {
                    float2 r[VE];
#pragma unroll
                    for (int i = 0; i < VE; i += 2) {
                        const float2* tab = cs + k * p.n + table_at<VE>(VE * w + i, p.n);
                        if constexpr (VE == 1) {
                            r[0] = tab[0];
                        } else {
                            const float4 pair = *reinterpret_cast<const float4*>(tab);
                            r[i] = make_float2(pair.x, pair.y);
                            r[i + 1] = make_float2(pair.z, pair.w);
                        }
                    }
                    if constexpr (INTER) {
                        // pairs lie side by side in the 2 VE values
                        float z[2 * VE];
#pragma unroll
                        for (int i = 0; i < VE; ++i) {
                            z[i] = a[i];
                            z[VE + i] = c[i];
                        }
#pragma unroll
                        for (int i = 0; i < VE; ++i) {
                            const float x0 = z[2 * i], x1 = z[2 * i + 1];
                            z[2 * i] = x0 * r[i].x - x1 * r[i].y;
                            z[2 * i + 1] = x1 * r[i].x + x0 * r[i].y;
                        }
#pragma unroll
                        for (int i = 0; i < VE; ++i) {
                            a[i] = z[i];
                            c[i] = z[VE + i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < VE; ++i) {
                            const float x0 = a[i], x1 = c[i];
                            a[i] = x0 * r[i].x - x1 * r[i].y;
                            c[i] = x1 * r[i].x + x0 * r[i].y;
                        }
                    }
                }
                if constexpr (E4M3) {
                    void* base = kind == kRotateKey ? p.kc : p.vc;
                    store_e4m3<VE>(base, o, a, sc);
                    if (two) store_e4m3<VE>(base, o + delta, c, sc);
                } else if constexpr (kind == kRotateKey) {
                    store_vec<C, VE>(p.kc, o, a);
                    if (two) store_vec<C, VE>(p.kc, o + delta, c);
                } else {
                    store_vec<T, VE>(p.q_out, o, a);
                    if (two) store_vec<T, VE>(p.q_out, o + delta, c);
                }
            }
        }
    };
    // one pass unless a head has more units than the block has threads
    for (int w = threadIdx.x % p.width; w < upq; w += p.width) {
        const bool turn = w < nrot;
        // columns of the unit's two vectors in a q or k head
        const int c0 = turn ? (INTER ? 2 * VE * w : VE * w) : 2 * p.n + 2 * VE * (w - nrot);
        const int delta = turn && !INTER ? p.n : VE;
        const bool two = c0 + delta < p.d;
        for (int h = h0 + lane_h; h < h_end; h += p.lanes) {
            if (h < first_k) {
                walk(std::integral_constant<RopeKind, kRotateQuery>{}, static_cast<const T*>(p.q) + h * p.qs.h + c0, at.q,
                     at.out, h * p.os.h + c0, delta, two, turn, w, Scale{});
            } else if (h < first_v) {
                const int hk = h - first_k;
                const Scale sc = sizeof(C) == 1 ? make_scale(p.k_scale[p.scale_by_head ? hk : 0]) : Scale{};
                walk(std::integral_constant<RopeKind, kRotateKey>{}, static_cast<const T*>(p.k) + hk * p.ks.h + c0, at.k,
                     at.cache, hk * p.k_head + c0, delta, two, turn, w, sc);
            } else {
                const int hv = (h - first_v) / p.vsub, wv = (h - first_v) % p.vsub * upq + w;
                if (wv >= upv) continue;
                const Scale sc = sizeof(C) == 1 ? make_scale(p.v_scale[p.scale_by_head ? hv : 0]) : Scale{};
                walk(std::integral_constant<RopeKind, kCopyValue>{}, static_cast<const T*>(p.v) + hv * p.vs.h + 2 * VE * wv,
                     at.v, at.cache, hv * p.v_head + 2 * VE * wv, VE, 2 * VE * wv + VE < p.dv, false, w, sc);
            }
        }
    }
}

bool vec_ok(const void* ptr, int bytes) { return (reinterpret_cast<uintptr_t>(ptr) % bytes) == 0; }
bool strides_ok(const RopeStrides& s, int ve) { return s.b % ve == 0 && s.h % ve == 0 && s.s % ve == 0; }

template <typename T, typename C>
cudaError_t rope_launch(RopeParams& p, bool inter, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    // the vector path wants every vector 16-byte aligned on the way in and whole on the way out; head dims and
    // strides that are not multiples of it take one value at a time
    const int cw = W * (int)sizeof(C);
    bool vec = p.n % W == 0 && p.d % W == 0 && vec_ok(p.q, 16) && vec_ok(p.q_out, 16) && strides_ok(p.qs, W) &&
               strides_ok(p.os, W);
    if (p.k) {
        vec = vec && vec_ok(p.k, 16) && strides_ok(p.ks, W) && vec_ok(p.kc, cw) && p.slab % W == 0 &&
              p.k_head % W == 0 && p.row % W == 0;
        vec = vec && p.dv % W == 0 && vec_ok(p.v, 16) && strides_ok(p.vs, W) && vec_ok(p.vc, cw) && p.v_head % W == 0;
    }
    const int ve = vec ? W : 1;
    const int upq = rot_units(p.n, ve) + copy_units(p.d - 2 * p.n, ve);
    p.width = std::min(upq, kRopeThreads);
    p.lanes = kRopeThreads / p.width;
    p.vsub = p.v ? cdiv(copy_units(p.dv, ve), upq) : 0;
    const long long vheads = p.h_q + (p.k ? (long long)p.h_kv * (1 + p.vsub) : 0);
    if (vheads >= (1ll << 30)) return cudaErrorInvalidValue;
    p.vheads = (int)vheads;
    if (!p.k) p.h_kv = 0;
    const long long tokens = (long long)p.B * p.s;
    // Many tokens: several per CTA, as many as the tables hold, such that the CTAs fill whole waves; few: one head per
    // thread, spread over the SMs.
    p.heads_per_cta = p.vheads;
    const long long slots = (long long)rope_blocks<C>() * sm_count(), most = std::min(kRopeMaxTokens, kRopeTable / p.n);
    const long long waves = (tokens + slots * most - 1) / (slots * most);
    p.tokens_per_cta = (int)((tokens + slots * waves - 1) / (slots * waves));
    if (tokens < 4LL * sm_count()) {
        const int want = (int)((4LL * sm_count() + tokens - 1) / tokens);
        p.heads_per_cta = std::max(p.lanes, cdiv(cdiv(p.vheads, want), p.lanes) * p.lanes);
    }
    p.heads_per_cta = std::max(p.heads_per_cta, cdiv(p.vheads, 32768));
    const dim3 grid((unsigned)((tokens + p.tokens_per_cta - 1) / p.tokens_per_cta), cdiv(p.vheads, p.heads_per_cta));
    TimedLaunch timer(st);
    if (vec) {
        if (inter)
            rope_kernel<T, C, W, true><<<grid, kRopeThreads, 0, st>>>(p);
        else
            rope_kernel<T, C, W, false><<<grid, kRopeThreads, 0, st>>>(p);
    } else {
        if (inter)
            rope_kernel<T, C, 1, true><<<grid, kRopeThreads, 0, st>>>(p);
        else
            rope_kernel<T, C, 1, false><<<grid, kRopeThreads, 0, st>>>(p);
    }
    timer.stop();
    return cudaPeekAtLastError();
}

bool elem_aligned(const void* ptr, int bytes) { return ptr && (reinterpret_cast<uintptr_t>(ptr) % bytes) == 0; }

// What every form checks of the sizes: rotated width d_rot of heads of d values.
lka_status_t rope_sizes(int B, int h, int s, int d, int d_rot, float amplitude) {
    if (B < 0 || h < 1 || s < 1 || d < 1 || d_rot < 2 || d_rot % 2 || d_rot > d) return LKA_ERR_INVALID_ARG;
    if (!(amplitude == amplitude) || amplitude - amplitude != 0.f) return LKA_ERR_INVALID_ARG;
    if (d_rot / 2 > kRopeMaxPairs || d > 65536 || h > 65536) return LKA_ERR_UNSUPPORTED;
    if ((long long)B * s >= (1ll << 31)) return LKA_ERR_UNSUPPORTED;
    return LKA_OK;
}

struct CacheDesc {
    void *kc, *vc;
    int64_t slab, k_head, v_head, row;
    const float *k_scale, *v_scale;
    bool fp8;
    int scale_by_head;
    int dv;
    const int32_t* table;
    int page_size, max_pages, num_pages;
};

lka_status_t append_run(const void* q, const void* k, const void* v, const int64_t* strides, const int32_t* lens,
                        const int32_t* positions, const double* inv_freq, void* q_out, int B, int h_q, int h_kv, int s,
                        int d, int d_rot, int Lmax, int interleaved, float amplitude, lka_dtype_t dtype,
                        const CacheDesc& c, void* ws, size_t ws_bytes, void* stream) {
    lka_status_t r = rope_sizes(B, h_q, s, d, d_rot, amplitude);
    if (r != LKA_OK) return r;
    if (h_kv < 1 || Lmax < 1 || c.dv < 1) return LKA_ERR_INVALID_ARG;
    if (dtype != LKA_BF16 && dtype != LKA_FP32) return LKA_ERR_UNSUPPORTED;
    if (c.fp8 && dtype != LKA_BF16) return LKA_ERR_UNSUPPORTED;
    if (h_kv > 65536 || c.dv > 65536) return LKA_ERR_UNSUPPORTED;
    if (B == 0) return LKA_OK;
    const int eb = dtype == LKA_BF16 ? 2 : 4, cb = c.fp8 ? 1 : eb;
    if (!strides || !elem_aligned(q, eb) || !elem_aligned(k, eb) || !elem_aligned(v, eb) || !elem_aligned(q_out, eb) ||
        !elem_aligned(c.kc, cb) || !elem_aligned(c.vc, cb) || !elem_aligned(lens, 4) || !elem_aligned(inv_freq, 8))
        return LKA_ERR_INVALID_ARG;
    if (c.kc == c.vc) return LKA_ERR_INVALID_ARG;  // keys and values would overwrite each other
    if (positions && !elem_aligned(positions, 4)) return LKA_ERR_INVALID_ARG;
    if (c.fp8 && (!elem_aligned(c.k_scale, 4) || !elem_aligned(c.v_scale, 4))) return LKA_ERR_INVALID_ARG;
    if (!ws || ws_bytes < kWsHeaderBytes) return LKA_ERR_WORKSPACE;
    if (!aligned16(ws)) return LKA_ERR_INVALID_ARG;
    // the caches and the rotated queries lie apart (the latent cache is one, its keys behind its values in every row)
    const size_t cache_bytes = (size_t)(c.table ? c.num_pages : B) * c.slab * cb, q_bytes = (size_t)B * h_q * s * d * eb;
    const bool one_cache = c.k_head == 0;
    if (overlap(q_out, q_bytes, c.vc, cache_bytes) ||
        (!one_cache && (overlap(q_out, q_bytes, c.kc, cache_bytes) || overlap(c.kc, cache_bytes, c.vc, cache_bytes))))
        return LKA_ERR_INVALID_ARG;
    RopeParams p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_out = q_out;
    p.qs = {strides[0], strides[1], strides[2]};
    p.ks = {strides[3], strides[4], strides[5]};
    p.vs = {strides[6], strides[7], strides[8]};
    p.os = {(int64_t)h_q * s * d, (int64_t)s * d, d};
    p.kc = c.kc;
    p.vc = c.vc;
    p.slab = c.slab;
    p.k_head = c.k_head;
    p.v_head = c.v_head;
    p.row = c.row;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.scale_by_head = c.scale_by_head;
    p.lens = lens;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.table = c.table;
    p.page_size = c.page_size;
    p.max_pages = c.max_pages;
    p.num_pages = c.num_pages;
    p.status = static_cast<uint32_t*>(ws);
    p.B = B;
    p.s = s;
    p.h_q = h_q;
    p.h_kv = h_kv;
    p.d = d;
    p.dv = c.dv;
    p.n = d_rot / 2;
    p.Lmax = Lmax;
    p.amplitude = amplitude;
    p.sign = 1.f;
    const cudaStream_t st = (cudaStream_t)stream;
    const bool inter = interleaved != 0;
    if (c.fp8) return call_status(rope_launch<__nv_bfloat16, __nv_fp8_e4m3>(p, inter, st));
    if (dtype == LKA_BF16) return call_status(rope_launch<__nv_bfloat16, __nv_bfloat16>(p, inter, st));
    return call_status(rope_launch<float, float>(p, inter, st));
}

bool rope_pages_ok(const int32_t* table, int B, int page_size, int max_pages, int num_pages) {
    return page_size >= 8 && (page_size & (page_size - 1)) == 0 && max_pages >= 1 && num_pages >= 1 &&
           (long long)max_pages * page_size < (1ll << 31) && (B <= 0 || elem_aligned(table, 4));
}

}  // namespace
}  // namespace lka

using namespace lka;

extern "C" {

lka_status_t rope_apply(const void* x, const int64_t* x_strides, const int32_t* positions, const double* inv_freq,
                        void* out, const int64_t* out_strides, int B, int h, int s, int d, int d_rot, int interleaved,
                        int backward, float amplitude, lka_dtype_t dtype, void* stream) {
    lka_status_t r = rope_sizes(B, h, s, d, d_rot, amplitude);
    if (r != LKA_OK) return r;
    if (dtype != LKA_BF16 && dtype != LKA_FP32) return LKA_ERR_UNSUPPORTED;
    if (B == 0) return LKA_OK;
    const int eb = dtype == LKA_BF16 ? 2 : 4;
    if (!x_strides || !out_strides || !elem_aligned(x, eb) || !elem_aligned(out, eb) || !elem_aligned(positions, 4) ||
        !elem_aligned(inv_freq, 8))
        return LKA_ERR_INVALID_ARG;
    RopeParams p{};
    p.q = x;
    p.q_out = out;
    p.qs = {x_strides[0], x_strides[1], x_strides[2]};
    p.os = {out_strides[0], out_strides[1], out_strides[2]};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.B = B;
    p.s = s;
    p.h_q = h;
    p.d = d;
    p.n = d_rot / 2;
    p.amplitude = amplitude;
    p.sign = backward ? -1.f : 1.f;
    const cudaStream_t st = (cudaStream_t)stream;
    if (dtype == LKA_BF16) return call_status(rope_launch<__nv_bfloat16, __nv_bfloat16>(p, interleaved != 0, st));
    return call_status(rope_launch<float, float>(p, interleaved != 0, st));
}

lka_status_t gqa_rope_append(const void* q, const void* k, const void* v, const int64_t* strides,
                             const int32_t* cache_lens, const int32_t* positions, const double* inv_freq, void* q_out,
                             void* k_cache, void* v_cache, int B, int h_q, int h_kv, int s_q, int d_h, int d_rot,
                             int Lmax, int interleaved, float amplitude, lka_dtype_t dtype, void* ws, size_t ws_bytes,
                             void* stream) {
    CacheDesc c{};
    c.kc = k_cache;
    c.vc = v_cache;
    c.slab = (long long)h_kv * Lmax * d_h;
    c.k_head = c.v_head = (long long)Lmax * d_h;
    c.row = c.dv = d_h;
    return append_run(q, k, v, strides, cache_lens, positions, inv_freq, q_out, B,
                      h_q, h_kv, s_q, d_h, d_rot, Lmax, interleaved, amplitude, dtype, c, ws, ws_bytes, stream);
}

lka_status_t gqa_rope_append_paged(const void* q, const void* k, const void* v, const int64_t* strides,
                                   const int32_t* block_table, const int32_t* cache_lens, const int32_t* positions,
                                   const double* inv_freq, void* q_out, void* k_pages, void* v_pages, int B, int h_q,
                                   int h_kv, int s_q, int d_h, int d_rot, int page_size, int max_pages, int num_pages,
                                   int interleaved, float amplitude, lka_dtype_t dtype, void* ws, size_t ws_bytes,
                                   void* stream) {
    if (!rope_pages_ok(block_table, B, page_size, max_pages, num_pages)) return LKA_ERR_INVALID_ARG;
    CacheDesc c{};
    c.kc = k_pages;
    c.vc = v_pages;
    c.slab = (long long)h_kv * page_size * d_h;
    c.k_head = c.v_head = (long long)page_size * d_h;
    c.row = c.dv = d_h;
    c.table = block_table;
    c.page_size = page_size;
    c.max_pages = max_pages;
    c.num_pages = num_pages;
    return append_run(q, k, v, strides, cache_lens, positions, inv_freq, q_out, B,
                      h_q, h_kv, s_q, d_h, d_rot, page_size * max_pages, interleaved, amplitude, dtype, c, ws,
                      ws_bytes, stream);
}

lka_status_t gqa_rope_append_fp8kv(const void* q, const void* k, const void* v, const int64_t* strides,
                                   const float* k_scale, const float* v_scale, const int32_t* cache_lens,
                                   const int32_t* positions, const double* inv_freq, void* q_out, void* k_cache,
                                   void* v_cache, int B, int h_q, int h_kv, int s_q, int d_h, int d_rot, int Lmax,
                                   int interleaved, float amplitude, void* ws, size_t ws_bytes, void* stream) {
    CacheDesc c{};
    c.kc = k_cache;
    c.vc = v_cache;
    c.slab = (long long)h_kv * Lmax * d_h;
    c.k_head = c.v_head = (long long)Lmax * d_h;
    c.row = c.dv = d_h;
    c.fp8 = true;
    c.k_scale = k_scale;
    c.v_scale = v_scale;
    c.scale_by_head = 1;
    return append_run(q, k, v, strides, cache_lens, positions, inv_freq, q_out, B,
                      h_q, h_kv, s_q, d_h, d_rot, Lmax, interleaved, amplitude, LKA_BF16, c, ws, ws_bytes, stream);
}

lka_status_t latent_rope_append(const void* q_r, const void* c_kv, const void* k_r, const int64_t* strides,
                                const int32_t* cache_lens, const int32_t* positions, const double* inv_freq,
                                void* q_out, void* latent, int B, int h_q, int s_q, int r_kv, int d_r, int Lmax,
                                int interleaved, float amplitude, lka_dtype_t dtype, void* ws, size_t ws_bytes,
                                void* stream) {
    if (r_kv < 1 || d_r < 1) return LKA_ERR_INVALID_ARG;
    const int eb = dtype == LKA_FP32 ? 4 : 2;
    CacheDesc c{};
    c.vc = latent;
    c.kc = latent ? static_cast<uint8_t*>(latent) + (size_t)r_kv * eb : nullptr;
    c.row = (long long)r_kv + d_r;
    c.slab = (long long)Lmax * c.row;
    c.dv = r_kv;
    return append_run(q_r, k_r, c_kv, strides, cache_lens, positions, inv_freq,
                      q_out, B, h_q, 1, s_q, d_r, d_r, Lmax, interleaved, amplitude, dtype, c, ws, ws_bytes, stream);
}

lka_status_t latent_rope_append_paged(const void* q_r, const void* c_kv, const void* k_r, const int64_t* strides,
                                      const int32_t* block_table, const int32_t* cache_lens, const int32_t* positions,
                                      const double* inv_freq, void* q_out, void* latent_pages, int B, int h_q, int s_q,
                                      int r_kv, int d_r, int page_size, int max_pages, int num_pages, int interleaved,
                                      float amplitude, lka_dtype_t dtype, void* ws, size_t ws_bytes, void* stream) {
    if (r_kv < 1 || d_r < 1 || !rope_pages_ok(block_table, B, page_size, max_pages, num_pages))
        return LKA_ERR_INVALID_ARG;
    const int eb = dtype == LKA_FP32 ? 4 : 2;
    CacheDesc c{};
    c.vc = latent_pages;
    c.kc = latent_pages ? static_cast<uint8_t*>(latent_pages) + (size_t)r_kv * eb : nullptr;
    c.row = (long long)r_kv + d_r;
    c.slab = (long long)page_size * c.row;
    c.dv = r_kv;
    c.table = block_table;
    c.page_size = page_size;
    c.max_pages = max_pages;
    c.num_pages = num_pages;
    return append_run(q_r, k_r, c_kv, strides, cache_lens, positions, inv_freq,
                      q_out, B, h_q, 1, s_q, d_r, d_r, page_size * max_pages, interleaved, amplitude, dtype, c, ws,
                      ws_bytes, stream);
}

lka_status_t latent_rope_append_fp8kv(const void* q_r, const void* c_kv, const void* k_r, const int64_t* strides,
                                      const float* kv_scale, const int32_t* cache_lens, const int32_t* positions,
                                      const double* inv_freq, void* q_out, void* latent, int B, int h_q, int s_q,
                                      int r_kv, int d_r, int Lmax, int interleaved, float amplitude, void* ws,
                                      size_t ws_bytes, void* stream) {
    if (r_kv < 1 || d_r < 1) return LKA_ERR_INVALID_ARG;
    CacheDesc c{};
    c.vc = latent;
    c.kc = latent ? static_cast<uint8_t*>(latent) + r_kv : nullptr;
    c.row = (long long)r_kv + d_r;
    c.slab = (long long)Lmax * c.row;
    c.dv = r_kv;
    c.fp8 = true;
    c.v_scale = kv_scale;
    c.k_scale = kv_scale ? kv_scale + 1 : nullptr;
    return append_run(q_r, k_r, c_kv, strides, cache_lens, positions, inv_freq,
                      q_out, B, h_q, 1, s_q, d_r, d_r, Lmax, interleaved, amplitude, LKA_BF16, c, ws, ws_bytes,
                      stream);
}

}  // extern "C"
