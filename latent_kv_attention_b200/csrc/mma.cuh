// mma.cuh -- warp-level building blocks of the cache operators: bf16
// m16n8k16 products, ldmatrix, asynchronous 16-byte copies into shared memory.
#pragma once

#include "common.cuh"

namespace lka {

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16).  Lane (g, t) = (lane / 4, lane % 4) holds
// A rows g, g + 8 at k = 2t, 2t + 1 (+ 8), B column g at the same k, D rows g, g + 8 at columns 2t, 2t + 1.
__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit values; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes to shared memory without passing through registers; `ok` false writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The row of token `tok` of one head in a cache: contiguous (table == nullptr), or pages
// [num_pages][heads][page_size].  An entry outside the pool raises kDevBadPage and gives -1.
struct CacheRows {
    const int32_t* table;  // the sequence's pages, or nullptr
    int page_size, num_pages;
    long long head_rows;   // contiguous: rows before this (sequence, head); paged: the head
    int heads;
};
__device__ __forceinline__ long long cache_row_or_none(const CacheRows& c, int tok, uint32_t* status) {
    if (!c.table) return c.head_rows + tok;
    const int page = c.table[tok / c.page_size];
    if (page < 0 || page >= c.num_pages) {
        atomicOr(status, kDevBadPage);
        return -1;
    }
    return ((long long)page * c.heads + c.head_rows) * c.page_size + tok % c.page_size;
}
// The same for reads, which take page 0 in the place of a page outside the pool.
__device__ __forceinline__ long long cache_row(const CacheRows& c, int tok, uint32_t* status) {
    const long long r = cache_row_or_none(c, tok, status);
    return r >= 0 ? r : c.head_rows * c.page_size + tok % c.page_size;
}

}  // namespace lka
