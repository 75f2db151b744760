// paged_load.cuh -- pages into shared memory by 16-byte asynchronous copies, for the
// kernels that stream the cache through registers.
#pragma once
#include "paged.h"
#include "ptx.cuh"

namespace ne {

// 16 bytes global -> shared; zeros when `live` is false (the source is then not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Position of 16-byte unit u of row r in a tile whose rows are U units long: eight rows
// that are read together (ldmatrix, or a lane per row) fall into eight different bank
// groups.
template <int U>
__device__ __forceinline__ uint32_t tile_unit(uint32_t r, uint32_t u) {
    if constexpr (U >= 8) return r * U + (u ^ (r & 7));
    return r * U + (u ^ ((r >> 1) & 3));                   // four units: two rows fill the banks
}

// Loads positions first .. first + ROWS-1 of one head of K and V into rows r0 .. of two
// swizzled tiles; a warp's work.  Rows at or behind kv_end become zeros, so what the cache
// holds there never reaches a product.  pid: the page of position first + lane (ROWS <=
// 32), fetched by the caller one step ahead.
template <int ROWS, int U>
__device__ __forceinline__ void load_rows(uint32_t sk, uint32_t sv, const char* k, const char* v, const PagedView& c,
                                          int esize, int r0, int first, int kv_end, int pid, int lane) {
    constexpr int PER = 32 / U > 0 ? 32 / U : 1;           // rows per pass of the warp
    const int mask = (1 << c.ps_shift) - 1;
    // All rows there (any step but a sequence's last): an address per eight rows, which lie in one
    // page, and additions from it (a step of 24 rows over 16384 positions: 37.5 -> 36.1 us).
    if constexpr (ROWS >= 8 && PER <= 8) {                 // (first is a multiple of 8 then)
        if (__all_sync(0xffffffffu, pid >= 0 || lane >= ROWS)) {
            const long long tok_bytes = c.tok_stride * esize;
            const long long lane_off = (lane / U) * tok_bytes + (lane % U) * 16;
#pragma unroll
            for (int x = 0; x < ROWS; x += 8) {
                long long off = (long long)__shfl_sync(0xffffffffu, pid, x) * c.page_stride * esize +
                                ((first + x) & mask) * tok_bytes + lane_off;
#pragma unroll
                for (int i = 0; i < 8; i += PER, off += PER * tok_bytes) {
                    const uint32_t at = tile_unit<U>(r0 + x + i + lane / U, lane % U) * 16;
                    cp_async16(sk + at, k + off, true);
                    cp_async16(sv + at, v + off, true);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; i += PER) {
        const int r = i + lane / U, u = lane % U;          // (ROWS >= PER)
        const int pos = first + r;
        const int page = __shfl_sync(0xffffffffu, pid, r);
        const bool live = pos < kv_end && page >= 0;
        const long long off =
            live ? ((long long)page * c.page_stride + (long long)(pos & mask) * c.tok_stride) * esize + u * 16 : 0;
        const uint32_t at = tile_unit<U>(r0 + r, u) * 16;
        cp_async16(sk + at, k + off, live);
        cp_async16(sv + at, v + off, live);
    }
}

// 32 positions of one head of one tensor, as load_rows does it.
template <int U>
__device__ __forceinline__ void load_tile(uint32_t st, const char* src, const PagedView& c, int esize, int first,
                                          int kv_end, int pid, int lane) {
    constexpr int PER = 32 / U;
    const int mask = (1 << c.ps_shift) - 1;
#pragma unroll
    for (int i = 0; i < 32; i += PER) {
        const int r = i + lane / U, u = lane % U;
        const int pos = first + r;
        const int page = __shfl_sync(0xffffffffu, pid, r);
        const bool live = pos < kv_end && page >= 0;
        const long long off =
            live ? ((long long)page * c.page_stride + (long long)(pos & mask) * c.tok_stride) * esize + u * 16 : 0;
        cp_async16(st + tile_unit<U>(r, u) * 16, src + off, live);
    }
}

// Page of position pos of a sequence (row: its table row), -1 at or behind kv_end.  The id
// is looked at only when it is used (checked_page): a branch on it here would hold the warp
// for the load.
__device__ __forceinline__ int page_at(const PagedView& c, const int* row, int pos, int kv_end) {
    return pos < kv_end ? __ldg(row + (pos >> c.ps_shift)) : -1;
}
// The same id, -1 when it lies outside the pool (reported).
__device__ __forceinline__ int checked_page(const PagedView& c, int page, int pos, int kv_end, int* err) {
    if ((unsigned)page < (unsigned)c.n_pages) return page;
    if (pos < kv_end) report_error(err, SITE_PAGED_PAGE);
    return -1;
}

}  // namespace ne
