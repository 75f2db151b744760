// paged_line.cuh -- a line of work over the sequences of a call: sequence b takes cost(b) of it, and a
// warp or CTA finds the sequence that its share begins in.
#pragma once
#include "paged_sched.cuh"

namespace ne {

template <int T>
struct Line {
    long long incl[T];                 // inclusive sums of the chunk of T sequences scanned last
    long long warp_sum[T / 32];
};

// All T threads: sequences b0 .. b0 + T-1 into line.incl, behind `before`; returns their end.
template <int T, typename F>
__device__ __forceinline__ long long line_scan(Line<T>& s, int b0, int B, const F& cost, long long before) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long x = b0 + tid < B ? cost(b0 + tid) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                                       // the chunk before has been read
    if (lane == 31) s.warp_sum[warp] = x;
    __syncthreads();
    long long total = before;
    for (int i = 0; i < T / 32; ++i) {
        if (i == warp) x += total;
        total += s.warp_sum[i];
    }
    s.incl[tid] = x;
    __syncthreads();
    return total;
}

// All T threads: the whole line's length.  (Up to T sequences stay in line.incl for line_find.)
template <int T, typename F>
__device__ __forceinline__ long long line_total(Line<T>& s, int B, const F& cost) {
    long long total = 0;
    for (int b0 = 0; b0 < B; b0 += T) total = line_scan(s, b0, B, cost, total);
    return total;
}

// All T threads, after line_total; each warp with an x of its own below the total (or not, and then b
// becomes B): the sequence that holds x, and where it starts.
template <int T, typename F>
__device__ __forceinline__ void line_find(Line<T>& s, int B, const F& cost, long long x, int& b, long long& start) {
    constexpr int STEP = T / 32;
    const int lane = threadIdx.x & 31;
    static_assert(STEP <= 32, "two probes");
    b = B;
    start = 0;
    long long before = 0;
    for (int b0 = 0; b0 < B; b0 += T) {
        const long long end = B > T ? line_scan(s, b0, B, cost, before) : s.incl[T - 1];
        if (b == B && x < end) {
            const unsigned m = __ballot_sync(0xffffffffu, s.incl[lane * STEP + STEP - 1] > x);
            const int g = (__ffs(m) - 1) * STEP;
            const unsigned k = __ballot_sync(0xffffffffu, lane < STEP && s.incl[g + min(lane, STEP - 1)] > x);
            const int i = g + __ffs(k) - 1;
            b = b0 + i;
            start = i ? s.incl[i - 1] : before;
        }
        before = end;
    }
}

// Share c of C of a line, inv = line_inv(C): from x0 up to x1.
__host__ __device__ constexpr unsigned long long line_inv(int C) { return C > 1 ? ~0ull / (unsigned)C + 1 : 0; }
__device__ __forceinline__ void line_share(long long total, int c, int C, unsigned long long inv, long long& x0, long long& x1) {
    x0 = (long long)__umul64hi((unsigned long long)total, inv * c);
    x1 = c + 1 == C ? total : (long long)__umul64hi((unsigned long long)total, inv * (c + 1));
}

// off / S, and what remains in off: an estimate put right (one step off at most below 2^20), as every CTA waits
// for this and a division in 64 bits takes longer.
__device__ __forceinline__ int line_head(long long& off, long long S) {
    int h = (int)__fdividef((float)off, (float)S);
    off -= h * S;
    while (off < 0) {
        --h;
        off += S;
    }
    while (off >= S) {
        ++h;
        off -= S;
    }
    return h;
}

// One warp, up to 32 sequences: its share of the line (share(total, x0, x1)), the sequence that holds x0, and
// where it starts.
template <typename F, typename G>
__device__ __forceinline__ void line_warp(int B, const F& cost, const G& share, long long& x0, long long& x1, int& b, long long& start) {
    const int lane = threadIdx.x & 31;
    const long long mine = lane < B ? cost(lane) : 0;
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    share(__shfl_sync(0xffffffffu, x, 31), x0, x1);
    const unsigned hit = __ballot_sync(0xffffffffu, x0 < x);
    b = hit ? __ffs(hit) - 1 : B;
    start = __shfl_sync(0xffffffffu, x - mine, min(b, 31));
}

}  // namespace ne
