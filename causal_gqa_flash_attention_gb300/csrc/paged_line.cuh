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

}  // namespace ne
