// pages_evict.cu -- sequences of a paged cache cut to fewer positions by accumulated attention
// weight, per layer and kv head.
//
// A row is one (layer, sequence, kv head): n slots, m of which stay.  Guarded slots (the first
// positions of the sequence and its newest) stay first, then the heaviest, ties to the lowest
// slot.  Kept slots at or behind m move into the slots below m that were given up, the j-th of the
// one kind into the j-th of the other: attention does not ask for an order (the keys are rotated
// already, positions[] remembers where a slot came from), so a step that gives up one position
// moves one row, not half the cache, and sources and targets never overlap.
//
// Two kernels.  The first, a CTA per row, finds the threshold: the weights' bits, mapped so that
// unsigned order is their order, in three digits of 11, 11 and 10 bits from the top; a histogram
// per digit in shared memory, the digit that holds the m-th largest from a suffix sum.  Warps own
// contiguous slots, so ranks among equal keys, holes and movers are one exchange of warp totals
// and a running count.  The second kernel fills the GPU with the moves.
#include "paged.h"
#include "ptx.cuh"

namespace ne {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;

// Unsigned order of the key = order of the weight (-0 counts as 0, NaN below everything).
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Lengths and offset of sequence b; `bad` collects what was out of range.
struct EvictSeq {
    int n, m, off;
};
__device__ __forceinline__ EvictSeq evict_seq(const EvictArgs& a, int b, bool& bad) {
    const int n = a.lens[b], m = a.new_lens[b], off = a.off[b];
    bad = n < 0 || n > a.T || m < 0 || off < 0 || off >= (1 << 30);
    EvictSeq s;
    s.n = min(max(n, 0), a.T);
    s.m = min(max(m, 0), s.n);
    s.off = min(max(off, 0), (1 << 30) - 1);
    return s;
}

struct SelectSmem {
    int hist[kBins];
    int warp[2][kWarps];
    int digit, rest;
};

// Exclusive sums over the warps of x (each warp's own total), all threads.
__device__ __forceinline__ int before_warp(int x, int* cnt) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) cnt[warp] = x;
    __syncthreads();
    const int v = lane < warp && lane < kWarps ? cnt[lane] : 0;
    return __reduce_add_sync(0xffffffffu, v);
}
__device__ __forceinline__ int all_warps(const int* cnt) {
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < kWarps ? cnt[lane] : 0);
}

// CACHED: the row's keys and guard bits fit into shared memory; otherwise they are formed again
// from global memory in every pass.
template <bool CACHED>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
    extern __shared__ uint32_t s_dyn[];
    __shared__ SelectSmem sm;
    uint32_t* const s_key = s_dyn;                         // [T]
    uint32_t* const s_guard = s_dyn + a.T;                 // [T / 32] (T is a multiple of 8, rounded up)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kBins; i += kThreads) sm.hist[i] = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int x = blockIdx.x, b = x / a.Hkv % a.B;
    bool bad;
    const EvictSeq q = evict_seq(a, b, bad);
    if (bad && tid == 0) report_error(a.err, SITE_PAGED_LEN);
    const float* w = a.w + (size_t)x * a.T;
    const int* pos = a.pos + (size_t)x * a.T;
    float* w_out = a.w_out + (size_t)x * a.T;
    int* pos_out = a.pos_out + (size_t)x * a.T;
    const int n = q.n, m = q.m, newest = n + q.off - a.recent;

    const int words = (n + 31) >> 5, per = (words + kWarps - 1) / kWarps;
    const int w0 = min(words, warp * per), w1 = min(words, w0 + per);
    auto place = [&](int slot) {                           // the position that a slot holds
        const int p = pos[slot];
        return p < 0 ? slot + q.off : p;
    };
    auto guarded = [&](int slot) {
        const int p = place(slot);
        return p < a.sink || p >= newest;
    };
    // Keys and guards into shared memory, guarded slots counted.
    int count = 0;
#pragma unroll 4
    for (int i = w0; i < w1; ++i) {
        const int slot = i * 32 + lane;
        const bool in = slot < n;
        const bool g = in && guarded(slot);
        if (CACHED && in) s_key[slot] = weight_key(w[slot]);
        const uint32_t gm = __ballot_sync(0xffffffffu, g);
        if (CACHED && lane == 0) s_guard[i] = gm;
        count += __popc(gm);
    }
    before_warp(count, sm.warp[0]);
    const int n_guard = all_warps(sm.warp[0]);
    if (CACHED) __syncwarp();
    auto key_of = [&](int slot) { return CACHED ? s_key[slot] : weight_key(w[slot]); };
    auto guard_of = [&](int i) -> bool {                   // of slot 32 i + lane (in front of n)
        if (CACHED) return (s_guard[i] >> lane) & 1u;
        return guarded(i * 32 + lane);
    };
    // Who competes: guarded slots among themselves where they do not all fit, else the others for
    // what the guarded leave.
    const bool crowd = n_guard > m;
    int rest = crowd ? m : m - n_guard;
    uint32_t prefix = 0, fixed = 0;
    if (rest == 0) {
        prefix = 0xffffffffu;                              // (no weight has this key)
    } else {
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            for (int i = w0; i < w1; ++i) {
                const int slot = i * 32 + lane;
                if (slot < n && guard_of(i) == crowd) {
                    const uint32_t k = key_of(slot);
                    if ((k & fixed) == prefix) atomicAdd(&sm.hist[(k >> shift) & digits], 1);
                }
            }
            __syncthreads();
            // Thread t holds four bins, the highest first; it finds the rest-th of the line in its own.
            int c[4], sum = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int* bin = &sm.hist[kBins - 1 - (4 * tid + i)];
                c[i] = *bin;
                *bin = 0;
                sum += c[i];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            int at = before_warp(__shfl_sync(0xffffffffu, incl, 31), sm.warp[1]) + incl - sum;
            if (at < rest && rest <= at + sum) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (at < rest && rest <= at + c[i]) {
                        sm.digit = kBins - 1 - (4 * tid + i);
                        sm.rest = rest - at;
                    }
                    at += c[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)sm.digit << shift;
            fixed |= digits << shift;
            rest = sm.rest;
        }
    }
    // Slots above the threshold stay, and the first `rest` of those on it.
    int equal = 0;
    for (int i = w0; i < w1; ++i) {
        const int slot = i * 32 + lane;
        equal += __popc(__ballot_sync(0xffffffffu, slot < n && guard_of(i) == crowd && key_of(slot) == prefix));
    }
    // (The two places for warp totals take turns: a warp still reading one is behind the other's barrier.)
    const int equal_before = before_warp(equal, sm.warp[1]);
    auto keep_mask = [&](int i, int& eq) -> uint32_t {     // of word i; eq counts the equal keys so far
        const int slot = i * 32 + lane;
        bool keep = false, same = false;
        if (slot < n) {
            const bool g = guard_of(i);
            const uint32_t k = key_of(slot);
            same = g == crowd && k == prefix;
            keep = g == crowd ? k > prefix : g;
        }
        const uint32_t sm_ = __ballot_sync(0xffffffffu, same);
        if (same && eq + __popc(sm_ & ((1u << lane) - 1u)) < rest) keep = true;
        eq += __popc(sm_);
        return __ballot_sync(0xffffffffu, keep);
    };
    // Slots of word i in front of m.
    auto front = [&](int i) -> uint32_t { return m >= 32 * i + 32 ? 0xffffffffu : m <= 32 * i ? 0u : (1u << (m - 32 * i)) - 1u; };
    int holes = 0, movers = 0, eq = equal_before;
    for (int i = w0; i < w1; ++i) {
        const uint32_t k = keep_mask(i, eq), f = front(i);
        holes += __popc(~k & f);
        movers += __popc(k & ~f);
    }
    int hole_at = before_warp(holes, sm.warp[0]);
    int move_at = before_warp(movers, sm.warp[1]);
    const int moves = all_warps(sm.warp[1]);
    int* dst = a.list + (size_t)x * a.T;                   // targets, then sources: T / 2 of each at most
    int* src = dst + (a.T >> 1);
    const bool same_w = a.w == a.w_out, same_pos = a.pos == a.pos_out;
    eq = equal_before;
    for (int i = w0; i < w1; ++i) {
        const int slot = i * 32 + lane;
        const uint32_t k = keep_mask(i, eq), f = front(i), below = (1u << lane) - 1u;
        const uint32_t h = ~k & f, mv = k & ~f;
        if ((h >> lane) & 1u) dst[hole_at + __popc(h & below)] = slot;
        if ((mv >> lane) & 1u) src[move_at + __popc(mv & below)] = slot;
        if ((k & f) >> lane & 1u) {
            const int p = pos[slot], r = p < 0 ? slot + q.off : p;
            if (!same_pos || p != r) pos_out[slot] = r;
            if (!same_w) w_out[slot] = w[slot];
        }
        hole_at += __popc(h);
        move_at += __popc(mv);
    }
    __syncthreads();
    for (int j = tid; j < moves; j += kThreads) {
        const int s = src[j], d = dst[j];
        w_out[d] = w[s];
        pos_out[d] = place(s);
    }
    __syncthreads();
    for (int i = m + tid; i < n; i += kThreads) {
        w_out[i] = 0.f;
        pos_out[i] = -1;
    }
    if (tid == 0) a.moves[x] = moves;
}

// Block (x, y): rows of moves y R, (y + gridDim.y) R, ... of row x, a 16-byte unit of K and of V per
// thread.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    const int x = blockIdx.x, tid = threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    const int h = x % a.Hkv, b = x / a.Hkv % a.B, l = x / a.Hkv / a.B;
    if (h == 0 && l == 0 && blockIdx.y == 0 && tid == 0) {
        bool bad;
        const EvictSeq q = evict_seq(a, b, bad);
        a.off_out[b] = q.off + q.n - q.m;
    }
    const int moves = a.moves[x];
    const int R = kMoveThreads >> a.row_shift;             // moves per pass of the block
    const int u = (tid & (a.row_vecs - 1)) * 16;
    const int* dst = a.list + (size_t)x * a.T;
    const int* src = dst + (a.T >> 1);
    const int* row = a.table + (size_t)b * a.W;
    const int mask = (1 << a.ps_shift) - 1;
    const long long base = l * a.layer_stride + h * a.head_stride + u;
    for (int j = blockIdx.y * R + (tid >> a.row_shift); j < moves; j += gridDim.y * R) {
        const int s = src[j], d = dst[j];
        const int ps = __ldg(row + (s >> a.ps_shift)), pd = __ldg(row + (d >> a.ps_shift));
        if ((unsigned)ps >= (unsigned)a.n_pages || (unsigned)pd >= (unsigned)a.n_pages) {
            report_error(a.err, SITE_PAGED_PAGE);
            continue;
        }
        const long long from = base + ps * a.page_stride + (s & mask) * a.tok_stride;
        const long long to = base + pd * a.page_stride + (d & mask) * a.tok_stride;
        const uint4 k = *reinterpret_cast<const uint4*>(a.k + from), v = *reinterpret_cast<const uint4*>(a.v + from);
        *reinterpret_cast<uint4*>(a.k + to) = k;
        *reinterpret_cast<uint4*>(a.v + to) = v;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
    const int rows = a.layers * a.B * a.Hkv;
    const size_t bytes = (size_t)a.T * 4 + ((size_t)a.T + 31) / 32 * 4;
    cudaError_t e;
    if (bytes <= 200 * 1024) {
        static std::atomic<uint64_t> done{0};
        if ((e = allow_smem(evict_select_kernel<true>, 200 * 1024, done)) != cudaSuccess) return e;
        e = launch_k(evict_select_kernel<true>, dim3(rows), dim3(kThreads), bytes, st, a);
    } else {
        e = launch_k(evict_select_kernel<false>, dim3(rows), dim3(kThreads), 0, st, a);
    }
    if (e != cudaSuccess) return e;
    // About two waves of blocks (eight to an SM), at most as many as a row has moves for.
    const int R = kMoveThreads >> a.row_shift;
    const int most = (a.T / 2 + R - 1) / R, want = (2 * 8 * 152 + rows - 1) / rows;
    const int y = most < 1 ? 1 : most < want ? most : want;
    return launch_k(evict_move_kernel, dim3(rows, y), dim3(kMoveThreads), 0, st, a);
}

}  // namespace ne
