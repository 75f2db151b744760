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
// Two kernels.  The first, a CTA per row, reads the row once into registers and finds the threshold:
// the weights' bits, mapped so that unsigned order is their order, in digits from the top (8 bits, 11 in
// the wide CTAs); a histogram per digit in shared memory, the digit that holds the m-th largest from a
// suffix sum.  Where only a few slots go, they are the minima of as many rounds instead.  Warps own
// contiguous slots, so ranks among equal keys, holes and movers are ballots and one exchange of warp
// totals.  Rows of more than 16384 slots keep their keys in shared memory, or form them again in every pass.
// The second kernel fills the GPU with the moves.
#include "paged.h"
#include "ptx.cuh"

namespace ne {
namespace {

constexpr int kThreads = 512;          // of the kernel for long rows
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kRounds = 4;             // slots of a row that are found as minima, at most
constexpr int kMoveThreads = 128;
constexpr int kMoves = 4;              // moves of a thread at a time

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

// Exclusive and whole sums of x over a CTA's warps; x the warp's own, the same in every lane.  Two places
// take turns: a warp that still reads one is behind the other's barrier.
template <int W>
struct WarpSums {
    int cnt[2][W];
    __device__ __forceinline__ void exchange(int x, int turn, int& before, int& all) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) cnt[turn][warp] = x;
        __syncthreads();
        const int v = lane < W ? cnt[turn][lane] : 0;
        before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
        all = __reduce_add_sync(0xffffffffu, v);
    }
};

// The offset of sequence b behind the cut.
__device__ __forceinline__ void put_offset(const EvictArgs& a, int b) {
    bool bad;
    const EvictSeq q = evict_seq(a, b, bad);
    a.off_out[b] = q.off + q.n - q.m;
}

// Moves of row x: a CTA of THREADS, the y-th of ny for it.  Four moves of a thread at a time: lists, table and
// rows are a chain of three loads.
template <int THREADS, typename L>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int x, int moves, const L* src, const L* dst, int y, int ny) {
    const int tid = threadIdx.x;
    const int h = x % a.Hkv, b = x / a.Hkv % a.B, l = x / a.Hkv / a.B;
    const int R = THREADS >> a.row_shift;                  // moves per pass of the CTA
    const int* row = a.table + (size_t)b * a.W;
    const int mask = (1 << a.ps_shift) - 1;
    const long long base = l * a.layer_stride + h * a.head_stride + (tid & (a.row_vecs - 1)) * 16;
    for (int j0 = y * kMoves * R + (tid >> a.row_shift); j0 < moves; j0 += ny * kMoves * R) {
        int s[kMoves], d[kMoves];
        uint4 k[kMoves], v[kMoves];
        long long from[kMoves], to[kMoves];
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            const bool in = j0 + i * R < moves;
            s[i] = in ? (int)src[j0 + i * R] : -1;
            d[i] = in ? (int)dst[j0 + i * R] : -1;
        }
#pragma unroll
        for (int i = 0; i < kMoves; ++i) {
            from[i] = to[i] = -1;
            if (s[i] < 0) continue;
            const int ps = __ldg(row + (s[i] >> a.ps_shift)), pd = __ldg(row + (d[i] >> a.ps_shift));
            if ((unsigned)ps >= (unsigned)a.n_pages || (unsigned)pd >= (unsigned)a.n_pages) {
                report_error(a.err, SITE_PAGED_PAGE);
                continue;
            }
            from[i] = base + ps * a.page_stride + (s[i] & mask) * a.tok_stride;
            to[i] = base + pd * a.page_stride + (d[i] & mask) * a.tok_stride;
        }
#pragma unroll
        for (int i = 0; i < kMoves; ++i)
            if (from[i] >= 0) {
                k[i] = *reinterpret_cast<const uint4*>(a.k + from[i]);
                v[i] = *reinterpret_cast<const uint4*>(a.v + from[i]);
            }
#pragma unroll
        for (int i = 0; i < kMoves; ++i)
            if (from[i] >= 0) {
                *reinterpret_cast<uint4*>(a.k + to[i]) = k[i];
                *reinterpret_cast<uint4*>(a.v + to[i]) = v[i];
            }
    }
}

// THREADS x KPT >= T: warp w holds slots 32 KPT w .., lane l of it slots 4 l .. 4 l + 3 of every 128.
// MOVE: the CTA moves its row's keys and values itself.
template <int THREADS, int KPT, int BITS, bool MOVE>
__global__ void __launch_bounds__(THREADS) evict_rows_kernel(const EvictArgs a) {
    constexpr int W = THREADS / 32, Q = KPT / 4, BINS = 1 << BITS, BPT = BINS / THREADS;
    static_assert(BPT >= 1 && KPT <= 32, "bins per thread, slots per mask");
    __shared__ int s_hist[BINS];
    __shared__ WarpSums<W> s_sums;
    __shared__ int2 s_min[2][W];
    __shared__ int s_digit, s_rest, s_left, s_n;
    __shared__ __align__(4) uint16_t s_hole[THREADS * KPT / 2];   // targets in order; before that, keys
    __shared__ uint16_t s_src[MOVE ? THREADS * KPT / 2 : 1];      // sources
    uint32_t* const s_key = reinterpret_cast<uint32_t*>(s_hole);
    static_assert(KPT >= 4, "a key per thread fits");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < BINS; i += THREADS) s_hist[i] = 0;
    if (tid == 0) s_n = 0;
    griddep_launch_dependents();
    griddep_wait();
    const int x = blockIdx.x, b = x / a.Hkv % a.B;
    const size_t row = (size_t)x * a.T;
    const int s0 = warp * 32 * KPT + lane * 4;             // the thread's slots: s0 + 128 i + k
    // The row (T is a multiple of 8: whole units of four), on its way while the lengths are fetched.
    float w[KPT];
    int pos[KPT];
#pragma unroll
    for (int i = 0; i < Q; ++i)
        if (s0 + 128 * i < a.T) {
            const float4 f = *reinterpret_cast<const float4*>(a.w + row + s0 + 128 * i);
            const int4 p = *reinterpret_cast<const int4*>(a.pos + row + s0 + 128 * i);
            w[4 * i] = f.x, w[4 * i + 1] = f.y, w[4 * i + 2] = f.z, w[4 * i + 3] = f.w;
            pos[4 * i] = p.x, pos[4 * i + 1] = p.y, pos[4 * i + 2] = p.z, pos[4 * i + 3] = p.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[4 * i + k] = 0.f, pos[4 * i + k] = 0;
        }
    bool bad;
    const EvictSeq q = evict_seq(a, b, bad);
    if (bad && tid == 0) report_error(a.err, SITE_PAGED_LEN);
    const int n = q.n, m = q.m, newest = n + q.off - a.recent;
    auto slot = [&](int j) { return s0 + 128 * (j >> 2) + (j & 3); };
    uint32_t live = 0, guard = 0;                          // bit j: the thread's j-th slot
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
        if (pos[j] < 0) pos[j] = slot(j) + q.off;
        const bool in = slot(j) < n;
        live |= (uint32_t)in << j;
        guard |= (uint32_t)(in && (pos[j] < a.sink || pos[j] >= newest)) << j;
    }
    int before, n_guard;
    s_sums.exchange(__reduce_add_sync(0xffffffffu, __popc(guard)), 0, before, n_guard);
    // Who competes: guarded slots among themselves where they do not all fit, else the others for
    // what the guarded leave.
    const bool crowd = n_guard > m;
    const uint32_t field = crowd ? guard : live & ~guard;
    int rest = crowd ? m : m - n_guard;
    const int gone = (crowd ? n_guard : n - n_guard) - rest;   // slots of the field that go
    uint32_t keep = field;
    if (rest == 0) {
        keep = 0;
    } else if (gone <= kRounds) {
#pragma unroll 1
        for (int r = 0; r < gone; ++r) {                   // the lowest key's last slot
            uint32_t low = 0xffffffffu;
            int at = -1;
#pragma unroll
            for (int j = 0; j < KPT; ++j) {
                const uint32_t k = weight_key(w[j]);
                if ((keep >> j & 1u) && k <= low) low = k, at = slot(j);
            }
            const uint32_t wl = __reduce_min_sync(0xffffffffu, low);
            const int wa = __reduce_max_sync(0xffffffffu, low == wl ? at : -1);
            if (lane == 0) s_min[r & 1][warp] = make_int2((int)wl, wa);
            __syncthreads();
            const int2 v = lane < W ? s_min[r & 1][lane] : make_int2(-1, -1);
            const uint32_t bl = __reduce_min_sync(0xffffffffu, (uint32_t)v.x);
            const int ba = __reduce_max_sync(0xffffffffu, (uint32_t)v.x == bl ? v.y : -1);
#pragma unroll
            for (int j = 0; j < KPT; ++j)
                if (slot(j) == ba) keep &= ~(1u << j);
        }
    } else if (gone > 0) {
        // From the first bit in which the field's keys differ: digits from the top would put the
        // few exponents that weights have into a few bins, whose atomics wait for each other.
        uint32_t low = 0xffffffffu, high = 0;
#pragma unroll
        for (int j = 0; j < KPT; ++j)
            if (field >> j & 1u) {
                const uint32_t k = weight_key(w[j]);
                low = min(low, k);
                high = max(high, k);
            }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        if (lane == 0) s_min[0][warp] = make_int2((int)low, (int)high);
        __syncthreads();
        const int2 v = lane < W ? s_min[0][lane] : make_int2(-1, 0);
        low = __reduce_min_sync(0xffffffffu, (uint32_t)v.x);
        high = __reduce_max_sync(0xffffffffu, (uint32_t)v.y);
        const int top = 32 - __clz((int)(low ^ high));     // bits below the common ones
        uint32_t fixed = top == 32 ? 0u : ~((1u << top) - 1u), prefix = high & fixed, mine = 0;
        int left = -1;                                     // keys that still compete, one per thread (-1: in their places)
#pragma unroll 1
        for (int shift = max(0, top - BITS); top > 0; shift = max(0, shift - BITS)) {
            // (The last digit may overlap the one before: its bits above are those found already.)
            const uint32_t digits = BINS - 1;
            if (left >= 0) {
                if (tid < left && (mine & fixed) == prefix) atomicAdd(&s_hist[(mine >> shift) & digits], 1);
            } else {
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    const uint32_t k = weight_key(w[j]);
                    if ((field >> j & 1u) && (k & fixed) == prefix) atomicAdd(&s_hist[(k >> shift) & digits], 1);
                }
            }
            __syncthreads();
            // A thread holds BPT bins, the first thread the highest; it finds the rest-th of the line in its own.
            int c[BPT], sum = 0;
#pragma unroll
            for (int i = 0; i < BPT; ++i) {
                int* bin = &s_hist[BINS - 1 - (BPT * tid + i)];
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
            int at, all;
            s_sums.exchange(__shfl_sync(0xffffffffu, incl, 31), 1, at, all);
            at += incl - sum;
            if (at < rest && rest <= at + sum) {
#pragma unroll
                for (int i = 0; i < BPT; ++i) {
                    if (at < rest && rest <= at + c[i]) {
                        s_digit = BINS - 1 - (BPT * tid + i);
                        s_rest = rest - at;
                        s_left = c[i];
                    }
                    at += c[i];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_digit << shift;
            fixed |= digits << shift;
            rest = s_rest;
            if (shift == 0) break;
            if (left < 0 && s_left <= THREADS) {           // few are left: one per thread from here on
                left = s_left;
#pragma unroll
                for (int j = 0; j < KPT; ++j) {
                    const uint32_t k = weight_key(w[j]);
                    if ((field >> j & 1u) && (k & fixed) == prefix) s_key[atomicAdd(&s_n, 1)] = k;
                }
                __syncthreads();
                if (tid < left) mine = s_key[tid];
            }
        }
        // Slots above the threshold stay, and the first `rest` of those on it.
        uint32_t same = 0;
        keep = 0;
#pragma unroll
        for (int j = 0; j < KPT; ++j) {
            const uint32_t k = weight_key(w[j]);
            same |= (uint32_t)(k == prefix) << j;
            keep |= (uint32_t)(k > prefix) << j;
        }
        same &= field;
        keep &= field;
        int eq, all;
        s_sums.exchange(__reduce_add_sync(0xffffffffu, __popc(same)), 0, eq, all);
        if (all == rest) {
            keep |= same;
        } else {
            const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                uint32_t v[4];
                int at = eq;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = __ballot_sync(0xffffffffu, same >> (4 * i + k) & 1u);
                    at += __popc(v[k] & lower);
                    eq += __popc(v[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (same >> (4 * i + k) & 1u) {
                        if (at < rest) keep |= 1u << (4 * i + k);
                        ++at;
                    }
            }
        }
    }
    if (!crowd) keep |= guard;
    uint32_t front = 0;                                    // slots below m
#pragma unroll
    for (int j = 0; j < KPT; ++j) front |= (uint32_t)(slot(j) < m) << j;
    const uint32_t hole = front & ~keep, move = keep & ~front;
    int hole_at, move_at, holes, moves;
    s_sums.exchange(__reduce_add_sync(0xffffffffu, __popc(hole)), 1, hole_at, holes);
    s_sums.exchange(__reduce_add_sync(0xffffffffu, __popc(move)), 0, move_at, moves);
    int* dst = a.list + row;                               // targets, then sources: T / 2 of each at most
    int* src = dst + (a.T >> 1);
    const uint32_t lower = (1u << lane) - 1u;
    int first[Q];                                          // rank of the thread's first mover of group i
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        first[i] = 0;
        if (moves == 0) continue;
        const int g0 = warp * 32 * KPT + 128 * i;
        if (g0 < m) {
            int at = hole_at;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t v = __ballot_sync(0xffffffffu, hole >> (4 * i + k) & 1u);
                at += __popc(v & lower);
                hole_at += __popc(v);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (hole >> (4 * i + k) & 1u) {
                    s_hole[at] = (uint16_t)slot(4 * i + k);
                    if (!MOVE) dst[at] = slot(4 * i + k);
                    ++at;
                }
        }
        if (g0 + 128 > m && g0 < n) {
            first[i] = move_at;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t v = __ballot_sync(0xffffffffu, move >> (4 * i + k) & 1u);
                first[i] += __popc(v & lower);
                move_at += __popc(v);
            }
        }
    }
    __syncthreads();                                       // the targets are there
    float* w_out = a.w_out + row;
    int* pos_out = a.pos_out + row;
    const bool same_w = a.w == a.w_out;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        int at = first[i];
        const int s4 = slot(4 * i);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (move >> (4 * i + k) & 1u) {
                const int d = s_hole[at];
                if (MOVE) s_src[at] = (uint16_t)(s4 + k);
                else src[at] = s4 + k;
                ++at;
                w_out[d] = w[4 * i + k];
                pos_out[d] = pos[4 * i + k];
            }
        const uint32_t f = front >> 4 * i & 15u, l = live >> 4 * i & 15u, kp = keep >> 4 * i & f;
        if (f == 0 && l == 15) {                           // four that go (or have moved), four that stay, or a mixture
            *reinterpret_cast<float4*>(w_out + s4) = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<int4*>(pos_out + s4) = make_int4(-1, -1, -1, -1);
        } else if (kp == 15) {
            if (!same_w) *reinterpret_cast<float4*>(w_out + s4) = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            *reinterpret_cast<int4*>(pos_out + s4) = make_int4(pos[4 * i], pos[4 * i + 1], pos[4 * i + 2], pos[4 * i + 3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kp >> k & 1u) {
                    if (!same_w) w_out[s4 + k] = w[4 * i + k];
                    pos_out[s4 + k] = pos[4 * i + k];
                } else if (l & ~f & 1u << k) {
                    w_out[s4 + k] = 0.f;
                    pos_out[s4 + k] = -1;
                }
            }
        }
    }
    if constexpr (MOVE) {
        if (x < a.Hkv * a.B && x % a.Hkv == 0 && tid == 0 && a.off != a.off_out) a.off_out[b] = q.off + n - m;
        __syncthreads();                                   // the sources are there
        move_rows<THREADS>(a, x, moves, s_src, s_hole, 0, 1);
    } else if (tid == 0) {
        a.moves[x] = moves;
    }
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

// Block (x, y): moves y kMoves R .. of row x, then gridDim.y blocks further on; a 16-byte unit of K and of V
// per thread and move.
__global__ void __launch_bounds__(kMoveThreads, 6) evict_move_kernel(const EvictArgs a) {
    const int x = blockIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    if (x < a.Hkv * a.B && x % a.Hkv == 0 && blockIdx.y == 0 && threadIdx.x == 0) put_offset(a, x / a.Hkv);
    const int* dst = a.list + (size_t)x * a.T;
    move_rows<kMoveThreads>(a, x, a.moves[x], dst + (a.T >> 1), dst, blockIdx.y, gridDim.y);
}

// pos_offset_out in its input's place: behind the kernel whose rows all read it.
__global__ void evict_offset_kernel(const EvictArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < a.B) put_offset(a, b);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
    const int rows = a.layers * a.B * a.Hkv;
    // The narrowest CTA that holds a row in registers.
    const size_t bytes = (size_t)a.T * 4 + ((size_t)a.T + 31) / 32 * 4;
    cudaError_t e;
    if (a.T <= 1024) {
        // Up to 512 moves per row: a launch for them costs more than it spreads (16 layers x 16 sequences of
        // 513 slots, one given up each: 7.5 us with, 6.3 without).
        e = launch_k(evict_rows_kernel<128, 8, 8, true>, dim3(rows), dim3(128), 0, st, a);
        if (e != cudaSuccess || a.off != a.off_out) return e;
        return launch_k(evict_offset_kernel, dim3((a.B + 255) / 256), dim3(256), 0, st, a);
    } else if (a.T <= 2048) {
        e = launch_k(evict_rows_kernel<256, 8, 8, false>, dim3(rows), dim3(256), 0, st, a);
    } else if (a.T <= 4096) {
        e = launch_k(evict_rows_kernel<512, 8, 11, false>, dim3(rows), dim3(512), 0, st, a);
    } else if (a.T <= 8192) {
        e = launch_k(evict_rows_kernel<1024, 8, 11, false>, dim3(rows), dim3(1024), 0, st, a);
    } else if (a.T <= 16384) {
        e = launch_k(evict_rows_kernel<1024, 16, 11, false>, dim3(rows), dim3(1024), 0, st, a);
    } else if (bytes <= 200 * 1024) {
        static std::atomic<uint64_t> done{0};
        if ((e = allow_smem(evict_select_kernel<true>, 200 * 1024, done)) != cudaSuccess) return e;
        e = launch_k(evict_select_kernel<true>, dim3(rows), dim3(kThreads), bytes, st, a);
    } else {
        e = launch_k(evict_select_kernel<false>, dim3(rows), dim3(kThreads), 0, st, a);
    }
    if (e != cudaSuccess) return e;
    // Up to three waves of blocks (eight to an SM: rows differ in their moves), each of them with at
    // least four passes' worth where a row moves all it can.
    const int R = (kMoveThreads >> a.row_shift) * kMoves;
    const int most = (a.T / 2 + 4 * R - 1) / (4 * R), want = 3 * 8 * 152 / rows;
    const int y = most < 1 || want < 1 ? 1 : most < want ? most : want;
    return launch_k(evict_move_kernel, dim3(rows, y), dim3(kMoveThreads), 0, st, a);
}

}  // namespace ne
