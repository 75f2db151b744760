// paged_sched.cuh -- how the attention over a paged cache is cut into equal shares.
//
// Work units: a sequence's new tokens are cut into tiles of `tpt` tokens, and each tile and
// head group is one unit: up to `rows` query rows (token, head) that read the same keys,
// kv(r) = base + min((r + 1) tpt, n) of them in tile r (base = len - n: positions before
// the new tokens).  A unit costs ovh + kv(r) keys.  The units stand in one line, sequence
// by sequence, head group by head group, tile by tile; CTA c of C takes the interval
// [W c / C, W (c + 1) / C) of the total W and walks the units that it touches.  A unit that
// an interval's end cuts is cut at the key tile nearest to it (or not at all, where that leaves
// a part too small for its ends); both sides compute that tile alike.  So every CTA has the same
// work whatever the lengths (one sequence of 100,000 positions beside fifty of ten, a prompt
// beside single tokens), no list is built, and the split depends on the lengths alone, never on
// timing.
//
// Parts of cut units go to the workspace: a CTA has at most one part that begins inside a
// unit (its first, slot 0) and one that begins a unit and leaves its end to others (its
// last, slot 1).  The join kernel starts from the slot-1 records and walks the following
// CTAs' slot-0 records to the one marked last.
#pragma once
#include "paged.h"
#include "ptx.cuh"

namespace ne {

struct PagedSeq {
    int tok0, n, len;
};
// A member of a SHARED line: its table row, the positions in front of its first key, and whether it is a
// group's prefix (whose rows all see all keys).
struct PagedSharedSeq : PagedSeq {
    int row, skip;
    bool pre;
};
// The groups of a SHARED call, up to so many of them in shared memory.
struct PagedGroups {
    static constexpr int MAX = 16;
    int first[MAX + 1], len[MAX];      // first sequence; shared positions in use
    int tok0[MAX], n[MAX];             // rows of all its sequences
};
template <bool SH>
struct PagedSeqOf {
    typedef PagedSeq type;
};
template <>
struct PagedSeqOf<true> {
    typedef PagedSharedSeq type;
};

// Row offsets and length of sequence b as they stand in memory.
struct PagedRaw {
    int c0, c1, l;
};
__device__ __forceinline__ PagedRaw paged_raw(const PagedBatch& s, int b) {
    PagedRaw r;
    r.c0 = s.cu ? __ldg(s.cu + b) : b;
    r.c1 = s.cu ? __ldg(s.cu + b + 1) : b + 1;
    r.l = __ldg(s.lens + b);
    return r;
}
// The same, clamped to what the tensors hold; `bad` collects which argument was out of range.
__device__ __forceinline__ PagedSeq paged_clamp(const PagedBatch& s, const PagedRaw& r, int& bad) {
    PagedSeq q;
    if (r.c0 < 0 || r.c1 > s.N || r.c1 < r.c0) bad = SITE_PAGED_CU;
    q.tok0 = min(max(r.c0, 0), s.N);
    q.n = min(max(r.c1, q.tok0), s.N) - q.tok0;
    if (r.l < 0 || r.l > s.cap) bad = SITE_PAGED_LEN;
    q.len = min(max(r.l, 0), s.cap);
    return q;
}
__device__ __forceinline__ PagedSeq paged_seq(const PagedBatch& s, int b, int& bad) {
    return paged_clamp(s, paged_raw(s, b), bad);
}

// Shared positions of group r, which begins with sequence g0 (all in whole steps; 0 where there is
// nothing to share).
__device__ __forceinline__ int paged_shared(const PagedBatch& s, int r, int& g0, int& g1, int& bad) {
    g0 = __ldg(s.groups + r);
    g1 = __ldg(s.groups + r + 1);
    const int n = __ldg(s.shared + r);
    if (g0 < 0 || g1 > s.seqs || g1 < g0 || n < 0) {
        bad = SITE_PAGED_GROUP;
        g0 = g1 = 0;
        return 0;
    }
    return g1 - g0 < 2 ? 0 : min(n, min(max(__ldg(s.lens + g0), 0), s.cap)) & ~(kSharedStep - 1);
}
// Group r's prefix.
__device__ __forceinline__ PagedSharedSeq paged_prefix_seq(const PagedBatch& s, int r, int& bad) {
    PagedSharedSeq q;
    int g1;
    q.len = paged_shared(s, r, q.row, g1, bad);
    PagedRaw w;
    w.c0 = s.cu ? __ldg(s.cu + q.row) : q.row;
    w.c1 = s.cu ? __ldg(s.cu + g1) : g1;
    w.l = 0;
    const PagedSeq t = paged_clamp(s, w, bad);
    q.tok0 = t.tok0;
    q.n = q.len ? t.n : 0;
    q.skip = 0;
    q.pre = true;
    return q;
}
// Fills gs (all threads of the CTA; a barrier has to follow).
__device__ __forceinline__ void paged_load_groups(const PagedBatch& s, PagedGroups& gs) {
    if (s.R > PagedGroups::MAX) return;
    int bad = 0;
    for (int r = threadIdx.x; r < s.R; r += blockDim.x) {
        gs.first[r] = __ldg(s.groups + r);
        if (r == s.R - 1) gs.first[s.R] = __ldg(s.groups + s.R);
        const PagedSharedSeq q = paged_prefix_seq(s, r, bad);
        gs.len[r] = q.len;
        gs.tok0[r] = q.tok0;
        gs.n[r] = q.n;
    }
    if (blockIdx.x == 0 && bad) report_error(s.err, bad);
}
// What member b of a SHARED line reads of its own sequence (a prefix: nothing).
__device__ __forceinline__ PagedRaw paged_shared_raw(const PagedBatch& s, int b) {
    PagedRaw r = {0, 0, 0};
    if (b >= s.pre && b < s.B) r = paged_raw(s, b - s.pre);
    return r;
}
// Member b of a SHARED line.
__device__ __forceinline__ PagedSharedSeq paged_shared_seq(const PagedBatch& s, int b, int& bad, const PagedGroups& gs, const PagedRaw& raw) {
    PagedSharedSeq q;
    const bool near = s.R <= PagedGroups::MAX;
    if (b < s.pre) {
        if (!near) return paged_prefix_seq(s, b, bad);
        q.tok0 = gs.tok0[b];
        q.n = gs.n[b];
        q.len = gs.len[b];
        q.row = gs.first[b];
        q.skip = 0;
        q.pre = true;
        return q;
    }
    q.pre = false;
    b -= s.pre;
    int lo = -1, hi = s.R - 1;                             // the last group that begins at or before b
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((near ? gs.first[mid] : __ldg(s.groups + mid)) <= b) lo = mid;
        else hi = mid - 1;
    }
    q.skip = 0;
    if (lo >= 0 && near) {
        if (b < gs.first[lo + 1]) q.skip = gs.len[lo];
    } else if (lo >= 0) {
        int g0, g1;
        const int n = paged_shared(s, lo, g0, g1, bad);
        if (b < g1) q.skip = n;
    }
    const PagedSeq t = paged_clamp(s, raw, bad);
    if (q.skip > 0 && q.skip > t.len - t.n) bad = SITE_PAGED_GROUP;   // (new tokens among the shared positions)
    q.tok0 = t.tok0;
    q.n = t.n;
    q.len = max(0, t.len - q.skip);
    q.row = b;
    return q;
}
template <bool SH>
__device__ __forceinline__ typename PagedSeqOf<SH>::type paged_seq_of(const PagedBatch& s, int b, int& bad, const PagedGroups* gs,
                                                                      const PagedRaw* raw = nullptr) {
    if constexpr (SH) return paged_shared_seq(s, b, bad, *gs, raw ? *raw : paged_shared_raw(s, b));
    else return paged_seq(s, b, bad);
}

// Cost of tiles 0 .. r-1 of a sequence (r below its tile count, so they are full): each
// ovh + w_full max(0, base + (k+1) tpt).
__device__ __forceinline__ long long paged_prefix(int r, int base, const PagedSplit& p) {
    if (r == 0) return 0;
    const int r0 = base < 0 ? min(r, (int)fast_div((uint32_t)-base, p.div_tpt)) : 0;   // tiles without a key
    const long long m = r - r0;
    return (long long)r * p.ovh +
           p.w_full * (m * base + (long long)p.tpt * (((long long)r * (r + 1) - (long long)r0 * (r0 + 1)) / 2));
}

// The same of a member of a line: every tile of a prefix has all its keys.
__device__ __forceinline__ long long paged_prefix_of(int r, const PagedSeq& q, const PagedSplit& p) {
    return paged_prefix(r, q.len - q.n, p);
}
__device__ __forceinline__ long long paged_prefix_of(int r, const PagedSharedSeq& q, const PagedSplit& p) {
    return q.pre ? (long long)r * (p.ovh + (long long)p.w_full * q.len) : paged_prefix(r, q.len - q.n, p);
}

// Tiles of a sequence.
__device__ __forceinline__ int paged_tiles(int n, const PagedSplit& p) {
    return (int)fast_div((uint32_t)(n + p.tpt - 1), p.div_tpt);
}

// Cost of a key of a unit with ntok tokens.
__device__ __forceinline__ int paged_weight(int ntok, const PagedSplit& p) { return ntok > p.sub ? p.w_full : p.w_part; }

// Cost of one head group of a sequence.
__device__ __forceinline__ long long paged_group_cost(const PagedSeq& q, const PagedSplit& p) {
    if (q.n == 0) return 0;
    const int last = paged_tiles(q.n, p) - 1;
    return paged_prefix(last, q.len - q.n, p) + p.ovh + (long long)paged_weight(q.n - last * p.tpt, p) * q.len;
}

__device__ __forceinline__ long long paged_group_cost(const PagedSharedSeq& q, const PagedSplit& p) {
    if (!q.pre) return paged_group_cost(static_cast<const PagedSeq&>(q), p);
    if (q.n == 0) return 0;
    const int last = paged_tiles(q.n, p) - 1;
    return paged_prefix_of(last, q, p) + p.ovh + (long long)paged_weight(q.n - last * p.tpt, p) * q.len;
}

// What a CTA does with one unit: key tiles [t0, t1) of nt_keys, for tokens tok .. tok+ntok-1
// of the sequence.
struct PagedSeg {
    int b, hg;
    int tok, ntok;      // first token of the unit within the sequence, and how many
    int tok0, base;     // the sequence's first row; position of its token 0
    int len;            // the sequence's length
    int kv;             // keys the unit may see (0: rows with nothing to attend to)
    int t0, t1, nt;     // key tiles of this part; key tiles of the unit
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == nt; }
    __device__ __forceinline__ int slot() const { return t0 == 0 ? 1 : 0; }
};

struct PagedSharedSeg : PagedSeg {
    int row, skip;      // its sequence's table row, and positions in front of key 0
    bool pre;           // of a prefix
};
template <bool SH>
struct PagedSegOf {
    typedef PagedSeg type;
};
template <>
struct PagedSegOf<true> {
    typedef PagedSharedSeg type;
};
// The pages of a part's keys.
__device__ __forceinline__ const int* paged_row(const PagedAttnArgs& a, const PagedSeg& g) { return a.s.table + (size_t)g.b * a.s.W; }
__device__ __forceinline__ const int* paged_row(const PagedAttnArgs& a, const PagedSharedSeg& g) {
    return a.s.table + (size_t)g.row * a.s.W + (g.skip >> a.c.ps_shift);
}

template <bool SH>
struct PagedWalkOf {
    typedef typename PagedSegOf<SH>::type Seg;
    long long w0, w1;   // the CTA's interval
    long long cur;      // start of the current unit
    int snap;           // a cut this near to a unit's end, in tiles, moves there
    typename PagedSeqOf<SH>::type q;
    const PagedGroups* gs;   // (SHARED)
    PagedRaw ahead;     // the next sequence's, fetched while this one is walked
    int b, hg, r, nt;

    __device__ __forceinline__ void fetch(const PagedAttnArgs& a) {
        if (!SH && b + 1 < a.s.B) ahead = paged_raw(a.s, b + 1);
    }
    // Sequence b, whose values were fetched ahead.
    __device__ __forceinline__ void take(const PagedAttnArgs& a) {
        int bad = 0;
        if constexpr (SH) q = paged_seq_of<true>(a.s, b, bad, gs);
        else q = paged_clamp(a.s, ahead, bad);
        nt = paged_tiles(q.n, a.p);
        fetch(a);
    }
    __device__ __forceinline__ void load(const PagedAttnArgs& a) {
        if (!SH) ahead = paged_raw(a.s, b);
        take(a);
    }
    // From the sequence that holds w0 (q, set by the caller or by load) and where it starts.
    __device__ __forceinline__ void init(const PagedAttnArgs& a, long long w0_, long long w1_, int snap_, int b_,
                                         long long start, bool loaded = false) {
        snap = snap_;
        w0 = w0_;
        w1 = w1_;
        b = b_;
        cur = start;
        if (w0 >= w1) {
            cur = w1;
            return;
        }
        if (loaded) {
            nt = paged_tiles(q.n, a.p);
            fetch(a);
        } else {
            load(a);
        }
        const long long S = paged_group_cost(q, a.p);
        const long long off = w0 - start;
        // off / S by an estimate (off < S times the head groups, so it is off by one at most).
        hg = min(a.p.hg - 1, (int)__fdividef((float)off, (float)S));
        long long x = off - (long long)hg * S;
        if (x < 0) {
            --hg;
            x += S;
        } else if (x >= S) {
            ++hg;
            x -= S;
        }
        int lo = 0, hi = nt - 1;                           // the last tile whose start is at or before x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (paged_prefix_of(mid, q, a.p) <= x) lo = mid;
            else hi = mid - 1;
        }
        r = lo;
        cur = start + (long long)hg * S + paged_prefix_of(r, q, a.p);
    }
    // The next part of the interval, false at its end.
    __device__ __forceinline__ bool next(const PagedAttnArgs& a, Seg& g) {
        while (cur < w1) {
            bool all = false;                              // every row sees every key
            if constexpr (SH) all = q.pre;
            const int base = all ? q.len : q.len - q.n;
            const int kv = r == nt - 1 || all ? q.len : max(0, base + (r + 1) * a.p.tpt);
            const int ntok = min(a.p.tpt, q.n - r * a.p.tpt);
            const long long cost = a.p.ovh + (long long)paged_weight(ntok, a.p) * kv;
            const int ntk = (kv + (1 << a.p.bn_shift) - 1) >> a.p.bn_shift;
            // The tile nearest to each end of the interval (nocut: a whole unit goes to whoever holds
            // its middle).  In fp32: both CTAs at a cut compute it alike, it grows with x, and what
            // it is off by for units of more than 2^24 keys is a tile.
            const float per = __fdividef((float)ntk, (float)cost);
            auto cut = [&](long long x) -> int {
                if (a.p.nocut) return 2 * x >= cost ? ntk : 0;
                const int c = min(ntk, __float2int_rn(__fmul_rn((float)x, per)));
                return c <= snap ? 0 : ntk - c <= snap ? ntk : c;
            };
            g.t0 = w0 <= cur ? 0 : cut(w0 - cur);
            g.t1 = w1 >= cur + cost ? ntk : cut(w1 - cur);
            g.b = b;
            g.hg = hg;
            g.tok = r * a.p.tpt;
            g.ntok = ntok;
            g.tok0 = q.tok0;
            g.base = base;
            g.len = q.len;
            g.kv = kv;
            g.nt = ntk;
            if constexpr (SH) {
                g.row = q.row;
                g.skip = q.skip;
                g.pre = q.pre;
            }
            const bool mine = g.t0 < g.t1 || (ntk == 0 && w0 <= cur);   // a unit without keys: its rows are still written
            cur += cost;
            if (++r == nt) {
                r = 0;
                if (++hg == a.p.hg) {
                    hg = 0;
                    do ++b;
                    while (b < a.s.B && (take(a), q.n == 0));
                    if (b >= a.s.B) cur = w1 > cur ? w1 : cur;         // (the line ends here)
                }
            }
            if (mine) return true;
        }
        return false;
    }
};
typedef PagedWalkOf<false> PagedWalk;

// The CTA's share of `total`: CTA c of p.C, or of as many as have min_work each in a small call.
__device__ __forceinline__ void paged_interval(const PagedSplit& p, long long total, int c, long long& w0, long long& w1) {
    if (total < (long long)p.C << p.min_shift) {
        w0 = min((long long)c << p.min_shift, total);
        w1 = min((long long)(c + 1) << p.min_shift, total);
    } else {
        w0 = (long long)__umul64hi((unsigned long long)total, p.inv_C * c);
        w1 = c + 1 == p.C ? total : (long long)__umul64hi((unsigned long long)total, p.inv_C * (c + 1));
    }
}

// Parts of up to so many tiles are not worth their ends (a join more, a unit more to begin):
// at most p.snap, and less than the share of a CTA in a small call.
__device__ __forceinline__ int paged_snap(const PagedSplit& p, long long total) {
    return (int)min((long long)p.snap, (long long)__umul64hi((unsigned long long)total, p.inv_C) >> p.snap_shift);
}

// Shared scratch of paged_locate.
struct PagedLocate {
    long long warp_sum[32];
    long long w0, w1, start;
    int b, snap;
    PagedSharedSeq q;                  // SHARED: member b
};

// All T threads of the CTA: the total work, this CTA's interval, and the sequence that its
// start falls into.  Two passes over the lengths when they exceed T sequences (the first
// sums, the second finds), one otherwise.  (SHARED: raw is what sequence tid reads, loaded early.)
template <int T, bool SH = false>
__device__ __forceinline__ void paged_locate(const PagedAttnArgs& a, int c, PagedLocate& sm, bool report, const PagedGroups* gs = nullptr,
                                             const PagedRaw* raw = nullptr) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.s.B;
    int bad = 0;
    typename PagedSeqOf<SH>::type q = {};
    auto work = [&](int b, const PagedRaw* r) -> long long {
        if (b >= B) return 0;
        q = paged_seq_of<SH>(a.s, b, bad, gs, r);
        return paged_group_cost(q, a.p) * a.p.hg;
    };
    // Inclusive sums over the CTA; the total in sm.warp_sum[T / 32 - 1].
    auto scan = [&](long long x) -> long long {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sm.warp_sum[warp] = x;
        __syncthreads();
        if (warp == 0) {
            long long y = lane < T / 32 ? sm.warp_sum[lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += z;
            }
            sm.warp_sum[lane] = y;
        }
        __syncthreads();
        return x + (warp ? sm.warp_sum[warp - 1] : 0);
    };
    long long mine = work(tid, raw), incl = scan(mine);
    long long total = sm.warp_sum[T / 32 - 1];
    for (int b0 = T; b0 < B; b0 += T) {
        __syncthreads();
        scan(work(b0 + tid, nullptr));
        total += sm.warp_sum[T / 32 - 1];
    }
    if (tid == 0) {
        long long w0, w1;
        paged_interval(a.p, total, c, w0, w1);
        sm.w0 = w0;
        sm.w1 = w1;
        sm.start = 0;
        sm.b = 0;
        sm.snap = paged_snap(a.p, total);
    }
    __syncthreads();
    const long long w0 = sm.w0, w1 = sm.w1;
    if (w0 < w1) {
        long long before = 0;
        for (int b0 = 0; b0 < B; b0 += T) {
            if (B > T) {
                mine = work(b0 + tid, nullptr);
                __syncthreads();
                incl = scan(mine);
            }
            const long long end = before + incl;
            if (mine > 0 && w0 >= end - mine && w0 < end) {   // exactly one thread of one pass
                sm.b = b0 + tid;
                sm.start = end - mine;
                if constexpr (SH) sm.q = q;
            }
            before += sm.warp_sum[T / 32 - 1];
            if (w0 < before) break;                           // (uniform)
        }
    }
    if (report && bad) report_error(a.err, bad);
    __syncthreads();
}

// paged_locate for one warp: the walk of CTA c from its first unit on.  Written for few
// dependent steps: all CTAs wait for it at the start of a call.
template <bool SH>
__device__ __forceinline__ void paged_locate_warp(const PagedAttnArgs& a, int c, PagedWalkOf<SH>& walk, bool report,
                                                  const PagedRaw* raw = nullptr) {
    const int lane = threadIdx.x & 31, B = a.s.B;
    int bad = 0;
    typename PagedSeqOf<SH>::type q = {};
    auto work = [&](int b, const PagedRaw* r) -> long long {
        if (b >= B) return 0;
        q = paged_seq_of<SH>(a.s, b, bad, walk.gs, r);
        return paged_group_cost(q, a.p) * a.p.hg;
    };
    long long mine = work(lane, raw), total = mine;
#pragma unroll 1
    for (int b0 = 32; b0 < B; b0 += 32) total += work(b0 + lane, nullptr);
    // The sum over the warp in three limbs of 21 bits, one reduction each (units times 5 x 2^30
    // keys: below 2^60).
    const unsigned l0 = __reduce_add_sync(0xffffffffu, (unsigned)total & 0x1fffffu);
    const unsigned l1 = __reduce_add_sync(0xffffffffu, (unsigned)(total >> 21) & 0x1fffffu);
    const unsigned l2 = __reduce_add_sync(0xffffffffu, (unsigned)(total >> 42));
    total = (long long)l0 + ((long long)l1 << 21) + ((long long)l2 << 42);
    long long w0, w1, start = 0;
    paged_interval(a.p, total, c, w0, w1);
    int b = 0;
#pragma unroll 1
    for (int b0 = 0; w0 < w1 && b0 < B; b0 += 32) {
        if (B > 32) mine = work(b0 + lane, nullptr);
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, mine > 0 && w0 < start + x);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            start += __shfl_sync(0xffffffffu, x - mine, l);
            walk.q.tok0 = __shfl_sync(0xffffffffu, q.tok0, l);
            walk.q.n = __shfl_sync(0xffffffffu, q.n, l);
            walk.q.len = __shfl_sync(0xffffffffu, q.len, l);
            if constexpr (SH) {
                walk.q.row = __shfl_sync(0xffffffffu, q.row, l);
                walk.q.skip = __shfl_sync(0xffffffffu, q.skip, l);
                walk.q.pre = __shfl_sync(0xffffffffu, (int)q.pre, l);
            }
            break;
        }
        start += __shfl_sync(0xffffffffu, x, 31);
    }
    if (report && bad) report_error(a.err, bad);
    walk.init(a, w0, w1, paged_snap(a.p, total), b, start, true);
}

// The records of both slots of CTA c are written by every call (state 0: no such part).
__device__ __forceinline__ int4 paged_record(const PagedSeg& g) {
    return make_int4(g.t1 == g.nt ? 2 : 1, g.tok0 + g.tok, g.ntok, g.hg);
}

// SHARED: where the parts of a part's tokens are to be found (thread i of T, any number of them).
__device__ __forceinline__ void paged_where(const PagedAttnArgs& a, const PagedSharedSeg& g, int i, int T) {
    for (; i < g.ntok; i += T) {
        const size_t at = (size_t)(g.tok0 + g.tok + i) * a.p.hg + g.hg;
        if (g.nt == 0) a.rec_first[g.pre][at] = g.skip ? -2 : -1;
        else if (g.t0 == 0) a.rec_first[g.pre][at] = blockIdx.x | i << 16 | (g.skip ? kHasPrefix : 0);
        if (g.t1 == g.nt) a.rec_last[g.pre][at] = blockIdx.x;
    }
}

}  // namespace ne
