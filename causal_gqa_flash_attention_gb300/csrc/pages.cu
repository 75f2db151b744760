// pages.cu -- pages of sequences: fork, resize and compact over a device-resident pool
// state (a reference count per page, 0 = free) and page tables.
//
// Each call is two kernels.  The first is one cluster of eight CTAs that does what needs an
// order: counts the free pages, gives every sequence its place in the line, and lists the
// pages to take and to copy, lowest free id first (prefix sums inside the CTAs, the CTAs'
// totals through distributed shared memory, cluster barriers between the steps; no CTA
// waits on a flag).  The second fills the whole GPU: table entries, counts, and the page
// contents of every layer.
//
// Bound: the bookkeeping reads the counts two or three times out of the L2 (4 bytes per
// page) and is latency otherwise: a handful of cluster barriers and dependent loads.  The
// copies read and write 2 layers x 2 x slots x Hkv x D elements at the copy bandwidth.
// Measured (GB300, both kernels): compaction of 4096 pages x 16 layers, 411 MB, 73 us, 5.6 TB/s
// (83% of the copy rate); private copies of eight sequences of 2048 x 16 layers 49 us, 5.3
// TB/s; a sweep over 1024 sequences of a pool of 131072 pages 25.5 us; 64 sequences one token
// longer 11.8 us (0.15 of it looking at the ids of the pages that stay).
#include <cooperative_groups.h>
#include "paged.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace ne {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kBulkThreads = 256;

struct ScanSmem {
    int warp[32];
    int total;
    int cta[2][kCluster][3];           // [exchange] three totals of every CTA of the cluster, written by it
};

// Inclusive sum over the CTA; the total in sm.total.
__device__ __forceinline__ int cta_scan(int x, ScanSmem& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                   // the last scan's results have been read
    if (lane == 31) sm.warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = sm.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        sm.warp[lane] = y;
        if (lane == 31) sm.total = y;
    }
    __syncthreads();
    return x + (warp ? sm.warp[warp - 1] : 0);
}

// Tells every CTA of the cluster this CTA's three totals, and waits for theirs.  ROUND: a
// kernel's exchanges have a place each, as a faster CTA may be one ahead of a reader.
template <int ROUND>
__device__ __forceinline__ void exchange(cg::cluster_group& cl, ScanSmem& sm, int x, int y, int z) {
    const int me = (int)cl.block_rank();
    if (threadIdx.x < kCluster) {
        int* dst = cl.map_shared_rank(&sm.cta[ROUND][me][0], (int)threadIdx.x);
        dst[0] = x;
        dst[1] = y;
        dst[2] = z;
    }
    cl.sync();
}
template <int ROUND>
__device__ __forceinline__ int before(const ScanSmem& sm, int me, int k) {
    int s = 0;
    for (int i = 0; i < me; ++i) s += sm.cta[ROUND][i][k];
    return s;
}
template <int ROUND>
__device__ __forceinline__ int whole(const ScanSmem& sm, int k) {
    int s = 0;
    for (int i = 0; i < kCluster; ++i) s += sm.cta[ROUND][i][k];
    return s;
}

__device__ __forceinline__ int clamp_len(int l, int cap, int* err) {
    if (l < 0 || l > cap) report_error(err, SITE_PAGED_LEN);
    return min(max(l, 0), cap);
}
__device__ __forceinline__ bool page_ok(const PagesArgs& a, int p) { return (unsigned)p < (unsigned)a.n_pages; }

// A CTA's share of [0, n) in whole groups of four.
__device__ __forceinline__ void share(int n, int me, int& lo, int& hi) {
    const int each = ((n + kCluster - 1) / kCluster + 3) / 4 * 4;
    lo = min(n, me * each);
    hi = min(n, lo + each);
}

// Four counts from i on; those at or behind n count as `pad`.
__device__ __forceinline__ int4 counts4(const int* ref, int i, int n, int pad) {
    if (i + 4 <= n) return *reinterpret_cast<const int4*>(ref + i);
    int4 v = make_int4(pad, pad, pad, pad);
    if (i < n) v.x = ref[i];
    if (i + 1 < n) v.y = ref[i + 1];
    if (i + 2 < n) v.z = ref[i + 2];
    return v;
}

// Pages that sequence i of a fork or resize takes, as the second kernel needs it again.
struct Take {
    int len;           // fork: the parent's length; resize: the old length
    int now;           // fork: the same; resize: the new length
    int parent;        // fork: the parent, -1 for an empty child
    int split;         // resize: 1 when the partly filled last page is to be copied
    int first, count;  // table entries first .. first + count - 1 get new pages (after the split one)
};
__device__ __forceinline__ Take take_fork(const PagesArgs& a, int c) {
    Take t = {0, 0, -1, 0, 0, 0};
    const int p = a.other[c];
    if (p < 0 || p >= a.B) {
        if (p != -1) report_error(a.err, SITE_PAGES_PARENT);
        return t;
    }
    t.parent = p;
    t.len = t.now = clamp_len(a.lens[p], a.cap, a.err);
    const int pages = (t.len + a.ps - 1) >> a.ps_shift;
    t.first = a.deep ? 0 : t.len >> a.ps_shift;
    t.count = pages - t.first;
    return t;
}
// `counts`: the counts after the pages behind the new lengths were given back.
__device__ __forceinline__ Take take_resize(const PagesArgs& a, int b, const int* counts) {
    Take t = {0, 0, b, 0, 0, 0};
    t.len = clamp_len(a.lens[b], a.cap, a.err);
    t.now = clamp_len(a.other[b], a.cap, a.err);
    const int low = min(t.len, t.now);
    if (low & (a.ps - 1)) {
        const int p = a.table[(size_t)b * a.W + (low >> a.ps_shift)];
        t.split = page_ok(a, p) && __ldcg(counts + p) > 1;
    }
    const int po = (t.len + a.ps - 1) >> a.ps_shift, pn = (t.now + a.ps - 1) >> a.ps_shift;
    t.first = po;
    t.count = max(0, pn - po);
    return t;
}

// Adds `by` to the counts of the pages behind the new lengths: -1 gives them back, 1 takes
// that back.  Eight lanes per sequence.
__device__ __forceinline__ void give_back(const PagesArgs& a, int gt, int GT, int by) {
    for (int b = gt >> 3; b < a.n; b += GT / 8) {
        const int old = clamp_len(a.lens[b], a.cap, nullptr), now = clamp_len(a.other[b], a.cap, nullptr);
        const int po = (old + a.ps - 1) >> a.ps_shift, pn = (now + a.ps - 1) >> a.ps_shift;
        const int* row = a.table + (size_t)b * a.W;
        for (int i0 = pn + (gt & 7); i0 < po; i0 += 32) {
            int p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = i0 + 8 * k < po ? __ldg(row + i0 + 8 * k) : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i0 + 8 * k >= po) continue;
                if (page_ok(a, p[k])) atomicAdd(a.ref_out + p[k], by);
                else report_error(a.err, SITE_PAGED_PAGE);
            }
        }
    }
}

// ------------------------------------------------------------------ first kernel
template <int OP>
__global__ void __launch_bounds__(kThreads, 1) pages_plan_kernel(const PagesArgs a) {
    __shared__ ScanSmem sm;
    cg::cluster_group cl = cg::this_cluster();
    const int me = (int)cl.block_rank(), tid = threadIdx.x, lane = tid & 31;
    const int gt = me * kThreads + tid;                    // thread of the cluster
    constexpr int GT = kCluster * kThreads;
    griddep_launch_dependents();
    griddep_wait();
    if constexpr (OP != PAGES_RESIZE) cl.sync();           // every CTA runs before one writes into its shared memory
    int lo, hi;
    share(a.n_pages, me, lo, hi);
    // The counts, where the outputs are another array.
    if (a.ref_out != a.ref && OP != PAGES_COMPACT) {
        const int4* src = reinterpret_cast<const int4*>(a.ref);
        int4* dst = reinterpret_cast<int4*>(a.ref_out);
        const int q1 = hi / 4;                             // (lo is a multiple of four)
        for (int i0 = lo / 4 + tid; i0 < q1; i0 += 4 * kThreads) {
            int4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k * kThreads < q1) v[k] = __ldg(src + i0 + k * kThreads);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i0 + k * kThreads < q1) dst[i0 + k * kThreads] = v[k];
        }
        if (tid < hi - max(lo, q1 * 4)) a.ref_out[q1 * 4 + tid] = a.ref[q1 * 4 + tid];
    }

    if constexpr (OP == PAGES_COMPACT) {
        int live = 0;
        for (int i = lo + tid * 4; i < hi; i += kThreads * 4) {
            const int4 v = counts4(a.ref, i, hi, 0);
            live += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
        }
        cta_scan(live, sm);
        exchange<0>(cl, sm, sm.total, 0, 0);
        const int n_live = whole<0>(sm, 0);
        // Live pages at or behind n_live move, free ones in front of it receive.
        int mv = 0, ho = 0;
        for (int i = lo + tid * 4; i < hi; i += kThreads * 4) {
            const int4 v = counts4(a.ref, i, hi, 0);
            const int c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                mv += i + k < hi && c[k] > 0 && i + k >= n_live;
                ho += i + k < hi && c[k] <= 0 && i + k < n_live;
            }
        }
        cta_scan(mv, sm);
        const int mv_all = sm.total;
        cta_scan(ho, sm);
        const int ho_all = sm.total;
        exchange<1>(cl, sm, mv_all, ho_all, 0);
        int mv_at = before<1>(sm, me, 0), ho_at = before<1>(sm, me, 1);
        for (int i0 = lo; i0 < hi; i0 += kThreads * 4) {
            const int i = i0 + tid * 4;
            const int4 v = counts4(a.ref, i, hi, 0);
            const int c[4] = {v.x, v.y, v.z, v.w};
            int m = 0, h = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                m += i + k < hi && c[k] > 0 && i + k >= n_live;
                h += i + k < hi && c[k] <= 0 && i + k < n_live;
            }
            int mr = mv_at + cta_scan(m, sm) - m;
            mv_at += sm.total;
            int hr = ho_at + cta_scan(h, sm) - h;
            ho_at += sm.total;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int p = i + k;
                if (p >= hi) continue;
                if (c[k] > 0 && p >= n_live) a.list[mr++].x = p;
                else if (c[k] <= 0 && p < n_live) a.free_ids[hr++] = p;
                if (!(c[k] > 0 && p >= n_live)) a.lens_out[p] = c[k] > 0 ? p : -1;   // (movers: below)
            }
        }
        cl.sync();
        const int moves = whole<1>(sm, 0);
        for (int j = gt; j < moves; j += GT) {
            const int src = __ldcg(&a.list[j].x), dst = __ldcg(a.free_ids + j);
            a.list[j] = make_int4(src, dst, a.ps, 0);
            a.lens_out[src] = dst;
        }
        if (gt == 0) {
            a.head[0] = moves;
            a.head[1] = 0;
            a.head[2] = 0;
            a.short_out[0] = n_live;
        }
        cl.sync();
        return;
    } else {
        const int* counts = OP == PAGES_FORK ? a.ref : a.ref_out;
        if constexpr (OP == PAGES_RESIZE) {
            cl.sync();                                     // the counts are copied
            give_back(a, gt, GT, -1);
            cl.sync();
        }
        // What every sequence takes, and its place in the line.
        int slo, shi;
        share(a.n, me, slo, shi);
        auto take = [&](int i) { return OP == PAGES_FORK ? take_fork(a, i) : take_resize(a, i, counts); };
        int need = 0, splits = 0;
        for (int i = slo + tid; i < shi; i += kThreads) {
            const Take t = take(i);
            need += t.split + t.count;
            splits += t.split;
        }
        // Sixteen counts per thread and pass; bit k of the mask: page i + k is free.
        auto free_mask = [&](int i) -> unsigned {
            unsigned m = 0;
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                if (i + k + 4 <= hi) {
                    const int4 v = __ldcg(reinterpret_cast<const int4*>(counts + i + k));
                    m |= ((v.x <= 0) | (v.y <= 0) << 1 | (v.z <= 0) << 2 | (v.w <= 0) << 3) << k;
                } else {
                    for (int j = 0; j < 4; ++j)
                        if (i + k + j < hi && __ldcg(counts + i + k + j) <= 0) m |= 1u << (k + j);
                }
            }
            return m;
        };
        int nfree = 0;
        for (int i = lo + tid * 16; i < hi; i += kThreads * 16) nfree += __popc(free_mask(i));
        cta_scan(need, sm);
        const int need_cta = sm.total;
        cta_scan(splits, sm);
        const int splits_cta = sm.total;
        cta_scan(nfree, sm);
        exchange<0>(cl, sm, need_cta, sm.total, splits_cta);
        const int need_all = whole<0>(sm, 0), free_all = whole<0>(sm, 1);
        const int missing = max(0, need_all - free_all);
        if (gt == 0) {
            a.head[0] = missing ? 0 : OP == PAGES_FORK ? need_all : whole<0>(sm, 2);
            a.head[1] = missing;
            a.head[2] = missing ? 0 : need_all;
            a.short_out[0] = missing;
        }
        if (missing) {
            // Nothing changes: what was given back is taken again.
            if constexpr (OP == PAGES_RESIZE) give_back(a, gt, GT, 1);
            cl.sync();
            return;
        }
        // The free pages' ids in ascending order, as many as are needed.
        int at = before<0>(sm, me, 1);
        for (int i0 = lo; i0 < hi && at < need_all; i0 += kThreads * 16) {
            const int i = i0 + tid * 16;
            unsigned m = i < hi ? free_mask(i) : 0u;
            const int f = __popc(m);
            int r = at + cta_scan(f, sm) - f;
            at += sm.total;
            for (; m && r < need_all; m &= m - 1) a.free_ids[r++] = i + __ffs(m) - 1;
        }
        // First place of every sequence; a sequence that splits a page off: its copy's, too.
        int off = before<0>(sm, me, 0), soff = before<0>(sm, me, 2);
        for (int i0 = slo; i0 < shi; i0 += kThreads) {
            const int i = i0 + tid;
            int x = 0, sp = 0;
            if (i < shi) {
                const Take t = take(i);
                x = t.split + t.count;
                sp = t.split;
            }
            const int r = off + cta_scan(x, sm) - x;
            off += sm.total;
            int rs = 0;
            if (OP == PAGES_RESIZE) {
                rs = soff + cta_scan(sp, sm) - sp;
                soff += sm.total;
            }
            if (i < shi) a.off[i] = make_int2(r, sp ? rs : -1);
        }
        cl.sync();
        // The copies.
        if constexpr (OP == PAGES_RESIZE) {
            for (int i = gt; i < a.n; i += GT) {
                const int2 o = __ldcg(a.off + i);
                if (o.y < 0) continue;
                const int low = min(clamp_len(a.lens[i], a.cap, nullptr), clamp_len(a.other[i], a.cap, nullptr));
                a.list[o.y] = make_int4(a.table[(size_t)i * a.W + (low >> a.ps_shift)], __ldcg(a.free_ids + o.x),
                                        low & (a.ps - 1), 0);
            }
        } else {
            for (int i = gt >> 5; i < a.n; i += GT / 32) {     // a warp per child
                const Take t = take_fork(a, i);
                const int r0 = __ldcg(&a.off[i].x);
                for (int k = lane; k < t.count; k += 32) {
                    const int e = t.first + k, p = a.table[(size_t)t.parent * a.W + e];
                    if (!page_ok(a, p)) report_error(a.err, SITE_PAGED_PAGE);
                    a.list[r0 + k] = make_int4(page_ok(a, p) ? p : -1, __ldcg(a.free_ids + r0 + k), min(a.ps, t.len - e * a.ps), 0);
                }
            }
        }
        cl.sync();
    }
}

// ------------------------------------------------------------------ second kernel
// Table entries, counts and page contents.
constexpr int kVec = 8;                                    // 16-byte units in flight per lane

template <int OP>
__global__ void __launch_bounds__(kBulkThreads) pages_bulk_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const long long gt = (long long)blockIdx.x * kBulkThreads + threadIdx.x, GT = (long long)gridDim.x * kBulkThreads;
    const int copies = a.head[0], missing = a.head[1], taken = a.head[2];

    // Table entries.
    const int rows = OP == PAGES_COMPACT ? a.B : a.n;
    const uint32_t cells = (uint32_t)rows * (uint32_t)a.W;     // (below 2^31)
    for (uint32_t i = (uint32_t)gt; i < cells; i += (uint32_t)GT) {
        const int s = (int)fast_div(i, a.div_w), e = (int)(i - (uint32_t)s * (uint32_t)a.W);
        if (OP == PAGES_COMPACT) {
            const int p = a.table[i];
            if (p != -1 && !page_ok(a, p)) report_error(a.err, SITE_PAGED_PAGE);   // (-1: no page)
            a.table_out[i] = page_ok(a, p) ? a.lens_out[p] : -1;
        } else if (OP == PAGES_FORK) {
            const Take t = take_fork(a, s);
            if (missing) {                                 // (its ids are looked at all the same)
                if (e < t.first + t.count && !page_ok(a, a.table[(size_t)t.parent * a.W + e])) report_error(a.err, SITE_PAGED_PAGE);
                a.table_out[i] = -1;
                if (e == 0) a.lens_out[s] = 0;
                continue;
            }
            int v = -1;
            if (e >= t.first && e < t.first + t.count) {
                v = a.free_ids[a.off[s].x + e - t.first];
            } else if (e < t.first) {                      // a shared whole page
                const int p = a.table[(size_t)t.parent * a.W + e];
                if (page_ok(a, p)) {
                    v = p;
                    atomicAdd(a.ref_out + p, 1);
                } else {
                    report_error(a.err, SITE_PAGED_PAGE);
                }
            }
            a.table_out[i] = v;
            if (e == 0) a.lens_out[s] = t.len;
        } else {
            const int v = a.table[i];
            const int2 off = a.off[s];                     // (not written, nor used, when pages are missing)
            const int old = clamp_len(a.lens[s], a.cap, nullptr), now = clamp_len(a.other[s], a.cap, nullptr);
            const int po = (old + a.ps - 1) >> a.ps_shift, pn = (now + a.ps - 1) >> a.ps_shift;
            int out = -1;
            if (e < min(po, pn)) {                         // kept (those given back: in the first kernel)
                if (!page_ok(a, v)) report_error(a.err, SITE_PAGED_PAGE);
                out = !missing && off.y >= 0 && e == (min(old, now) >> a.ps_shift) ? a.free_ids[off.x] : v;
            } else if (missing) {
                out = v;
            } else if (e >= po && e < pn) {
                out = a.free_ids[off.x + (off.y >= 0 ? 1 : 0) + e - po];
            }
            a.table_out[i] = out;
        }
    }
    // Counts.
    if (OP == PAGES_COMPACT) {
        const int n_live = a.short_out[0];
        for (long long i = gt; i < a.n_pages; i += GT) {
            const int p = (int)i, to = a.lens_out[p];
            if (to == p) {
                a.ref_out[p] = a.ref[p];
            } else if (to < 0) {
                if (p >= n_live) a.ref_out[p] = 0;         // (a free page in front receives one)
            } else {
                const int c = a.ref[p];
                a.ref_out[to] = c;
                a.ref_out[p] = 0;
            }
        }
    } else {
        for (long long i = gt; i < taken; i += GT) a.ref_out[a.free_ids[i]] = 1;
        if (OP == PAGES_RESIZE)
            for (long long i = gt; i < copies; i += GT) atomicSub(a.ref_out + a.list[i].x, 1);
    }
    // Page contents: a warp takes 32 kVec units (4 KB) of one page, layer and pool at a time,
    // all loads before the stores.  (A CTA per piece left half of it idle on 8 KB pages.)
    const int lane = threadIdx.x & 31;
    const long long warps = GT / 32;
    const int units = a.ps * a.Hkv << a.row_shift;         // of a page
    const bool head_major = a.head_stride > a.tok_stride;
    const long long items = (long long)copies * a.pieces;
    for (long long it = gt >> 5; it < items; it += warps) {
        const int c = items < (1LL << 31) ? (int)fast_div((uint32_t)it, a.div_pieces) : (int)(it / a.pieces);
        const int piece = (int)(it - (long long)c * a.pieces);
        const int part = (int)fast_div((uint32_t)piece, a.div_chunks), ch = piece - part * a.chunks;
        const int4 li = a.list[c];
        if (li.x < 0) continue;
        char* pool = (part & 1 ? a.v : a.k) + (part >> 1) * a.layer_stride;
        const char* src = pool + li.x * a.page_stride;
        char* dst = pool + li.y * a.page_stride;
        uint4 x[kVec];
        long long at[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int v = ch * 32 * kVec + k * 32 + lane;
            const int row = v >> a.row_shift, u = v & ((1 << a.row_shift) - 1);
            int tok, h;
            if (head_major) {
                h = row >> a.ps_shift;
                tok = row & (a.ps - 1);
            } else {
                tok = (int)fast_div((uint32_t)row, a.div_heads);
                h = row - tok * a.Hkv;
            }
            at[k] = v < units && tok < li.z ? tok * a.tok_stride + h * a.head_stride + u * 16 : -1;
            if (at[k] >= 0) x[k] = __ldcs(reinterpret_cast<const uint4*>(src + at[k]));
        }
#pragma unroll
        for (int k = 0; k < kVec; ++k)
            if (at[k] >= 0) __stcs(reinterpret_cast<uint4*>(dst + at[k]), x[k]);
    }
}

template <int OP>
cudaError_t launch_op(const PagesArgs& a0, cudaStream_t st) {
    PagesArgs a = a0;
    const int units = a.ps * a.Hkv << a.row_shift;
    a.chunks = (units + 32 * kVec - 1) / (32 * kVec);
    a.pieces = a.layers * 2 * a.chunks;
    a.div_pieces = make_fastdiv((uint32_t)a.pieces);
    a.div_chunks = make_fastdiv((uint32_t)a.chunks);
    a.div_heads = make_fastdiv((uint32_t)a.Hkv);
    a.div_w = make_fastdiv((uint32_t)a.W);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, pages_plan_kernel<OP>, a);
    if (e != cudaSuccess) return e;
    return launch_k(pages_bulk_kernel<OP>, dim3(8 * 152), dim3(kBulkThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_pages(PagesOp op, const PagesArgs& a, cudaStream_t st) {
    switch (op) {
        case PAGES_FORK: return launch_op<PAGES_FORK>(a, st);
        case PAGES_RESIZE: return launch_op<PAGES_RESIZE>(a, st);
        case PAGES_COMPACT: return launch_op<PAGES_COMPACT>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ne
