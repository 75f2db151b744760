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
    int cta[2][kCluster][2];           // [exchange] two totals of every CTA of the cluster, written by it
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

// Tells every CTA of the cluster this CTA's two totals, and waits for theirs.  ROUND: a
// kernel's exchanges have a place each, as a faster CTA may be one ahead of a reader.
template <int ROUND>
__device__ __forceinline__ void exchange(cg::cluster_group& cl, ScanSmem& sm, int x, int y) {
    const int me = (int)cl.block_rank();
    if (threadIdx.x < kCluster) {
        int* dst = cl.map_shared_rank(&sm.cta[ROUND][me][0], (int)threadIdx.x);
        dst[0] = x;
        dst[1] = y;
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
    int lo, hi;
    share(a.n_pages, me, lo, hi);
    // The counts, where the outputs are another array.
    if (a.ref_out != a.ref && OP != PAGES_COMPACT)
        for (int i = lo + tid; i < hi; i += kThreads) a.ref_out[i] = a.ref[i];

    if constexpr (OP == PAGES_COMPACT) {
        int live = 0;
        for (int i = lo + tid * 4; i < hi; i += kThreads * 4) {
            const int4 v = counts4(a.ref, i, hi, 0);
            live += (v.x > 0) + (v.y > 0) + (v.z > 0) + (v.w > 0);
        }
        cta_scan(live, sm);
        exchange<0>(cl, sm, sm.total, 0);
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
        exchange<1>(cl, sm, mv_all, ho_all);
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
            a.short_out[0] = n_live;
        }
        cl.sync();
        return;
    } else {
        const int* counts = OP == PAGES_FORK ? a.ref : a.ref_out;
        if constexpr (OP == PAGES_RESIZE) {
            cl.sync();                                     // the counts are copied
            // Pages behind the new length are given back: a warp per sequence.
            for (int b = gt >> 5; b < a.n; b += GT / 32) {
                const int old = clamp_len(a.lens[b], a.cap, nullptr), now = clamp_len(a.other[b], a.cap, nullptr);
                const int po = (old + a.ps - 1) >> a.ps_shift, pn = (now + a.ps - 1) >> a.ps_shift;
                for (int i = pn + lane; i < po; i += 32) {
                    const int p = a.table[(size_t)b * a.W + i];
                    if (page_ok(a, p)) atomicSub(a.ref_out + p, 1);
                    else report_error(a.err, SITE_PAGED_PAGE);
                }
            }
            cl.sync();
        }
        // What every sequence takes, and its place in the line.
        int slo, shi;
        share(a.n, me, slo, shi);
        int need = 0;
        for (int i = slo + tid; i < shi; i += kThreads) {
            const Take t = OP == PAGES_FORK ? take_fork(a, i) : take_resize(a, i, counts);
            need += t.split + t.count;
        }
        int nfree = 0;
        for (int i = lo + tid * 4; i < hi; i += kThreads * 4) {
            int4 v;
            if (i + 4 <= hi) {
                v = __ldcg(reinterpret_cast<const int4*>(counts + i));
            } else {
                v = make_int4(1, 1, 1, 1);
                if (i < hi) v.x = __ldcg(counts + i);
                if (i + 1 < hi) v.y = __ldcg(counts + i + 1);
                if (i + 2 < hi) v.z = __ldcg(counts + i + 2);
            }
            nfree += (v.x <= 0) + (v.y <= 0) + (v.z <= 0) + (v.w <= 0);
        }
        cta_scan(need, sm);
        const int need_cta = sm.total;
        cta_scan(nfree, sm);
        exchange<0>(cl, sm, need_cta, sm.total);
        const int need_all = whole<0>(sm, 0), free_all = whole<0>(sm, 1);
        const int missing = max(0, need_all - free_all);
        if (gt == 0) {
            a.head[0] = missing ? 0 : need_all;
            a.head[1] = missing;
            a.short_out[0] = missing;
        }
        if (missing) {
            // Nothing changes: what was given back is taken again.
            if constexpr (OP == PAGES_RESIZE)
                for (int b = gt >> 5; b < a.n; b += GT / 32) {
                    const int old = clamp_len(a.lens[b], a.cap, nullptr), now = clamp_len(a.other[b], a.cap, nullptr);
                    const int po = (old + a.ps - 1) >> a.ps_shift, pn = (now + a.ps - 1) >> a.ps_shift;
                    for (int i = pn + lane; i < po; i += 32) {
                        const int p = a.table[(size_t)b * a.W + i];
                        if (page_ok(a, p)) atomicAdd(a.ref_out + p, 1);
                    }
                }
            cl.sync();
            return;
        }
        // The free pages' ids in ascending order, as many as are needed.
        int at = before<0>(sm, me, 1);
        for (int i0 = lo; i0 < hi && at < need_all; i0 += kThreads * 4) {
            const int i = i0 + tid * 4;
            int c[4] = {1, 1, 1, 1};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k < hi) c[k] = __ldcg(counts + i + k);
            const int f = (c[0] <= 0) + (c[1] <= 0) + (c[2] <= 0) + (c[3] <= 0);
            int r = at + cta_scan(f, sm) - f;
            at += sm.total;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c[k] <= 0) {
                    if (r < need_all) a.free_ids[r] = i + k;
                    ++r;
                }
        }
        // Offsets of the sequences' entries.
        int off = before<0>(sm, me, 0);
        for (int i0 = slo; i0 < shi; i0 += kThreads) {
            const int i = i0 + tid;
            int x = 0;
            if (i < shi) {
                const Take t = OP == PAGES_FORK ? take_fork(a, i) : take_resize(a, i, counts);
                x = t.split + t.count;
            }
            const int r = off + cta_scan(x, sm) - x;
            off += sm.total;
            if (i < shi) a.off[i] = r;
        }
        cl.sync();
        // The list: a warp per sequence.
        for (int i = gt >> 5; i < a.n; i += GT / 32) {
            const Take t = OP == PAGES_FORK ? take_fork(a, i) : take_resize(a, i, counts);
            const int r0 = __ldcg(a.off + i);
            if (t.split && lane == 0) {
                const int low = min(t.len, t.now);
                a.list[r0] = make_int4(a.table[(size_t)i * a.W + (low >> a.ps_shift)], __ldcg(a.free_ids + r0),
                                       low & (a.ps - 1), 1);
            }
            for (int k = lane; k < t.count; k += 32) {
                const int r = r0 + t.split + k, e = t.first + k;
                int4 it = make_int4(-1, __ldcg(a.free_ids + r), 0, 0);
                if (OP == PAGES_FORK) {
                    const int p = a.table[(size_t)t.parent * a.W + e];
                    it.z = min(a.ps, t.len - e * a.ps);
                    if (page_ok(a, p)) it.x = p;
                    else report_error(a.err, SITE_PAGED_PAGE);
                }
                a.list[r] = it;
            }
        }
        cl.sync();
    }
}

// ------------------------------------------------------------------ second kernel
// Table entries, counts and page contents.
template <int OP>
__global__ void __launch_bounds__(kBulkThreads) pages_bulk_kernel(const PagesArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const long long gt = (long long)blockIdx.x * kBulkThreads + threadIdx.x, GT = (long long)gridDim.x * kBulkThreads;
    const int entries = a.head[0], missing = a.head[1];

    // Table entries.
    const long long cells = (long long)(OP == PAGES_COMPACT ? a.B : a.n) * a.W;
    for (long long i = gt; i < cells; i += GT) {
        const int s = (int)(i / a.W), e = (int)(i - (long long)s * a.W);
        if (OP == PAGES_COMPACT) {
            const int p = a.table[i];
            if (p >= a.n_pages) report_error(a.err, SITE_PAGED_PAGE);
            a.table_out[i] = page_ok(a, p) ? a.lens_out[p] : -1;
        } else if (OP == PAGES_FORK) {
            if (missing) {
                a.table_out[i] = -1;
                if (e == 0) a.lens_out[s] = 0;
                continue;
            }
            const Take t = take_fork(a, s);
            int v = -1;
            if (e >= t.first && e < t.first + t.count) {
                v = a.free_ids[a.off[s] + e - t.first];
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
            if (missing) {
                a.table_out[i] = v;
                continue;
            }
            const int old = clamp_len(a.lens[s], a.cap, nullptr), now = clamp_len(a.other[s], a.cap, nullptr);
            const int po = (old + a.ps - 1) >> a.ps_shift, pn = (now + a.ps - 1) >> a.ps_shift;
            const int low = min(old, now);
            int out = -1;
            // A split is marked in the first list entry of its sequence.
            const bool maybe = (low & (a.ps - 1)) != 0 || (e >= po && e < pn);
            const int r0 = maybe ? a.off[s] : 0;
            const int next = s + 1 < a.n ? 1 : 0;
            const bool split = (low & (a.ps - 1)) != 0 && r0 < (next ? a.off[s + 1] : entries) && a.list[r0].w == 1;
            if (e < min(po, pn)) out = split && e == (low >> a.ps_shift) ? a.list[r0].y : v;
            else if (e >= po && e < pn) out = a.list[r0 + (split ? 1 : 0) + e - po].y;
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
        for (long long i = gt; i < entries; i += GT) {
            const int4 it = a.list[i];
            a.ref_out[it.y] = 1;
            if (OP == PAGES_RESIZE && it.w == 1) atomicSub(a.ref_out + it.x, 1);
        }
    }
    // Page contents: each CTA takes 1024 16-byte units of one page, layer and pool at a time.
    const int unit_shift = a.row_shift;
    const int rows_per = a.ps * a.Hkv;
    const long long vecs = (long long)rows_per << unit_shift;      // units of a page
    const int chunks = (int)((vecs + 4 * kBulkThreads - 1) / (4 * kBulkThreads));
    const bool head_major = a.head_stride > a.tok_stride;
    const long long items = (long long)entries * a.layers * 2 * chunks;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int ch = (int)(it % chunks);
        long long rest = it / chunks;
        const int kv = (int)(rest & 1);
        rest >>= 1;
        const int layer = (int)(rest % a.layers);
        const int4 li = a.list[rest / a.layers];
        if (li.x < 0 || li.z <= 0) continue;
        char* pool = (kv ? a.v : a.k) + layer * a.layer_stride;
        const char* src = pool + li.x * a.page_stride;
        char* dst = pool + li.y * a.page_stride;
        uint4 x[4];
        long long at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const long long v = (long long)ch * 4 * kBulkThreads + k * kBulkThreads + threadIdx.x;
            const int row = (int)(v >> unit_shift), u = (int)(v & ((1 << unit_shift) - 1));
            int tok, h;
            if (head_major) {
                h = row >> a.ps_shift;
                tok = row & (a.ps - 1);
            } else {
                tok = row / a.Hkv;
                h = row - tok * a.Hkv;
            }
            at[k] = v < vecs && tok < li.z ? tok * a.tok_stride + h * a.head_stride + u * 16 : -1;
            if (at[k] >= 0) x[k] = *reinterpret_cast<const uint4*>(src + at[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (at[k] >= 0) *reinterpret_cast<uint4*>(dst + at[k]) = x[k];
    }
}

template <int OP>
cudaError_t launch_op(const PagesArgs& a, cudaStream_t st) {
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
