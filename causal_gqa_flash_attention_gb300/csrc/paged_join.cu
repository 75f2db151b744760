// paged_join.cu -- the parts of cut units put together: for every query row the parts
// (m_i, l_i, o_i) of its keys give o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i with m
// the largest m_i, and LSE = m + log2 of that sum.  Reads 4 (D + 2) bytes per row and part,
// writes a row: bound by the latency of a few dependent loads and by the kernel boundary itself
// (3 us of a step over 8 x 16384 positions, 6 us after a mixed batch of chunks, whatever the
// grid between 4 and 16 blocks per part).
// Parts are added in the order of the key axis, so the result has one value.
#include <cuda_bf16.h>
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxParts = 1024;

__device__ __forceinline__ void put(__nv_bfloat16* dst, const float4& x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void put(float* dst, const float4& x) { *reinterpret_cast<float4*>(dst) = x; }

// (m, l, o) += (m2, l2, o2), both unnormalised; m = -inf for no keys.
__device__ __forceinline__ void add_part(float& m, float& l, float4& o, float m2, float l2, const float4& o2) {
    const float mx = fmaxf(m, m2);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float w1 = ex2(m - ref), w2 = ex2(m2 - ref);
    l = l * w1 + l2 * w2;
    o.x = o.x * w1 + o2.x * w2;
    o.y = o.y * w1 + o2.y * w2;
    o.z = o.z * w1 + o2.z * w2;
    o.w = o.w * w1 + o2.w * w2;
    m = mx;
}

// Block (j, y): the unit whose first part CTA j left in its slot 1; rows y, y + gridDim.y, ...
// in turn (or that stride in groups of rows).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedAttnArgs a) {
    constexpr int LPR = D / 4;                             // lanes of a row, four elements each
    constexpr int GR = kThreads / LPR;                     // lane groups
    __shared__ int s_part[kMaxParts], s_n;
    __shared__ float s_m[GR], s_l[GR];
    __shared__ float4 s_o[kThreads];
    const int tid = threadIdx.x, j = blockIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    const int4 rec = a.part_info[j * 2 + 1];
    auto state = [&](int c) { return c < a.p.C ? a.part_info[c * 2].x : 0; };
    int st = tid < 32 ? state(j + 1 + tid) : 0;            // (beside the record's load)
    if (rec.x == 0) return;
    if (tid < 32) {
        // The parts in order: this slot, then the following CTAs' slots 0 up to the last.
        int n = 1;
        if (tid == 0) s_part[0] = j * 2 + 1;
        for (int c0 = j + 1; c0 < a.p.C; c0 += 32) {
            const int c = c0 + tid;
            if (c0 > j + 1) st = state(c);
            const unsigned ends = __ballot_sync(0xffffffffu, st == 2);
            const unsigned upto = ends ? (ends & (0u - ends)) * 2u - 1u : 0xffffffffu;   // lanes up to the first end
            const unsigned have = __ballot_sync(0xffffffffu, st != 0) & upto;
            if ((have >> tid) & 1u) s_part[n + __popc(have & ((1u << tid) - 1u))] = c * 2;
            n += __popc(have);
            if (ends) break;
        }
        if (tid == 0) s_n = n;
    }
    __syncthreads();
    const int np = s_n;
    const int ngrp = (a.G + a.p.gs - 1) / a.p.gs;
    const int hkv = rec.w / ngrp, hs = rec.w % ngrp;
    const int gs = min(a.p.gs, a.G - hs * a.p.gs);
    const int live = rec.z * gs;
    const int grp = tid / LPR, e = (tid % LPR) * 4;
    auto stored = [&](int i) { return a.p.sub == 0 || i < a.p.sub * gs ? i : i - a.p.sub * gs + 128; };
    auto finish = [&](int i, float m, float l, const float4& o) {
        const long long row = (long long)(rec.y + i / gs) * a.Hq + hkv * a.G + hs * a.p.gs + i % gs;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        put(static_cast<T*>(a.o) + row * D + e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (e == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    };
    if (live > 2 * (int)gridDim.y) {                       // many rows: one per lane group, four parts in flight
        for (int i = blockIdx.y * GR + grp; i < live; i += gridDim.y * GR) {
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < np; k0 += 4) {
                float2 ml[4];
                float4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const size_t at = (size_t)s_part[min(k0 + k, np - 1)] * a.p.rows + stored(i);
                    ml[k] = a.part_ml[at];
                    x[k] = *reinterpret_cast<const float4*>(a.part_o + at * D + e);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k0 + k < np) add_part(m, l, o, ml[k].x, ml[k].y, x[k]);
            }
            finish(i, m, l, o);
        }
        return;
    }
    for (int i = blockIdx.y; i < live; i += gridDim.y) {   // few rows: the groups share a row's parts
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int per = (np + GR - 1) / GR;
        for (int k = grp * per; k < min(np, (grp + 1) * per); ++k) {
            const size_t at = (size_t)s_part[k] * a.p.rows + stored(i);
            const float2 ml = a.part_ml[at];
            add_part(m, l, o, ml.x, ml.y, *reinterpret_cast<const float4*>(a.part_o + at * D + e));
        }
        s_o[tid] = o;
        if (e == 0) {
            s_m[grp] = m;
            s_l[grp] = l;
        }
        __syncthreads();
        if (grp == 0) {
            for (int k = 1; k < GR; ++k) add_part(m, l, o, s_m[k], s_l[k], s_o[k * LPR + tid]);
            finish(i, m, l, o);
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_paged_join(bool f32, int D, const PagedAttnArgs& a, cudaStream_t st) {
    const dim3 grid(a.p.C, a.p.rows <= 32 ? 4 : 8), block(kThreads);
    switch (D) {
        case 32:
            return f32 ? launch_k(paged_join_kernel<float, 32>, grid, block, 0, st, a)
                       : launch_k(paged_join_kernel<__nv_bfloat16, 32>, grid, block, 0, st, a);
        case 64:
            return f32 ? launch_k(paged_join_kernel<float, 64>, grid, block, 0, st, a)
                       : launch_k(paged_join_kernel<__nv_bfloat16, 64>, grid, block, 0, st, a);
        case 128: return launch_k(paged_join_kernel<__nv_bfloat16, 128>, grid, block, 0, st, a);
    }
    return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------- which kernel, which split
int paged_short_bn(int D);
int paged_f32_bn(bool many);

constexpr int kSms = 152;
static_assert(2 * kSms <= kMaxParts, "the part list holds every CTA");

PagedKind paged_kind(bool f32, int D, int G, int max_new) {
    const long long rows = (long long)G * max_new;
    if (f32) return rows <= 4 ? PAGED_F32_FEW4 : rows <= 8 ? PAGED_F32_FEW8 : rows <= 32 ? PAGED_F32_FEW16 : PAGED_F32_MANY;
    if (rows <= 16) return PAGED_SHORT16;
    return rows <= 32 || D == 32 || G > 128 ? PAGED_SHORT32 : PAGED_TILES;
}

PagedSplit paged_split(PagedKind kind, int D, int Hkv, int G, int cap) {
    PagedSplit p = {};
    auto rows = [&](int r) {
        p.rows = r;
        p.gs = G < r ? G : r;
        p.tpt = r / p.gs;
        p.hg = Hkv * ((G + p.gs - 1) / p.gs);
    };
    // A unit's ends (pages and queries of the next, the join of the warps) keep a CTA about as long as
    // 384 keys; with 128, 256 sequences of 128 to 512 positions took 29.7 us instead of 27.6.
    p.ovh = 384;
    p.w_full = p.w_part = 1;
    p.min_shift = 7;
    auto tile = [&](int keys) {
        while ((1 << p.bn_shift) < keys) ++p.bn_shift;
    };
    switch (kind) {
        case PAGED_SHORT16:
        case PAGED_SHORT32:
            rows(kind == PAGED_SHORT16 ? 16 : 32);
            tile(paged_short_bn(D));
            p.C = 2 * kSms;
            p.snap = 3;                                    // (64 sequences of 2048: 31.4 -> 30.5 us)
            p.snap_shift = p.bn_shift + 2;                 // but a quarter of a CTA's share at most
            break;
        case PAGED_F32_FEW4:
        case PAGED_F32_FEW8:
        case PAGED_F32_FEW16:
            rows(kind == PAGED_F32_FEW4 ? 4 : kind == PAGED_F32_FEW8 ? 8 : 16);
            tile(paged_f32_bn(false));
            p.C = D == 32 && kind != PAGED_F32_FEW16 ? 2 * kSms : kSms;
            break;
        case PAGED_F32_MANY:
            rows(64);
            tile(paged_f32_bn(true));
            p.C = 2 * kSms;
            break;
        case PAGED_TILES:                                  // G <= 128
            p.rows = 256;
            p.gs = G;
            p.sub = 128 / G;
            p.tpt = 2 * p.sub;
            p.hg = Hkv;
            tile(128);
            p.C = kSms;
            // A key tile takes a unit with both subtiles 1.35 us and one with a single subtile 1.0 us
            // (D 64), the ends of a unit about two tiles.
            p.w_full = 5;
            p.w_part = 4;
            p.ovh = 1024;
            p.min_shift = 11;
            p.snap = 1;                                    // (a prompt of 2048 at D 128: 35.4 -> 34.0 us)
            break;
    }
    // Contexts of at most 256 positions: a unit's keys take less time than the join would.
    p.nocut = cap <= 256;
    p.inv_C = ~0ull / (unsigned)p.C;
    p.div_tpt = make_fastdiv((uint32_t)p.tpt);
    return p;
}

size_t paged_part_bytes(const PagedSplit& p, int D) {
    const size_t parts = 2 * (size_t)p.C;
    return parts * p.rows * D * sizeof(float) + parts * p.rows * sizeof(float2) + parts * sizeof(int4);
}

}  // namespace ne
