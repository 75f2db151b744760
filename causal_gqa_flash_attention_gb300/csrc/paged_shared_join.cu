// paged_shared_join.cu -- rows of sequences that share a prefix put together: a row's parts are those of
// its sequence's own positions and those of its group's prefix, (m_i, l_i, o_i) each;
// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i with m the largest m_i, LSE = m + log2 of that sum.
// A unit that one CTA finished left its rows in row_o, a cut one in slots of consecutive CTAs;
// rec_first and rec_last say for every token and head group which.  Reads 4 (D + 2) bytes per row and part
// out of the L2: bound by the latency of two dependent loads and by the kernel boundary.
// Parts are added in one order, whatever the timing.
#include <cuda_bf16.h>
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void put(__nv_bfloat16* dst, const float4& x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void put(float* dst, const float4& x) { *reinterpret_cast<float4*>(dst) = x; }

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

// The parts that one of the two lines holds of a row: n of them, on CTAs first, first + 1, ..., at `row` of a
// slot; or one in row_o.
struct RowParts {
    int n, first, row;
    bool whole;
};
// (Records of tokens that no sequence had, which only bad row offsets leave, are bounded here.)
__device__ __forceinline__ RowParts row_parts(const PagedAttnArgs& a, int first, int last, int g) {
    RowParts p = {0, first & 0xffff, 0, false};
    if (first < 0 || p.first >= a.p.C || last < p.first || last >= a.p.C) return p;
    const int hs = g / a.p.gs, gs = min(a.p.gs, a.G - hs * a.p.gs);
    const int i = ((first & (kHasPrefix - 1)) >> 16) * gs + g - hs * a.p.gs;
    p.row = a.p.sub == 0 || i < a.p.sub * gs ? i : i - a.p.sub * gs + 128;
    p.whole = last == p.first;
    p.n = p.row < a.p.rows ? last - p.first + 1 : 0;
    return p;
}

// LG lane groups of D / 4 lanes share a row; kThreads / (LG D / 4) rows per block.
template <typename T, int D, int LG>
__global__ void __launch_bounds__(kThreads) paged_shared_join_kernel(const PagedAttnArgs pre, const PagedAttnArgs own) {
    constexpr int LPR = D / 4, ROWS = kThreads / (LG * LPR);
    __shared__ float s_m[kThreads / LPR], s_l[kThreads / LPR];
    __shared__ float4 s_o[kThreads];
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, grp = tid / LPR, e = (tid % LPR) * 4, lg = grp % LG;
    const long long row = (long long)blockIdx.x * ROWS + grp / LG;
    // (In 32 bits: N Hq D is below 2^31.  A block's rows behind the last one look at that.)
    const uint32_t at_row = (uint32_t)min(row, (long long)own.s.N * own.Hq - 1);
    const int tok = (int)(at_row / (uint32_t)own.Hq), h = (int)(at_row - (uint32_t)tok * own.Hq);
    const int hkv = h / own.G, g = h - hkv * own.G;
    auto at = [&](const PagedAttnArgs& a) {
        const int ngrp = (a.G + a.p.gs - 1) / a.p.gs;
        return (size_t)tok * a.p.hg + hkv * ngrp + g / a.p.gs;
    };
    const size_t io = at(own), ip = at(pre);
    const int of = own.rec_first[0][io], ol = own.rec_last[0][io], pf = pre.rec_first[1][ip], pl = pre.rec_last[1][ip];
    const int c0 = own.s.cu ? max(__ldg(own.s.cu), 0) : 0, c1 = own.s.cu ? __ldg(own.s.cu + own.s.seqs) : own.s.N;
    const bool live = row == (long long)at_row && tok >= c0 && tok < min(c1, own.s.N);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        const RowParts po = row_parts(own, of, ol, g);
        RowParts pp = row_parts(pre, pf, pl, g);
        if (of == -1 || (of >= 0 && !(of & kHasPrefix))) pp.n = 0;
        auto part = [&](int k, float2& ml, float4& x) -> bool {
            const bool mine = k < po.n;
            const PagedAttnArgs& a = mine ? own : pre;
            const RowParts& p = mine ? po : pp;
            const int j = mine ? k : k - po.n, c = p.first + j;
            const size_t r = p.whole ? (size_t)row : (size_t)(2 * c + (j == 0 ? 1 : 0)) * a.p.rows + p.row;
            const int st = p.whole || j == 0 ? 1 : a.part_info[2 * c].x;
            ml = (p.whole ? a.row_ml[!mine] : a.part_ml)[r];
            x = *reinterpret_cast<const float4*>((p.whole ? a.row_o[!mine] : a.part_o) + r * D + e);
            return st != 0;
        };
        const int n = po.n + pp.n;
        for (int k0 = lg; k0 < n; k0 += 4 * LG) {          // four parts in flight
            float2 ml[4];
            float4 x[4];
            bool have[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) have[i] = k0 + i * LG < n && part(k0 + i * LG, ml[i], x[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (have[i]) add_part(m, l, o, ml[i].x, ml[i].y, x[i]);
        }
    }
    if constexpr (LG > 1) {
        s_o[tid] = o;
        if (e == 0) {
            s_m[grp] = m;
            s_l[grp] = l;
        }
        __syncthreads();
        for (int half = LG / 2; half > 0; half >>= 1) {    // (LG is a power of two)
            if (lg < half) {
                add_part(m, l, o, s_m[grp + half], s_l[grp + half], s_o[tid + half * LPR]);
                s_o[tid] = o;
                if (e == 0) {
                    s_m[grp] = m;
                    s_l[grp] = l;
                }
            }
            __syncthreads();
        }
    }
    if (live && lg == 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        put(static_cast<T*>(own.o) + row * D + e, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (e == 0) own.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <typename T, int D>
cudaError_t launch_t(const PagedAttnArgs& pre, const PagedAttnArgs& own, cudaStream_t st) {
    constexpr int GR = kThreads / (D / 4);
    const long long rows = (long long)own.s.N * own.Hq;
    // A block per row while few rows have many parts each.
    if (rows <= 4096) return launch_k(paged_shared_join_kernel<T, D, GR>, dim3((unsigned)rows), dim3(kThreads), 0, st, pre, own);
    return launch_k(paged_shared_join_kernel<T, D, 1>, dim3((unsigned)((rows + GR - 1) / GR)), dim3(kThreads), 0, st, pre, own);
}

}  // namespace

cudaError_t launch_shared_join(bool f32, int D, const PagedAttnArgs& pre, const PagedAttnArgs& own, cudaStream_t st) {
    switch (D) {
        case 32: return f32 ? launch_t<float, 32>(pre, own, st) : launch_t<__nv_bfloat16, 32>(pre, own, st);
        case 64: return f32 ? launch_t<float, 64>(pre, own, st) : launch_t<__nv_bfloat16, 64>(pre, own, st);
        case 128: return launch_t<__nv_bfloat16, 128>(pre, own, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ne
