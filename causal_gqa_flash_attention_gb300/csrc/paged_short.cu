// paged_short.cu -- attention over the paged cache for few query rows per kv head (one or
// a few new tokens), bf16.
//
// With R = tokens x query heads of a kv head in a unit (up to 16 or 32), a key and a value
// row (4 D bytes) serve R dot products: 4 D R flops per 4 D bytes, so up to 32 flops per
// byte against the machine's ~280: the read of the cache bounds it.  The products still go
// through tensor instructions (mma.sync m16n8k16, all R rows at once): on the CUDA cores
// they would cost more issue slots than the loads leave (the contiguous decode kernel,
// which also rotates its keys, runs at half the copy bandwidth because of that), while
// tcgen05 needs 128-row tiles and a TMEM round trip for the 3 to 32 rows there are.
//
// Every warp streams on its own: it takes every fourth KT-key step of the CTA's key range
// through a private ring of three stages (16-byte cp.async, page ids fetched two steps ahead and
// looked at only when they are used: a branch on one at its load holds the warp for it), with its
// own running max, sum and output, so the loop has no barrier at all.  The four warps are
// joined through shared memory at the end of a unit, beside the next unit's first loads.  The
// ring keeps 2 x 8 KB of loads per warp in flight, 128 KB per SM: bandwidth times latency is
// about 45 KB.
//
// Measured (GB300): 8 sequences x 65536 positions, 12/4 heads of 64, 86-88 us with the join (by
// GPU), 6.1-6.3 TB/s (91% of the 6.78 TB/s copy); x 16384 29.5-30.0 us (19.8 at the copy rate): 2.3
// us to find the shares, 21 us of reading, the spread of the CTAs' ends and 3 us of join; 16/4
// heads of 128 50 us (39.6), 12/4 heads of 32 25 us (9.9: half the bytes for the same steps).  More
// CTAs than fit at once (36 us at three per SM), 16-key steps, 2 or 4 stages, a warm-up pass
// through the code and an L2 prefetch of the page table measured no better; cache hints on the
// copies were taken out again (an illegal-instruction error in the fp32 kernel came with them).
// Chunks at head_dim 32 or with more than 128 heads per kv head come here too, whatever their
// rows: 2048 tokens over 16384 at head_dim 32 300 us, 0.16 PFLOP/s (the tile kernel has neither).
#include <cuda_bf16.h>
#include "paged_load.cuh"
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;

template <int D>
struct ShortCfg {
    static constexpr int KT = D == 128 ? 16 : 32;          // keys per warp step
    static constexpr int U = D / 8;                        // 16-byte units per row
    static constexpr int TILE = KT * D * 2;                // bytes of a K or V step
    static constexpr int RING = kStages * 2 * TILE;        // one warp's
    static constexpr int BN = kWarps * KT;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// c [16 x 8] += a [16 x 16] b [16 x 8], bf16 products, fp32 sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// MT: 16-row tiles of a unit.
template <int D, int MT>
__global__ void __launch_bounds__(kThreads, 2) paged_short_kernel(const PagedAttnArgs a) {
    using C = ShortCfg<D>;
    constexpr int KT = C::KT, U = C::U, NT = KT / 8, NO = D / 8;
    constexpr bool PRE = 16 * MT * D * 4 <= 2 * C::TILE;   // a warp's output fits into one stage
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ PagedLocate loc;
    __shared__ PagedSeg s_part[2];                         // the CTA's parts in turn (b < 0: the end)
    __shared__ float s_m[kWarps][16 * MT], s_l[kWarps][16 * MT];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t ring0 = smem_u32(ring) + warp * C::RING;
    const int ngrp = (a.G + a.p.gs - 1) / a.p.gs;          // head groups of a kv head
    // This warp's stream of the part begun last: step j, keys first + j C::BN on, goes through
    // stage (s0 + j) % kStages.
    const int* trow = nullptr;
    const char *kp = nullptr, *vp = nullptr;
    int first = 0, nsteps = 0, kv = 0, s0 = 0, pid = -1, pid1 = -1;
    // Page ids are fetched two steps ahead of the copies that need them, which run two steps
    // ahead of the products.
    auto issue = [&](int j) {
        if (j < nsteps) {
            const int at = first + j * C::BN;
            const int pid2 = j + 2 < nsteps ? page_at(a.c, trow, at + 2 * C::BN + lane, kv) : -1;
            const uint32_t st = ring0 + ((s0 + j) % kStages) * 2 * C::TILE;
            load_rows<KT, U>(st, st + C::TILE, kp, vp, a.c, 2, 0, at, kv, checked_page(a.c, pid, at + lane, kv, a.err), lane);
            pid = pid1;
            pid1 = pid2;
        }
        cp_async_commit();
    };
    uint32_t qf[MT][D / 16][4];                            // the part's query rows as A fragments
    int lim[MT][2];                                        // keys that rows g8 and g8 + 8 see
    auto begin = [&](const PagedSeg& p) {
        const long long head = (long long)(p.hg / ngrp) * a.c.head_stride * 2;
        trow = a.s.table + (size_t)p.b * a.s.W;
        kp = static_cast<const char*>(a.c.k) + head;
        vp = static_cast<const char*>(a.c.v) + head;
        kv = p.kv;
        nsteps = p.t1 - p.t0;
        first = p.t0 * C::BN + warp * KT;                  // keys (t C::BN + warp KT) of the part's tiles t
        pid = nsteps > 0 ? page_at(a.c, trow, first + lane, kv) : -1;
        pid1 = nsteps > 1 ? page_at(a.c, trow, first + C::BN + lane, kv) : -1;
#pragma unroll 1
        for (int j = 0; j < kStages - 1; ++j) issue(j);
        const int h0 = (p.hg / ngrp) * a.G + (p.hg % ngrp) * a.p.gs;   // first query head of the unit
        const int gs = min(a.p.gs, a.G - (p.hg % ngrp) * a.p.gs);      // its heads
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = m * 16 + g8 + 8 * i;
                const bool live = row < p.ntok * gs;
                const int tok = live ? row / gs : 0, h = live ? row - tok * gs : 0;
                lim[m][i] = live ? p.base + p.tok + tok + 1 : 0;
                const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                           (long long)(p.tok0 + p.tok + tok) * a.q_ld + (long long)(h0 + h) * D;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[m][ks][i] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + ks * 16 + t4 * 2)) : 0u;
                    qf[m][ks][2 + i] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + t4 * 2)) : 0u;
                }
            }
    };
    // Warp 0 finds the CTA's parts, one ahead; where its share begins, it finds alone among up to
    // 32 sequences, and the whole CTA among more (256 sequences: 3 us less a call).
    PagedWalk walk;
    int turn = 0;
    if (a.s.B > 32) paged_locate<kThreads>(a, blockIdx.x, loc, blockIdx.x == 0);
    if (warp == 0) {
        PagedSeg n;
        if (a.s.B <= 32) paged_locate_warp(a, blockIdx.x, walk, blockIdx.x == 0);
        else walk.init(a, loc.w0, loc.w1, loc.snap, loc.b, loc.start);
        if (lane < 2) a.part_info[blockIdx.x * 2 + lane] = make_int4(0, 0, 0, 0);
        if (!walk.next(a, n)) n.b = -1;
        if (lane == 0) s_part[0] = n;
    }
    __syncthreads();
    PagedSeg g = s_part[0];
    if (PRE && g.b >= 0) begin(g);
    while (g.b >= 0) {
        const int h0 = (g.hg / ngrp) * a.G + (g.hg % ngrp) * a.p.gs;   // first query head of the unit
        const int gs = min(a.p.gs, a.G - (g.hg % ngrp) * a.p.gs);      // its heads
        const int live_rows = g.ntok * gs;

        float mx[MT][2], sum[MT][2], o[MT][NO][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[m][i] = -INFINITY;
                sum[m][i] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[m][n][e] = 0.f;
        }

        ++turn;
        if (warp == 0) {
            PagedSeg n;
            if (!walk.next(a, n)) n.b = -1;
            if (lane == 0) s_part[turn & 1] = n;
        }
        __syncthreads();                                   // the next part is known, the join before has been read
        if (!PRE) begin(g);
#pragma unroll 1
        for (int j = 0; j < nsteps; ++j) {
            __syncwarp();                                  // step j - 1 has been read by the whole warp
            issue(j + kStages - 1);                        // into its stage
            cp_async_wait<kStages - 1>();
            __syncwarp();                                  // step j has landed for the whole warp
            const uint32_t sk = ring0 + ((s0 + j) % kStages) * 2 * C::TILE, sv = sk + C::TILE;
            const int k0 = first + j * C::BN;

            float s[MT][NT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    // Keys n*8 .. n*8+15, elements ks*16 .. +15: four 8x8 blocks.
                    uint32_t kf[4];
                    const int r = n * 8 + (lane >> 4) * 8 + (lane & 7), u = ks * 2 + ((lane >> 3) & 1);
                    ldsm4(sk + tile_unit<U>(r, u) * 16, kf);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816(s[m][n], qf[m][ks], kf[0], kf[1]);
                        mma16816(s[m][n + 1], qf[m][ks], kf[2], kf[3]);
                    }
                }
            // A step that reaches behind the first row's limit is masked.
            if (k0 + KT > g.base + g.tok + 1) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (k0 + n * 8 + t4 * 2 + (e & 1) >= lim[m][e >> 1]) s[m][n][e] = -INFINITY;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float al[2], ref[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NT; ++n) x = fmaxf(x, fmaxf(s[m][n][2 * i], s[m][n][2 * i + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    const float now = fmaxf(mx[m][i], x * a.scale_log2);
                    ref[i] = now == -INFINITY ? 0.f : now;
                    al[i] = ex2(mx[m][i] - ref[i]);
                    mx[m][i] = now;
                    sum[m][i] *= al[i];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[m][n][e] = ex2(fmaf(s[m][n][e], a.scale_log2, -ref[e >> 1]));
                        sum[m][e >> 1] += s[m][n][e];
                    }
#pragma unroll
                for (int n = 0; n < NO; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[m][n][e] *= al[e >> 1];
            }
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk) {
                // P as the A operand, in two bf16 terms (value and remainder): the weights then
                // carry 16 bits, and the output's own rounding to bf16 is the only one that
                // shows.  The second product costs tensor time that the loads leave idle.
                uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = s[m][2 * kk + (i >> 1)][2 * (i & 1)], y = s[m][2 * kk + (i >> 1)][2 * (i & 1) + 1];
                        ph[m][i] = pack2(x, y);
                        const float2 h = unpack2(ph[m][i]);
                        pl[m][i] = pack2(x - h.x, y - h.y);
                    }
#pragma unroll
                for (int n = 0; n < NO; n += 2) {
                    // Keys kk*16 .. +15, elements n*8 .. n*8+15, transposed on the way.
                    uint32_t vf[4];
                    const int r = kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), u = n + (lane >> 4);
                    ldsm4t(sv + tile_unit<U>(r, u) * 16, vf);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16816(o[m][n], ph[m], vf[0], vf[1]);
                        mma16816(o[m][n + 1], ph[m], vf[2], vf[3]);
                        mma16816(o[m][n], pl[m], vf[0], vf[1]);
                        mma16816(o[m][n + 1], pl[m], vf[2], vf[3]);
                    }
                }
            }
        }
        // The next part's first steps go out before this one is joined: they take the two stages
        // that the last step did not use.  The join takes that one (PRE), or all rings.
        const int last = (s0 + nsteps + kStages - 1) % kStages;
        const PagedSeg next = s_part[turn & 1];
        if (PRE) {
            __syncwarp();
            if (next.b >= 0) {
                s0 = (s0 + nsteps) % kStages;
                begin(next);
            }
        } else {
            cp_async_wait<0>();
            __syncthreads();                               // every ring is idle
        }
        float* const s_o = reinterpret_cast<float*>(PRE ? ring + last * 2 * C::TILE : ring);
        constexpr int S_O = (PRE ? C::RING : 16 * MT * D * 4) / 4;     // from one warp's rows [16 MT][D] to the next's

#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = sum[m][i];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (t4 == 0) {
                    s_m[warp][m * 16 + g8 + 8 * i] = mx[m][i];
                    s_l[warp][m * 16 + g8 + 8 * i] = x;
                }
            }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NO; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<float2*>(s_o + warp * S_O + (m * 16 + g8 + 8 * i) * D + n * 8 + t4 * 2) =
                        make_float2(o[m][n][2 * i], o[m][n][2 * i + 1]);
        __syncthreads();
        const int pslot = blockIdx.x * 2 + g.slot();
        for (int i = tid; i < live_rows * (D / 4); i += kThreads) {
            const int row = i / (D / 4), e = (i % (D / 4)) * 4;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][row]);
            const float ref = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float wt = ex2(s_m[w][row] - ref);
                const float4 x = *reinterpret_cast<const float4*>(s_o + w * S_O + row * D + e);
                l += s_l[w][row] * wt;
                acc.x += x.x * wt;
                acc.y += x.y * wt;
                acc.z += x.z * wt;
                acc.w += x.w * wt;
            }
            if (g.whole()) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const long long orow = (long long)(g.tok0 + g.tok + row / gs) * a.Hq + h0 + row % gs;
                uint2 pk = make_uint2(pack2(acc.x * inv, acc.y * inv), pack2(acc.z * inv, acc.w * inv));
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + orow * D + e) = pk;
                if (e == 0) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else {
                const size_t prow = (size_t)pslot * a.p.rows + row;
                *reinterpret_cast<float4*>(a.part_o + prow * D + e) = acc;
                if (e == 0) a.part_ml[prow] = make_float2(m, l);
            }
        }
        if (!g.whole() && tid == 0) a.part_info[pslot] = paged_record(g);
        g = next;
    }
}

template <int D, int MT>
cudaError_t launch_short_t(const PagedAttnArgs& a, cudaStream_t st) {
    using C = ShortCfg<D>;
    auto kfn = paged_short_kernel<D, MT>;
    constexpr int smem = kWarps * C::RING;
    static_assert(smem >= kWarps * 16 * MT * D * 4, "the join fits into the rings");
    static_assert(2 * (smem + 4096) <= 227 * 1024, "two CTAs per SM");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kfn, smem, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(a.p.C), dim3(kThreads), smem, st, a);
}

}  // namespace

int paged_short_bn(int D) { return D == 128 ? ShortCfg<128>::BN : ShortCfg<64>::BN; }

cudaError_t launch_paged_short(PagedKind kind, int D, const PagedAttnArgs& a, cudaStream_t st) {
    const bool two = kind == PAGED_SHORT32;
    switch (D) {
        case 32: return two ? launch_short_t<32, 2>(a, st) : launch_short_t<32, 1>(a, st);
        case 64: return two ? launch_short_t<64, 2>(a, st) : launch_short_t<64, 1>(a, st);
        case 128: return two ? launch_short_t<128, 2>(a, st) : launch_short_t<128, 1>(a, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ne
