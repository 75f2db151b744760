// paged_f32.cu -- attention over the paged cache for fp32 tensors, in fp32 throughout.
//
// The fp32 entry points of the training kernels use TF32 tensor cores; a cache that is
// kept in fp32 is kept for its precision, so here products and sums are fp32 FMAs (packed,
// two per instruction).  Few rows per kv head are bound by the read of the cache (8 D bytes
// per key against 4 D FMAs per row: 8 rows use about a third of the FMA rate at the copy
// bandwidth); many rows by the FMAs and the shared-memory reads that feed them.
//
// A warp holds RW query rows.  S: lane = key, the query rows broadcast from shared memory;
// O: lane = two (or one) elements of D, the weights broadcast.  FEW (up to 32 rows per kv head):
// eight warps take interleaved 32-key steps of the same 4, 8 or 16 rows, each with a private ring
// of three K or V tiles, and are joined at the end of a unit.  MANY: eight warps take 8 of 64
// rows each over one shared ring.
//
// Measured (GB300): one step over 8 x 16384 positions, 12/4 heads of 64: 49 us, 5.5 TB/s; with
// 32/4 heads 54 us; four new tokens each, 12/4 heads: 78 us (MANY would take 279: its warps
// without rows wait); 512 new tokens over 4096 positions: 217 us, 28 TFLOP/s of the 75 that fp32
// FMAs give.  Four warps with twice the keys in flight took 54, 64 and 99 us (a scheduler with
// one warp waits for its chain), a ring of whole K and V steps 60, 89 and -.
#include "paged_load.cuh"
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kStages = 3;
// RW: query rows per warp.
template <int D, int RW, bool MANY>
struct F32Cfg {
    static constexpr int WK = MANY ? 1 : 8;                // warps along the keys
    static constexpr int WR = MANY ? 8 : 1;                // warps along the rows
    static constexpr int WARPS = WK * WR;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int ROWS = WR * RW;
    static constexpr int BN = 32 * WK;
    static constexpr int U = D / 4;                        // 16-byte units per row
    static constexpr int TILE = 32 * D * 4;                // one K or V step of 32 keys
    static constexpr int SLOTS = MANY ? 2 * kStages : 3;   // tiles of a ring
    static constexpr int RINGS = WK * SLOTS * TILE;
    static constexpr int Q_BYTES = ROWS * D * 4;
    static constexpr int P_BYTES = WARPS * 32 * RW * 4;
    static constexpr int SMEM = RINGS + Q_BYTES + P_BYTES;
    static constexpr int DL = D / 32;                      // output elements per lane
    static constexpr int CTAS = MANY || (D == 32 && RW < 16) ? 2 : 1;   // of an SM: what shared memory and registers hold
    static_assert(WK * ROWS * D * 4 <= RINGS, "the join fits into the rings");
};

template <int D, int RW, bool MANY>
__global__ void __launch_bounds__(F32Cfg<D, RW, MANY>::THREADS, F32Cfg<D, RW, MANY>::CTAS) paged_f32_kernel(const PagedAttnArgs a) {
    using C = F32Cfg<D, RW, MANY>;
    constexpr int U = C::U, DL = C::DL;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PagedLocate loc;
    __shared__ int s_lim[C::ROWS];                         // keys that a row sees
    __shared__ float s_m[C::WK][C::ROWS], s_l[C::WK][C::ROWS];
    float* s_q = reinterpret_cast<float*>(smem + C::RINGS);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wk = MANY ? 0 : warp, row0 = MANY ? warp * RW : 0;
    float* s_p = reinterpret_cast<float*>(smem + C::RINGS + C::Q_BYTES) + warp * 32 * RW;   // [key][RW]

    griddep_launch_dependents();
    griddep_wait();
    PagedWalk walk;
    paged_locate<C::THREADS>(a, blockIdx.x, loc, blockIdx.x == 0);
    walk.init(a, loc.w0, loc.w1, loc.snap, loc.b, loc.start);
    if (tid < 2) a.part_info[blockIdx.x * 2 + tid] = make_int4(0, 0, 0, 0);

    const int ngrp = (a.G + a.p.gs - 1) / a.p.gs;          // head groups of a kv head
    const uint32_t ring0 = smem_u32(smem) + wk * C::SLOTS * C::TILE;
    PagedSeg g;
    while (walk.next(a, g)) {
        const int hkv = g.hg / ngrp, hs = g.hg % ngrp;
        const int h0 = hkv * a.G + hs * a.p.gs;
        const int gs = min(a.p.gs, a.G - hs * a.p.gs);
        const int live_rows = g.ntok * gs;
        const int* trow = a.s.table + (size_t)g.b * a.s.W;
        const char* kp = static_cast<const char*>(a.c.k) + (long long)hkv * a.c.head_stride * 4;
        const char* vp = static_cast<const char*>(a.c.v) + (long long)hkv * a.c.head_stride * 4;

        // Pages of the warp's first two steps, on their way while the query rows are staged.
        const int nsteps = g.t1 - g.t0;
        const int first = g.t0 * C::BN + wk * 32;
        const int lfirst = first + (MANY ? warp * 4 : 0);  // (MANY: a warp loads four rows of every step)
        int pid = page_at(a.c, trow, lfirst + lane, g.kv);
        int pid1 = nsteps > 1 ? page_at(a.c, trow, lfirst + C::BN + lane, g.kv) : -1;
        for (int i = tid; i < C::ROWS * U; i += C::THREADS) {
            const int row = i / U, u = i % U;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < live_rows) {
                const float* src = static_cast<const float*>(a.q) + (long long)(g.tok0 + g.tok + row / gs) * a.q_ld +
                                   (long long)(h0 + row % gs) * D;
                x = __ldg(reinterpret_cast<const float4*>(src) + u);
            }
            reinterpret_cast<float4*>(s_q)[i] = x;
        }
        if (tid < C::ROWS) s_lim[tid] = tid < live_rows ? g.base + g.tok + tid / gs + 1 : 0;

        float m[RW], l[RW], o[RW][DL];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < DL; ++e) o[r][e] = 0.f;
        }

        // Scores of the warp's rows against keys key0 .. key0 + 31 (lane: key), softmax, weights to s_p.
        auto scores = [&](const float4* sk, int key0) {
            // Behind the first token's position rows are masked.  (MANY always looks: the branch
            // cost its loop 4 to 11%.)
            const bool edge = MANY || key0 + 32 > g.base + g.tok + 1;
            float2 acc[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) acc[r] = make_float2(0.f, 0.f);
#pragma unroll (RW == 4 ? 8 : 4)
            for (int u = 0; u < U; ++u) {
                const float4 kf = sk[tile_unit<U>(lane, u)];
#pragma unroll
                for (int r = 0; r < RW; ++r) {
                    const float4 qv = reinterpret_cast<const float4*>(s_q)[(row0 + r) * U + u];
                    acc[r] = __ffma2_rn(make_float2(kf.x, kf.y), make_float2(qv.x, qv.y), acc[r]);
                    acc[r] = __ffma2_rn(make_float2(kf.z, kf.w), make_float2(qv.z, qv.w), acc[r]);
                }
            }
            float p[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
                const float s = !edge || key0 + lane < s_lim[row0 + r] ? (acc[r].x + acc[r].y) * a.scale_log2 : -INFINITY;
                float x = s;
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                const float now = fmaxf(m[r], x);
                const float ref = now == -INFINITY ? 0.f : now;
                const float al = ex2(m[r] - ref);
                p[r] = ex2(s - ref);
                m[r] = now;
                l[r] = l[r] * al + p[r];
#pragma unroll
                for (int e = 0; e < DL; ++e) o[r][e] *= al;
            }
#pragma unroll
            for (int r = 0; r < RW; r += 4)
                *reinterpret_cast<float4*>(s_p + lane * RW + r) = make_float4(p[r], p[r + 1], p[r + 2], p[r + 3]);
        };
        auto outputs = [&](const float* sv) {
#pragma unroll (RW == 4 ? 8 : 4)
            for (int k = 0; k < 32; ++k) {
                float pr[RW];
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(s_p + k * RW + r);
                    pr[r] = x.x;
                    pr[r + 1] = x.y;
                    pr[r + 2] = x.z;
                    pr[r + 3] = x.w;
                }
                if constexpr (DL == 2) {
                    const float2 v = *reinterpret_cast<const float2*>(sv + tile_unit<U>(k, lane >> 1) * 4 + (lane & 1) * 2);
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        const float2 x = __ffma2_rn(make_float2(pr[r], pr[r]), v, make_float2(o[r][0], o[r][1]));
                        o[r][0] = x.x;
                        o[r][1] = x.y;
                    }
                } else {
                    const float v = sv[tile_unit<U>(k, lane >> 2) * 4 + (lane & 3)];
#pragma unroll
                    for (int r = 0; r < RW; ++r) o[r][0] = fmaf(pr[r], v, o[r][0]);
                }
            }
        };

        const uint8_t* ring = smem + wk * C::SLOTS * C::TILE;
        if constexpr (!MANY) {
            // A private ring of three tiles, K and V of a step in turn: the next two are in flight
            // while one is worked on.
            int page = -1;                                 // this step's, checked
            long long off[4] = {0, 0, 0, 0};               // its four groups of eight rows (a page has eight or more)
            bool full = false;                             // every row of it is there
            const int mask = (1 << a.c.ps_shift) - 1;
            const long long tok_bytes = a.c.tok_stride * 4;
            const long long lane_off = (lane / U) * tok_bytes + (lane % U) * 16;
            int slot = 0;                                  // of the next tile to load
            auto load = [&](const char* src, int j) {
                const uint32_t st = ring0 + slot * C::TILE;
                if (j < nsteps && full) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const char* s = src + off[x];
#pragma unroll
                        for (int i = 0; i < 8; i += 32 / U, s += 32 / U * tok_bytes)
                            cp_async16(st + tile_unit<U>(8 * x + i + lane / U, lane % U) * 16, s, true);
                    }
                } else if (j < nsteps) {
                    load_tile<U>(st, src, a.c, 4, first + j * C::BN, g.kv, page, lane);
                }
                cp_async_commit();
                slot = slot == 2 ? 0 : slot + 1;
            };
            auto load_k = [&](int j) {
                if (j < nsteps) {
                    const int at = first + j * C::BN;
                    page = checked_page(a.c, pid, at + lane, g.kv, a.err);
                    pid = pid1;
                    pid1 = j + 2 < nsteps ? page_at(a.c, trow, at + 2 * C::BN + lane, g.kv) : -1;
                    full = __all_sync(0xffffffffu, page >= 0);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        off[x] = ((long long)__shfl_sync(0xffffffffu, page, 8 * x) * a.c.page_stride) * 4 +
                                 ((at + 8 * x) & mask) * tok_bytes + lane_off;
                }
                load(kp, j);
            };
            load_k(0);
            load(vp, 0);
            __syncthreads();                               // the query rows are there
            int at = 0;                                    // slot of the tile to work on
            for (int j = 0; j < nsteps; ++j) {
                cp_async_wait<1>();
                __syncwarp();                              // K is there; the last step's V is read
                load_k(j + 1);
                const int key0 = first + j * C::BN;        // (behind the unit's keys: this warp's share of the last tile)
                if (key0 < g.kv) scores(reinterpret_cast<const float4*>(ring + at * C::TILE), key0);
                at = at == 2 ? 0 : at + 1;
                cp_async_wait<1>();
                __syncwarp();                              // V and the weights are there, K is read
                load(vp, j + 1);
                if (key0 < g.kv) outputs(reinterpret_cast<const float*>(ring + at * C::TILE));
                at = at == 2 ? 0 : at + 1;
            }
        } else {
            // One ring for all warps.
            constexpr int LROWS = 4;
            auto issue = [&](int j) {
                if (j < nsteps) {
                    const int at = lfirst + j * C::BN;
                    const int pid2 = j + 2 < nsteps ? page_at(a.c, trow, at + 2 * C::BN + lane, g.kv) : -1;
                    const uint32_t st = ring0 + (j % kStages) * 2 * C::TILE;
                    load_rows<LROWS, U>(st, st + C::TILE, kp, vp, a.c, 4, warp * LROWS, at, g.kv,
                                        checked_page(a.c, pid, at + lane, g.kv, a.err), lane);
                    pid = pid1;
                    pid1 = pid2;
                }
                cp_async_commit();
            };
#pragma unroll
            for (int j = 0; j < kStages - 1; ++j) issue(j);
            __syncthreads();                               // the query rows are there
            for (int j = 0; j < nsteps; ++j) {
                cp_async_wait<kStages - 2>();
                __syncthreads();
                issue(j + kStages - 1);
                if (row0 >= live_rows) continue;           // (a warp without rows only loads)
                const uint8_t* st = ring + (j % kStages) * 2 * C::TILE;
                scores(reinterpret_cast<const float4*>(st), first + j * C::BN);
                __syncwarp();
                outputs(reinterpret_cast<const float*>(st + C::TILE));
            }
        }
        cp_async_wait<0>();
        __syncthreads();                                   // rings and query rows are idle
#pragma unroll
        for (int r = 0; r < RW; ++r) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], off);
            if (lane == 0) {
                s_m[wk][row0 + r] = m[r];
                s_l[wk][row0 + r] = l[r];
            }
        }
        float* s_o = reinterpret_cast<float*>(smem);       // [WK][ROWS][D]
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
            for (int e = 0; e < DL; ++e) s_o[(size_t)(wk * C::ROWS + row0 + r) * D + lane * DL + e] = o[r][e];
        __syncthreads();
        const int pslot = blockIdx.x * 2 + g.slot();
        for (int i = tid; i < live_rows * U; i += C::THREADS) {
            const int row = i / U, e = (i % U) * 4;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < C::WK; ++w) mm = fmaxf(mm, s_m[w][row]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < C::WK; ++w) {
                const float wt = ex2(s_m[w][row] - ref);
                const float4 x = *reinterpret_cast<const float4*>(s_o + (size_t)(w * C::ROWS + row) * D + e);
                ll += s_l[w][row] * wt;
                acc.x += x.x * wt;
                acc.y += x.y * wt;
                acc.z += x.z * wt;
                acc.w += x.w * wt;
            }
            if (g.whole()) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;
                const long long orow = (long long)(g.tok0 + g.tok + row / gs) * a.Hq + h0 + row % gs;
                *reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * D + e) =
                    make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (e == 0) a.lse[orow] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.6931471805599453f;
            } else {
                const size_t prow = (size_t)pslot * a.p.rows + row;
                *reinterpret_cast<float4*>(a.part_o + prow * D + e) = acc;
                if (e == 0) a.part_ml[prow] = make_float2(mm, ll);
            }
        }
        if (!g.whole() && tid == 0) a.part_info[pslot] = paged_record(g);
        __syncthreads();
    }
}

template <int D, int RW, bool MANY>
cudaError_t launch_f32_t(const PagedAttnArgs& a, cudaStream_t st) {
    using C = F32Cfg<D, RW, MANY>;
    auto kfn = paged_f32_kernel<D, RW, MANY>;
    static_assert(C::SMEM + 4096 <= 227 * 1024, "shared memory");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kfn, C::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(a.p.C), dim3(C::THREADS), C::SMEM, st, a);
}

template <int D>
cudaError_t launch_f32_d(PagedKind kind, const PagedAttnArgs& a, cudaStream_t st) {
    switch (kind) {
        case PAGED_F32_FEW4: return launch_f32_t<D, 4, false>(a, st);
        case PAGED_F32_FEW8: return launch_f32_t<D, 8, false>(a, st);
        case PAGED_F32_FEW16: return launch_f32_t<D, 16, false>(a, st);
        default: return launch_f32_t<D, 8, true>(a, st);
    }
}

}  // namespace

int paged_f32_bn(bool many) { return many ? F32Cfg<64, 8, true>::BN : F32Cfg<64, 8, false>::BN; }

cudaError_t launch_paged_f32(PagedKind kind, int D, const PagedAttnArgs& a, cudaStream_t st) {
    if (D == 32) return launch_f32_d<32>(kind, a, st);
    if (D == 64) return launch_f32_d<64>(kind, a, st);
    return cudaErrorInvalidValue;
}

}  // namespace ne
