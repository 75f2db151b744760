// paged_weights.cu -- the attention weight that every cached position has received from the new
// tokens of its sequence: for sequence b, kv head g and key j
//   out[b][g][j] = w[b][g][j] + sum over tokens i at t_i >= j and heads h of g of
//                  2^(s log2(e) q_ih k_j - log2(e) lse_ih).
// The log-sum-exp is the attention's own, so there is no running maximum, no second product and
// no join of rows: keys are independent of each other.  Every kernel therefore has the keys as rows
// of its product and sums along the query rows, within one thread or four.
//
// Few rows (up to 32 per kv head): read of the keys (2 D bytes against 2 D flops per row).  The line of
// all 32-key steps is cut into one share per warp; a warp streams its steps through a private ring
// (16-byte cp.async) and multiplies with mma.sync, keys as the 16-row operand and query rows as its 8
// columns, so that three rows waste five eighths of a product instead of thirteen sixteenths.
// Many rows, bf16: tcgen05, 128 keys (a TMEM lane each) times 128 query rows per tile.  2 * 128 *
// 128 * D flops, 512 cycles of the tensor core at D 128, and 16384 exponentials, 512 cycles: the
// exponentials bound D 64 and both D 128.  A unit is (sequence, kv head, 256 keys) and the query tiles
// that see it; a share cuts units between query tiles, cut units' sums are added by a join.
// Many rows, fp32: units of 128 keys on fp32 FMAs, two keys per lane in registers, the query rows
// broadcast from shared memory.
//
// Measured (GB300): one token over 8 x 16384 positions, 12/4 heads of 64: 16.2 us, 4.4 TB/s (10.6 at the copy
// rate; 3 to begin and find the shares, then 5.3 TB/s); the small fp32 step 3.1.  2048 tokens over 16384
// positions, 16/4 heads of 128: 107 us, 1.20 PFLOP/s (62% of the bf16 GEMM; the tensor pipe and the exponential units 48%
// busy each, operands out of shared memory, 128 bytes a cycle, bound the products); of 64: 99.5 us, 0.65 PFLOP/s, the
// exponential units 52% busy and the tensor pipe 26%: of the 3000 cycles of a tile its warps spend 2200 in the section
// that has the exponentials; fp32, of 64: 1.94 ms, 33 TFLOP/s.  Twelve sequences, single tokens beside chunks up to 512
// over up to 4096: 18.9 us (2.0), 5 before the first product, then 5 query tiles in 3 parts per CTA, then the join.
// Tried for many rows and left out: part of the exponentials as a polynomial on the FMA pipes (D 64 119 -> 144
// us, then with eight exponential warps), keys as the TMEM operand with 96-row query tiles (D 128 120 ->
// 138: it is the issue of products, some 90 cycles each, that counts), S in halves with buffers of their own
// (D 64 105 -> 113), all 128 columns of S in registers at once (119 -> 133), or 64 (104 -> 117), 16 columns on
// their way behind those at work (101 -> 103), one product for two query tiles (S then has one buffer per key tile: D
// 128 109 -> 141).
#include <cuda_bf16.h>
#include <type_traits>
#include "paged_line.cuh"
#include "paged_load.cuh"

namespace ne {
namespace {

// ------------------------------------------------------------------ few rows
constexpr int kFewWarps = 8;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewStages = 3;

// One step's 32 keys of a head into a tile (load_rows' layout, keys alone).
template <int U>
__device__ __forceinline__ void load_keys(uint32_t st, const char* k, const PagedView& c, int esize, int first, int kv, int pid,
                                          int lane) {
    constexpr int PER = 32 / U;
    const int mask = (1 << c.ps_shift) - 1;
    const long long tok_bytes = c.tok_stride * esize;
    if (PER <= 8 && __all_sync(0xffffffffu, pid >= 0)) {
        const long long lane_off = (lane / U) * tok_bytes + (lane % U) * 16;
#pragma unroll
        for (int x = 0; x < 32; x += 8) {
            long long off = (long long)__shfl_sync(0xffffffffu, pid, x) * c.page_stride * esize + ((first + x) & mask) * tok_bytes + lane_off;
#pragma unroll
            for (int i = 0; i < 8; i += PER, off += PER * tok_bytes)
                cp_async16(st + tile_unit<U>(x + i + lane / U, lane % U) * 16, k + off, true);
        }
        return;
    }
    load_tile<U>(st, k, c, esize, first, kv, pid, lane);
}

// A warp's place in the line of steps: sequence, kv head, step.
struct StepWalk {
    int b, h, st, steps, len;
    long long left;                    // steps that are still to come, this one included
    __device__ __forceinline__ void take(const WeightArgs& a) {
        len = min(max(__ldg(a.s.lens + b), 0), a.s.cap);
        steps = (len + 31) >> 5;
    }
    __device__ __forceinline__ void init(const WeightArgs& a, int b_, long long off, long long n) {
        b = b_;
        left = n;
        h = st = 0;
        if (left <= 0) return;
        take(a);
        h = line_head(off, steps);
        st = (int)off;
    }
    // True where the next step is another head's.
    __device__ __forceinline__ bool next(const WeightArgs& a) {
        if (--left <= 0 || ++st < steps) return false;
        st = 0;
        if (++h == a.Hkv) {
            h = 0;
            do ++b;
            while (take(a), steps == 0);                   // (left > 0: there is a sequence with steps)
        }
        return true;
    }
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr float kLog2e = 1.4426950408889634f;

// RC query rows at a time; a sequence with more takes its rows in turn over every step.
template <int D, int RC>
struct FewBf16 {
    static constexpr int ESIZE = 2, U = D / 8, NT = RC / 8, EXTRA = 0;
    uint32_t qf[NT][D / 16][2];
    float nl[NT][2];                   // -log2(e) lse of the lane's two rows of every eight (-inf: nobody)
    int lim[NT][2];                    // keys that they see

    __device__ __forceinline__ void rows(const WeightArgs& a, float*, const PagedSeq& q, int h, int r0, int lane) {
        const int g8 = lane >> 2, t4 = lane & 3, R = q.n * a.G;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = r0 + n * 8 + g8;
            const bool live = r < R;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q);
            if (live) src += (long long)(q.tok0 + r / a.G) * a.q_ld + (long long)(h * a.G + r % a.G) * D;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                qf[n][ks][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + ks * 16 + t4 * 2)) : 0u;
                qf[n][ks][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + t4 * 2)) : 0u;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = r0 + n * 8 + t4 * 2 + i;
                const bool in = c < R;
                nl[n][i] = in ? -kLog2e * __ldg(a.lse + (long long)(q.tok0 + c / a.G) * a.Hq + h * a.G + c % a.G) : -INFINITY;
                lim[n][i] = in ? q.len - q.n + c / a.G + 1 : 0;
            }
        }
    }
    // Adds this chunk's weights of the step's keys: sums [m][i] of keys 16 m + 8 i + lane / 4.
    __device__ __forceinline__ void add(const WeightArgs& a, uint32_t st, const float*, int k0, bool edge, float (&sum)[2][2], int lane) const {
        const int g8 = lane >> 2;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float c[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t kf[4];
                ldsm4(st + tile_unit<U>(m * 16 + (lane & 15), ks * 2 + (lane >> 4)) * 16, kf);
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(c[n], kf, qf[n][ks][0], qf[n][ks][1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = ex2(fmaf(c[n][e], a.scale_log2, nl[n][e & 1]));
                    const bool seen = !edge || k0 + m * 16 + (e >> 1) * 8 + g8 < lim[n][e & 1];
                    sum[m][e >> 1] += seen ? p : 0.f;
                }
        }
    }
    // The lane's key among the step's 32 and its sum.
    static __device__ __forceinline__ int key(int lane) { return ((lane & 2) >> 1) * 16 + (lane & 1) * 8 + (lane >> 2); }
    static __device__ __forceinline__ float total(const float (&sum)[2][2], int lane) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[i] = sum[i >> 1][i & 1];
            s[i] += __shfl_xor_sync(0xffffffffu, s[i], 1);
            s[i] += __shfl_xor_sync(0xffffffffu, s[i], 2);
        }
        return lane & 2 ? (lane & 1 ? s[3] : s[2]) : (lane & 1 ? s[1] : s[0]);
    }
};

template <int D, int RC>
struct FewF32 {
    static constexpr int ESIZE = 4, U = D / 4, EXTRA = RC * D;   // floats of shared memory per warp: the rows
    float nl[RC];
    int lim[RC];

    __device__ __forceinline__ void rows(const WeightArgs& a, float* s_q, const PagedSeq& q, int h, int r0, int lane) {
        const int R = q.n * a.G;
        __syncwarp();                                      // the rows before have been read
        for (int i = lane; i < RC * U; i += 32) {
            const int r = r0 + i / U;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < R)
                x = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (long long)(q.tok0 + r / a.G) * a.q_ld +
                                                          (long long)(h * a.G + r % a.G) * D) + i % U);
            reinterpret_cast<float4*>(s_q)[i] = x;
        }
#pragma unroll
        for (int i = 0; i < RC; ++i) {
            const int r = r0 + i;
            nl[i] = r < R ? -kLog2e * __ldg(a.lse + (long long)(q.tok0 + r / a.G) * a.Hq + h * a.G + r % a.G) : -INFINITY;
            lim[i] = r < R ? q.len - q.n + r / a.G + 1 : 0;
        }
        __syncwarp();
    }
    __device__ __forceinline__ void add(const WeightArgs& a, uint32_t, const float* tile, int k0, bool, float (&sum)[2][2], int lane,
                                        const float* s_q) const {
        float2 acc[RC];
#pragma unroll
        for (int r = 0; r < RC; ++r) acc[r] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int u = 0; u < U; ++u) {
            const float4 kf = reinterpret_cast<const float4*>(tile)[tile_unit<U>(lane, u)];
#pragma unroll
            for (int r = 0; r < RC; ++r) {
                const float4 qv = reinterpret_cast<const float4*>(s_q)[r * U + u];
                acc[r] = __ffma2_rn(make_float2(kf.x, kf.y), make_float2(qv.x, qv.y), acc[r]);
                acc[r] = __ffma2_rn(make_float2(kf.z, kf.w), make_float2(qv.z, qv.w), acc[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < RC; ++r) {
            const float p = ex2(fmaf(acc[r].x + acc[r].y, a.scale_log2, nl[r]));
            sum[0][0] += k0 + lane < lim[r] ? p : 0.f;
        }
    }
    static __device__ __forceinline__ int key(int lane) { return lane; }
    static __device__ __forceinline__ float total(const float (&sum)[2][2], int) { return sum[0][0]; }
};

template <int D, int RC, bool F32>
struct FewPick {
    typedef FewBf16<D, RC> type;
};
template <int D, int RC>
struct FewPick<D, RC, true> {
    typedef FewF32<D, RC> type;
};

template <int D, int RC, bool F32>
struct FewCfg {
    typedef typename FewPick<D, RC, F32>::type Rows;
    static constexpr int TILE = 32 * D * Rows::ESIZE;
    static constexpr int RING = kFewStages * TILE;
    static constexpr int SMEM = kFewWarps * (RING + Rows::EXTRA * 4);
    static constexpr int CTAS = SMEM > 108 * 1024 ? 1 : 2;
};

template <int D, int RC, bool F32>
__global__ void __launch_bounds__(kFewThreads, FewCfg<D, RC, F32>::CTAS) weights_few_kernel(const WeightArgs a) {
    using C = FewCfg<D, RC, F32>;
    using Rows = typename C::Rows;
    constexpr int U = Rows::U;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Line<kFewThreads> line;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    int bad = 0;
    auto cost = [&](int b) -> long long {
        const PagedSeq q = paged_seq(a.s, b, bad);
        return (long long)((q.len + 31) >> 5) * a.Hkv;
    };
    constexpr int GW = C::CTAS * kWeightCtas * kFewWarps;
    const auto share = [&](long long total, long long& x0, long long& x1) {
        line_share(total, blockIdx.x * kFewWarps + warp, GW, line_inv(GW), x0, x1);
    };
    int b;
    long long x0, x1, start;
    if (a.s.B <= 32) {
        line_warp(a.s.B, cost, share, x0, x1, b, start);
    } else {
        share(line_total(line, a.s.B, cost), x0, x1);
        line_find(line, a.s.B, cost, x0, b, start);
    }
    if (blockIdx.x == 0 && bad) report_error(a.err, bad);
    if (x0 >= x1) return;

    uint8_t* const ring = smem + warp * C::RING;
    float* const s_q = reinterpret_cast<float*>(smem + kFewWarps * C::RING) + warp * Rows::EXTRA;
    const uint32_t ring0 = smem_u32(ring);
    StepWalk in, at;                                       // of the copies, and of the products
    in.init(a, b, x0 - start, x1 - x0);
    at = in;
    auto fetch = [&]() { return page_at(a.c, a.s.table + (size_t)in.b * a.s.W, in.st * 32 + lane, in.len); };
    int pid = fetch(), filled = 0;
    auto issue = [&]() {
        if (in.left > 0) {
            const int first = in.st * 32;
            const int page = checked_page(a.c, pid, first + lane, in.len, a.err);
            load_keys<U>(ring0 + filled * C::TILE, static_cast<const char*>(a.c.k) + (long long)in.h * a.c.head_stride * Rows::ESIZE, a.c,
                         Rows::ESIZE, first, in.len, page, lane);
            in.next(a);
            if (in.left > 0) pid = fetch();
        }
        cp_async_commit();
        filled = filled == kFewStages - 1 ? 0 : filled + 1;
    };
    for (int j = 0; j < kFewStages - 1; ++j) issue();
    Rows rows;
    PagedSeq q = {0, 0, 0};
    bool fresh = true;                                     // the head's rows are still to be loaded
    for (int slot = 0; at.left > 0; slot = slot == kFewStages - 1 ? 0 : slot + 1) {
        const int k0 = at.st * 32, key = k0 + Rows::key(lane);
        const long long o = ((long long)at.b * a.Hkv + at.h) * a.s.cap + key;
        const float old = a.w && key < at.len ? a.w[o] : 0.f;
        if (fresh) q = paged_seq(a.s, at.b, bad);
        const int R = q.n * a.G, base = q.len - q.n;
        if (fresh && R > 0) rows.rows(a, s_q, q, at.h, 0, lane);
        __syncwarp();                                      // the step before has been read by the whole warp
        issue();                                           // into its place
        cp_async_wait<kFewStages - 1>();
        __syncwarp();
        float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
        for (int r0 = 0; r0 < R; r0 += RC) {
            if (R > RC) {
                if (base + (min(R, r0 + RC) - 1) / a.G < k0) continue;   // none of them sees a key of the step
                rows.rows(a, s_q, q, at.h, r0, lane);
            }
            const bool edge = k0 + 32 > base + r0 / a.G + 1;
            if constexpr (F32) rows.add(a, 0, reinterpret_cast<const float*>(ring + slot * C::TILE), k0, edge, sum, lane, s_q);
            else rows.add(a, ring0 + slot * C::TILE, nullptr, k0, edge, sum, lane);
        }
        const float got = Rows::total(sum, lane);
        if (key < at.len) a.w_out[o] = old + got;
        fresh = at.next(a);
    }
}

// ------------------------------------------------------------------ many rows: units and shares
// What a CTA does with one unit: query tiles [t0, t1) of [tf, nt) for keys kt 2^key_shift .. of head h.  Query
// tile t holds tokens (t / ngrp) sub .. and heads (t % ngrp) gs .. of the kv head.
struct WeightPart {
    int b, h, kt;
    int tok0, n, len;
    int tf, nt, t0, t1;
    __device__ __forceinline__ bool whole() const { return t0 == tf && t1 == nt; }
};

// Cost of key tiles 0 .. k-1 of a head, in tokens: each ovh + the tokens that see its first key.
__device__ __forceinline__ long long weight_prefix(const PagedSeq& q, long long k, const WeightArgs& a) {
    const long long base = q.len - q.n, all = k * (a.ovh + q.n);
    const long long k1 = base < 0 ? 0 : (base >> a.key_shift) + 1;      // the first tile that not every token sees
    if (k <= k1) return all;
    return all - (((k * (k - 1) - k1 * (k1 - 1)) >> 1 << a.key_shift) - base * (k - k1));
}
__device__ __forceinline__ int weight_tiles(const PagedSeq& q, const WeightArgs& a) { return (q.len + (1 << a.key_shift) - 1) >> a.key_shift; }
__device__ __forceinline__ long long weight_cost(const PagedSeq& q, const WeightArgs& a) { return weight_prefix(q, weight_tiles(q, a), a); }

struct WeightWalk {
    long long w0, w1, cur;
    PagedSeq q;
    int b, h, kt, nk;
    __device__ __forceinline__ void take(const WeightArgs& a) {
        int bad = 0;
        q = paged_seq(a.s, b, bad);
        nk = weight_tiles(q, a);
    }
    __device__ __forceinline__ void init(const WeightArgs& a, long long w0_, long long w1_, int b_, long long start) {
        w0 = w0_;
        w1 = w1_;
        b = b_;
        cur = start;
        h = kt = 0;
        if (w0 >= w1) {
            cur = w1;
            return;
        }
        take(a);
        const long long S = weight_cost(q, a);
        long long x = w0 - start;
        h = line_head(x, S);
        int lo = 0, hi = nk - 1;                           // the last tile that starts at or before x
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (weight_prefix(q, mid, a) <= x) lo = mid;
            else hi = mid - 1;
        }
        kt = lo;
        cur = start + h * S + weight_prefix(q, kt, a);
    }
    __device__ __forceinline__ bool next(const WeightArgs& a, WeightPart& p) {
        while (cur < w1) {
            const int first = max(0, (kt << a.key_shift) - (q.len - q.n));         // the first token that sees the tile
            const long long cost = a.ovh + q.n - first;
            p.b = b;
            p.h = h;
            p.kt = kt;
            p.tok0 = q.tok0;
            p.n = q.n;
            p.len = q.len;
            p.tf = first / a.sub * a.ngrp;
            p.nt = (q.n + a.sub - 1) / a.sub * a.ngrp;
            const int tiles = p.nt - p.tf;
            // The tile boundary nearest to each end of the share; both CTAs at a cut compute it alike.
            auto cut = [&](long long x) { return p.tf + min(tiles, __float2int_rn(__fdividef(__fmul_rn((float)x, (float)tiles), (float)cost))); };
            p.t0 = w0 <= cur ? p.tf : cut(w0 - cur);
            p.t1 = w1 >= cur + cost ? p.nt : cut(w1 - cur);
            const bool mine = p.t0 < p.t1 || (tiles == 0 && w0 <= cur);   // (a unit without rows: its weights are copied)
            cur += cost;
            if (++kt == nk) {
                kt = 0;
                if (++h == a.Hkv) {
                    h = 0;
                    do ++b;
                    while (b < a.s.B && (take(a), nk == 0));
                    if (b >= a.s.B) cur = w1 > cur ? w1 : cur;
                }
            }
            if (mine) return true;
        }
        return false;
    }
};

// The CTA's share for the warps that are `first`: each by itself for up to 32 sequences, with all T threads for more.
template <int T>
__device__ __forceinline__ void weight_locate(const WeightArgs& a, Line<T>& line, WeightWalk& walk, bool first) {
    int bad = 0;
    const auto cost = [&](int b) { return weight_cost(paged_seq(a.s, b, bad), a) * a.Hkv; };
    const auto share = [&](long long total, long long& w0, long long& w1) {
        line_share(total, blockIdx.x, kWeightCtas, line_inv(kWeightCtas), w0, w1);
    };
    int b;
    long long w0, w1, start;
    if (a.s.B <= 32) {
        if (!first) return;
        line_warp(a.s.B, cost, share, w0, w1, b, start);
    } else {
        share(line_total(line, a.s.B, cost), w0, w1);
        line_find(line, a.s.B, cost, w0, b, start);
    }
    if (blockIdx.x == 0 && bad) report_error(a.err, bad);
    if (first) walk.init(a, w0, w1, b, start);
}

// The sums of a unit, or of a part of it: one key per thread (key: within the tile).
__device__ __forceinline__ void weight_put(const WeightArgs& a, const WeightPart& p, int key, float sum, float old) {
    const int j = (p.kt << a.key_shift) + key;
    if (p.whole()) {
        if (j < p.len) a.w_out[((long long)p.b * a.Hkv + p.h) * a.s.cap + j] = old + sum;
        return;
    }
    const int slot = blockIdx.x * 2 + (p.t0 == p.tf ? 1 : 0);
    a.part[slot * kWeightKeys + key] = sum;
    if (key == 0) a.part_info[slot] = make_int4(p.t1 == p.nt ? 2 : 1, p.b, p.h, p.kt);
}
__device__ __forceinline__ float weight_old(const WeightArgs& a, const WeightPart& p, int key) {
    const int j = (p.kt << a.key_shift) + key;
    return a.w && p.whole() && j < p.len ? a.w[((long long)p.b * a.Hkv + p.h) * a.s.cap + j] : 0.f;
}

// Block j: the unit whose first part CTA j left in its slot 1; the following CTAs' slots 0 up to the one
// marked last are added in order.
__global__ void __launch_bounds__(kWeightKeys) weights_join_kernel(const WeightArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    const int4 rec = a.part_info[blockIdx.x * 2 + 1];
    if (rec.x == 0) return;
    const int j = (rec.w << a.key_shift) + threadIdx.x;
    const PagedRaw raw = paged_raw(a.s, rec.y);
    const bool in = (threadIdx.x >> a.key_shift) == 0 && j < min(max(raw.l, 0), a.s.cap);
    const long long o = ((long long)rec.y * a.Hkv + rec.z) * a.s.cap + j;
    const float old = a.w && in ? a.w[o] : 0.f;
    float sum = a.part[(blockIdx.x * 2 + 1) * kWeightKeys + threadIdx.x];
    const int lane = threadIdx.x & 31;
    for (int c0 = blockIdx.x + 1; c0 < gridDim.x; c0 += 32) {
        const int st = c0 + lane < gridDim.x ? a.part_info[(c0 + lane) * 2].x : 0;
        const unsigned ends = __ballot_sync(0xffffffffu, st == 2);
        unsigned have = __ballot_sync(0xffffffffu, st != 0) & (ends ? (ends & (0u - ends)) * 2u - 1u : 0xffffffffu);
        while (have) {                                     // four loads at a time, added in order
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                x[k] = have ? a.part[(c0 + __ffs(have) - 1) * 2 * kWeightKeys + threadIdx.x] : 0.f;
                have &= have - 1;
            }
            sum += (x[0] + x[1]) + (x[2] + x[3]);
        }
        if (ends) break;
    }
    if (in) a.w_out[o] = old + sum;
}

// ------------------------------------------------------------------ many rows, bf16
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

constexpr int kParts = 4;              // parts in the queue from warp 3 to the others
constexpr int kPartReaders = 19;       // all warps but 3

// D 32 runs as 64: TMA fills the columns behind a row's end with zeros.
template <int D>
struct ManyCfg {
    static constexpr int NCH = D / 64;
    static constexpr int CHUNK = 128 * 128;
    static constexpr int TILE = NCH * CHUNK;               // 128 rows of K or Q
    static constexpr int NK = D == 128 ? 3 : 4;            // key tiles (two to a unit) in shared memory
    static constexpr int NS = D == 128 ? 3 : 8;            // query tiles in the ring
    static constexpr int NL = 8;                           // log-sum-exps of so many (a slot of Q is free behind its
                                                           // products, they are read until the exponentials are done)
    static constexpr int SMEM = 1024 + (NK + NS) * TILE;
    static_assert(NS <= NL, "an issuer without keys passes the log-sum-exps of as many query tiles unseen");
    static constexpr int THREADS = 640;
};

// A unit holds two tiles of 128 keys, so that a query tile (16 KB at D 64, 32 at D 128; an SM receives some 35
// bytes a cycle) feeds two products.  Roles (20 warps): 0 producer (keys of a part, then query tiles through
// the ring), 1 and 2 UMMA issuers, 3 the CTA's parts and the log-sum-exps of every query tile, 4-19 the
// exponentials, a thread per key (TMEM lane): warps 4-7 and 12-15 the first 128 keys, the others the second,
// warps 4-11 the even query tiles, 12-19 the odd ones (a warp's loads and waits need others' products to fill
// the exponential units: with all tiles in eight warps 119 us at D 64 instead of 105; one issuer for both key
// tiles 120 at D 128 instead of 110).  S of key tile
// u and query tile i lies in TMEM columns 256 u + 128 (i % 2).  Dead rows of a query tile: those that TMA never
// writes are zero and their lse entry -inf; those that hold other sequences' rows are masked where they occur.
template <int D>
__global__ void __launch_bounds__(640, 1)
    weights_many_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const WeightArgs a) {
    using C = ManyCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sK = smem;
    uint8_t* sQ = smem + C::NK * C::TILE;
    __shared__ __align__(16) float s_nl[C::NL][128];       // -log2(e) lse
    __shared__ __align__(8) uint64_t bar_k_full[C::NK], bar_k_empty[C::NK], bar_q_full[C::NS], bar_q_empty[C::NS];
    __shared__ __align__(8) uint64_t bar_s_full[4], bar_s_free[4], bar_part_full[kParts], bar_part_empty[kParts], bar_final;
    __shared__ __align__(8) uint64_t bar_l_full[C::NL], bar_l_empty[C::NL];
    __shared__ Line<C::THREADS> line;
    __shared__ WeightPart s_part[kParts];
    __shared__ __align__(8) uint64_t bar_sum_full[2], bar_sum_free[2];
    __shared__ float s_sum[2][256];                        // the second half of the rows' sums, for parts in turn
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < C::NK; ++i) {
            mbar_init(smem_u32(&bar_k_full[i]), 1);
            mbar_init(smem_u32(&bar_k_empty[i]), 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(smem_u32(&bar_q_full[i]), 1);
            mbar_init(smem_u32(&bar_q_empty[i]), 2);       // the issuers
        }
        for (int i = 0; i < C::NL; ++i) {
            mbar_init(smem_u32(&bar_l_full[i]), 1);
            mbar_init(smem_u32(&bar_l_empty[i]), 8);       // the exponential warps of every second tile
        }
        for (int i = 0; i < 4; ++i) {                      // 2 u + item % 2
            mbar_init(smem_u32(&bar_s_full[i]), 2);        // the products, and the log-sum-exps
            mbar_init(smem_u32(&bar_s_free[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar_sum_full[i]), 8);
            mbar_init(smem_u32(&bar_sum_free[i]), 8);
        }
        for (int i = 0; i < kParts; ++i) {
            mbar_init(smem_u32(&bar_part_full[i]), 1);
            mbar_init(smem_u32(&bar_part_empty[i]), kPartReaders);
        }
        mbar_init(smem_u32(&bar_final), 2);
        abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    const int box = a.sub * a.gs;                          // rows of a query tile that TMA writes
    for (int i = tid; i < C::NS * C::NCH * (128 - box) * 8; i += C::THREADS) {
        const int u = i % 8, r = box + i / 8 % (128 - box), c = i / 8 / (128 - box);
        *reinterpret_cast<uint4*>(sQ + c * C::CHUNK + sw128_offset(r, u)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();                           // after the TMEM allocation
    griddep_wait();
    const uint32_t tm = tmem_slot;
    const WaitCtx w{a.err, &abort_flag, a.timeout_ns};
    WeightWalk walk;
    weight_locate(a, line, walk, warp == 3);
    WeightPart p;
    int npart = 0;
    auto next_part = [&]() -> bool {
        const int s = npart % kParts;
        if (!mbar_wait_warp(smem_u32(&bar_part_full[s]), (npart / kParts) & 1, w, SITE_PAGED_SEG)) return false;
        ++npart;
        p = s_part[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_part_empty[s]));
        return p.b >= 0;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int keys = 0, item = 0;                            // key tiles, query tiles
        bool ok = true;
        const int mask = (1 << a.c.ps_shift) - 1;
        const int npg = a.c.ps_shift >= 7 ? 1 : 128 >> a.c.ps_shift, rows = 128 / npg;
        while (ok && next_part()) {
            if (p.t0 == p.t1) continue;
            const int* trow = a.s.table + (size_t)p.b * a.s.W;
            int page[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int pos = p.kt * 256 + u * 128 + lane * rows;
                page[u] = lane < npg && pos < p.len ? __ldg(trow + (pos >> a.c.ps_shift)) : -1;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int k0 = p.kt * 256 + u * 128, s = keys % C::NK;
                if (k0 >= p.len) break;
                if (keys >= C::NK && !(ok = mbar_wait_warp(smem_u32(&bar_k_empty[s]), (keys / C::NK - 1) & 1, w, SITE_PAGED_KV_EMPTY))) break;
                if ((unsigned)page[u] >= (unsigned)a.c.n_pages) {  // (outside the pool TMA fills with zeros)
                    if (lane < npg && k0 + lane * rows < p.len) report_error(a.err, SITE_PAGED_PAGE);
                    page[u] = a.c.n_pages;
                }
                const uint32_t kf = smem_u32(&bar_k_full[s]);
                if (lane == 0) mbar_arrive_expect_tx(kf, C::TILE);
                __syncwarp();
                if (lane < npg)
#pragma unroll
                    for (int c = 0; c < C::NCH; ++c)
                        tma_load_4d(smem_u32(sK + s * C::TILE + c * C::CHUNK + lane * rows * 128), &tm_k, kf, c * 64, p.h, k0 & mask, page[u]);
                ++keys;
            }
            if (!ok) break;
            for (int t = p.t0; t < p.t1; ++t, ++item) {
                const int i = item % C::NS;
                if (item >= C::NS && !(ok = mbar_wait_warp(smem_u32(&bar_q_empty[i]), (item / C::NS - 1) & 1, w, SITE_PAGED_Q))) break;
                if (lane == 0) {
                    const uint32_t qf = smem_u32(&bar_q_full[i]);
                    mbar_arrive_expect_tx(qf, C::NCH * box * 128);
                    for (int c = 0; c < C::NCH; ++c)
                        tma_load_3d(smem_u32(sQ + i * C::TILE + c * C::CHUNK), &tm_q, qf, c * 64, p.h * a.G + t % a.ngrp * a.gs,
                                    p.tok0 + t / a.ngrp * a.sub);
                }
                __syncwarp();
            }
        }
        // Every copy this CTA started has landed before it ends.
        __syncwarp();
        if (lane == 0) {
            for (int i = max(0, keys - C::NK); i < keys; ++i)
                mbar_wait_drain(smem_u32(&bar_k_full[i % C::NK]), (i / C::NK) & 1, w, SITE_PAGED_DRAIN);
            for (int i = max(0, item - C::NS); i < item; ++i)
                mbar_wait_drain(smem_u32(&bar_q_full[i % C::NS]), (i / C::NS) & 1, w, SITE_PAGED_DRAIN);
        }
    } else if (warp < 3) {
        // ------------------------------------------------------------ UMMA issuer of key tile u
        constexpr uint32_t id_s = idesc_make(FMT_BF16, 128, 128, false, false);
        const uint64_t dk0 = sdesc(smem_u32(sK), 16, 1024), dq0 = sdesc(smem_u32(sQ), 16, 1024);
        const int u = warp - 1;
        int keys = 0, item = 0, uses[2] = {0, 0};          // uses: of S buffers 2 u + item % 2 so far
        bool ok = true;
        while (ok && next_part()) {
            if (p.t0 == p.t1) continue;
            const int nu = p.kt * 256 + 128 < p.len ? 2 : 1, kslot = (keys + u) % C::NK;
            const bool mine = u < nu;
            if (mine && !(ok = mbar_wait_warp(smem_u32(&bar_k_full[kslot]), ((keys + u) / C::NK) & 1, w, SITE_PAGED_KV_FULL))) break;
            const uint64_t dk = sdesc_add(dk0, kslot * C::TILE);
            for (int t = p.t0; t < p.t1; ++t, ++item) {
                const int i = item % C::NS, odd = item & 1, s = 2 * u + odd;
                if (!(ok = mbar_wait_warp(smem_u32(&bar_q_full[i]), (item / C::NS) & 1, w, SITE_PAGED_Q))) break;
                if (!mine) {
                    if (lane == 0) mbar_arrive(smem_u32(&bar_q_empty[i]));
                    __syncwarp();
                    continue;
                }
                const int n = odd ? uses[1]++ : uses[0]++;
                if (n >= 1 && !(ok = mbar_wait_warp(smem_u32(&bar_s_free[s]), (n - 1) & 1, w, SITE_PAGED_S_FULL))) break;
                tc_fence_after();
                const uint64_t dq = sdesc_add(dq0, i * C::TILE);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks * 32) >> 7) * C::CHUNK + ((ks * 32) & 127);
                        umma_ss<false>(tm + s * 128, sdesc_add(dk, off), sdesc_add(dq, off), id_s, ks > 0);
                    }
                }
                __syncwarp();
                // The exponentials wait for S alone, so its log-sum-exps have to be there.  A commit's arrival orders this
                // thread's products, not what warp 3 stored: an ordinary arrival beside it passes that on (a wait of
                // the exponentials' own costs D 64 99.2 -> 101.5 us).
                if (!(ok = mbar_wait_warp(smem_u32(&bar_l_full[item % C::NL]), (item / C::NL) & 1, w, SITE_PAGED_Q))) break;
                if (elect_one()) {
                    mbar_arrive(smem_u32(&bar_s_full[s]));
                    umma_commit(smem_u32(&bar_s_full[s]));
                    umma_commit(smem_u32(&bar_q_empty[i]));
                    if (t + 1 == p.t1) umma_commit(smem_u32(&bar_k_empty[kslot]));
                }
                __syncwarp();
            }
            keys += nu;
        }
        umma_commit_e(smem_u32(&bar_final));
    } else if (warp == 3) {
        // ------------------------------------------------------------ the CTA's parts, and their log-sum-exps
        if (lane < 2) a.part_info[blockIdx.x * 2 + lane] = make_int4(0, 0, 0, 0);
        __syncwarp();                                      // both in front of lane 0's arrivals, and so of any record
        // Part k + 1 is queued before the log-sum-exps of part k, which wait for the exponentials.
        int queued = 0, item = 0;
        bool more = true, ok = true;
        auto queue = [&](WeightPart& q) -> bool {
            const int s = queued % kParts;
            more = walk.next(a, q);
            if (!more) q.b = -1;
            if (queued >= kParts && !mbar_wait_warp(smem_u32(&bar_part_empty[s]), (queued / kParts - 1) & 1, w, SITE_PAGED_SEG)) return false;
            if (lane == 0) {
                s_part[s] = q;
                mbar_arrive(smem_u32(&bar_part_full[s]));
            }
            __syncwarp();
            ++queued;
            return true;
        };
        WeightPart ahead;
        ok = queue(ahead);
        int tk[4], hd[4];                                  // token and head of rows lane, lane + 32, ... of a tile
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            tk[k] = (lane + 32 * k) / a.gs;
            hd[k] = (lane + 32 * k) % a.gs;
        }
        while (ok && ahead.b >= 0) {
            p = ahead;
            if (!(ok = queue(ahead))) break;
            int tg = p.t0 / a.ngrp, th = p.t0 - tg * a.ngrp;
            const float* lse = a.lse + (long long)p.tok0 * a.Hq + p.h * a.G;
            for (int t0 = p.t0; ok && t0 < p.t1; t0 += 4) {   // four tiles' loads at a time: one by one their latency bounds all
                // (Loads without a condition, or each would be waited for in a branch of its own.)
                float v[4][4];
                unsigned in = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int tok = tg * a.sub, h0 = th * a.gs;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const bool live = t0 + j < p.t1 && lane + 32 * k < box && tok + tk[k] < p.n && h0 + hd[k] < a.G;
                        in |= (unsigned)live << (4 * j + k);
                        v[j][k] = __ldg(lse + (live ? (long long)(tok + tk[k]) * a.Hq + h0 + hd[k] : 0));
                    }
                    if (++th == a.ngrp) {
                        th = 0;
                        ++tg;
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (t0 + j >= p.t1) break;
                    const int i = item % C::NL;
                    if (item >= C::NL && !(ok = mbar_wait_warp(smem_u32(&bar_l_empty[i]), (item / C::NL - 1) & 1, w, SITE_PAGED_Q))) break;
#pragma unroll
                    for (int k = 0; k < 4; ++k) s_nl[i][lane + 32 * k] = in >> (4 * j + k) & 1u ? -kLog2e * v[j][k] : -INFINITY;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bar_l_full[i]));
                    ++item;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ exponentials
        const int u = ((warp - 4) >> 2) & 1, half = (warp - 4) >> 3, lk = (warp & 3) * 32 + lane, key = u * 128 + lk;
        const uint32_t lt = tm + ((uint32_t)((warp & 3) * 32) << 16) + u * 256;
        const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
        int item = 0, uses = 0, parts = 0;                 // query tiles; those of this half; parts
        bool ok = true;
        while (ok && next_part()) {
            const int k0 = p.kt * 256 + u * 128;           // the warps' first key
            const bool mine = k0 < p.len;
            const float old = half == 0 ? weight_old(a, p, key) : 0.f;
            float2 s2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            // Every second query tile is this half's, in S buffer `half`.
            const int skip = (item ^ half) & 1, n = p.t1 - p.t0;
            // Tiles t_lo .. t_hi-1 are full and see all of the warps' keys.
            const int t_lo = (max(0, k0 + 127 - (p.len - p.n)) + a.sub - 1) / a.sub * a.ngrp;
            const int t_hi = a.G % a.gs ? 0 : p.n / a.sub * a.ngrp;
            for (int j = skip; j < n; j += 2) {
                const int i = (item + j) % C::NL;
                if (!mine && !(ok = mbar_wait_warp(smem_u32(&bar_l_full[i]), ((item + j) / C::NL) & 1, w, SITE_PAGED_Q))) break;
                if (mine) {                                // (the issuer waited for the log-sum-exps, and passes them on)
                    if (!(ok = mbar_wait_warp(smem_u32(&bar_s_full[2 * u + half]), uses & 1, w, SITE_PAGED_S_FULL))) break;
                    ++uses;
                    tc_fence_after();
                    const int t = p.t0 + j;
                    int c_min = 0, live = 128;             // rows c_min .. live-1 of the tile see this thread's key
                    const float4* nl = reinterpret_cast<const float4*>(s_nl[i]);
                    // (Edge tiles in a loop: a call with few tiles waits for its instructions, 21.0 -> 20 us.)
                    auto tile = [&](auto edge) {
                        constexpr int kUnroll = decltype(edge)::value ? 1 : 4;
#pragma unroll kUnroll
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            uint32_t x[32];
                            tmem_ld_cols<1>(lt + half * 128 + c0, x);
                            if (c0 == 96) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(smem_u32(&bar_s_free[2 * u + half]));
                            }
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 l4 = nl[(c0 + e) / 4];
                                const float2 y0 = __ffma2_rn(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), sl2, make_float2(l4.x, l4.y));
                                const float2 y1 = __ffma2_rn(make_float2(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), sl2, make_float2(l4.z, l4.w));
                                float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
                                if constexpr (decltype(edge)::value) {
                                    const int c = c0 + e;
                                    p0.x = c >= c_min && c < live ? p0.x : 0.f;
                                    p0.y = c + 1 >= c_min && c + 1 < live ? p0.y : 0.f;
                                    p1.x = c + 2 >= c_min && c + 2 < live ? p1.x : 0.f;
                                    p1.y = c + 3 >= c_min && c + 3 < live ? p1.y : 0.f;
                                }
                                s2[e / 4 % 2 * 2] = __fadd2_rn(s2[e / 4 % 2 * 2], p0);
                                s2[e / 4 % 2 * 2 + 1] = __fadd2_rn(s2[e / 4 % 2 * 2 + 1], p1);
                            }
                        }
                    };
                    if (t >= t_lo && t < t_hi) {
                        tile(std::false_type());
                    } else {
                        const int tg = t / a.ngrp, th = t - tg * a.ngrp, tok = tg * a.sub;
                        live = min(a.gs, a.G - th * a.gs) * min(a.sub, p.n - tok);
                        const int d = k0 + lk - (p.len - p.n + tok);
                        c_min = d <= 0 ? 0 : d >= a.sub ? 128 : d * a.gs;
                        tile(std::true_type());
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_l_empty[i]));
            }
            item += n;
            if (!ok) break;
            const float sum = ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
            const int k = parts & 1;
            if (half == 1) {
                if (parts >= 2 && !(ok = mbar_wait_warp(smem_u32(&bar_sum_free[k]), (parts / 2 - 1) & 1, w, SITE_PAGED_O_FULL))) break;
                s_sum[k][key] = sum;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_sum_full[k]));
            } else {
                if (!(ok = mbar_wait_warp(smem_u32(&bar_sum_full[k]), (parts / 2) & 1, w, SITE_PAGED_O_FULL))) break;
                const float other = s_sum[k][key];
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_sum_free[k]));
                weight_put(a, p, key, sum + other, old);
            }
            ++parts;
        }
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        mbar_wait_drain(smem_u32(&bar_final), 0, w, SITE_PAGED_DRAIN);
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------ many rows, fp32
// Eight warps: two halves of the 128 keys (two keys per lane, their rows in registers) times four shares of
// every tile of 64 query rows, which lie in shared memory and are broadcast: 16 bytes feed four packed
// FMAs, so the FMAs bound it.
template <int D>
struct ManyF32Cfg {
    static constexpr int U = D / 4, RT = 64;
    static constexpr int K_BYTES = 128 * D * 4, Q_BYTES = RT * D * 4;
    static constexpr int SMEM = K_BYTES + 2 * Q_BYTES;
    static constexpr int THREADS = 256;
};

template <int D>
__global__ void __launch_bounds__(256, 1) weights_many_f32_kernel(const WeightArgs a) {
    using C = ManyF32Cfg<D>;
    constexpr int U = C::U, RT = C::RT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Line<C::THREADS> line;
    __shared__ WeightPart s_part;
    __shared__ float s_nl[2][RT], s_sum[4][128];
    __shared__ int s_lim[2][RT];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = warp & 1, rg = warp >> 1;
    uint8_t* const sQ = smem + C::K_BYTES;
    griddep_launch_dependents();
    griddep_wait();
    WeightWalk walk;
    weight_locate(a, line, walk, warp == 0);
    if (tid < 2) a.part_info[blockIdx.x * 2 + tid] = make_int4(0, 0, 0, 0);
    for (;;) {
        __syncthreads();                                   // (the records are cleared; the part before is done)
        if (warp == 0) {
            WeightPart n;
            if (!walk.next(a, n)) n.b = -1;
            if (lane == 0) s_part = n;
        }
        __syncthreads();
        const WeightPart p = s_part;
        if (p.b < 0) break;
        const int base = p.len - p.n;
        auto load_q = [&](int t, int buf) {
            if (t < p.t1) {
                const int tok = t / a.ngrp * a.sub, h0 = t % a.ngrp * a.gs;
                auto live = [&](int r) { return r < a.sub * a.gs && tok + r / a.gs < p.n && h0 + r % a.gs < a.G; };
#pragma unroll
                for (int i = tid; i < RT * U; i += C::THREADS) {
                    const int r = i / U;
                    const bool in = live(r);
                    const float* src = static_cast<const float*>(a.q);
                    if (in) src += (long long)(p.tok0 + tok + r / a.gs) * a.q_ld + (long long)(p.h * a.G + h0 + r % a.gs) * D + i % U * 4;
                    cp_async16(smem_u32(sQ + buf * C::Q_BYTES) + i * 16, src, in);
                }
                if (tid < RT) {
                    const bool in = live(tid);
                    s_nl[buf][tid] = in ? -kLog2e * __ldg(a.lse + (long long)(p.tok0 + tok + tid / a.gs) * a.Hq + p.h * a.G + h0 + tid % a.gs)
                                        : -INFINITY;
                    s_lim[buf][tid] = in ? base + tok + tid / a.gs + 1 : 0;
                }
            }
            cp_async_commit();
        };
        if (p.t0 < p.t1 && warp < 4) {
            const int first = p.kt * 128 + warp * 32;
            const int page = checked_page(a.c, page_at(a.c, a.s.table + (size_t)p.b * a.s.W, first + lane, p.len), first + lane, p.len, a.err);
            load_keys<U>(smem_u32(smem) + warp * 32 * D * 4, static_cast<const char*>(a.c.k) + (long long)p.h * a.c.head_stride * 4, a.c, 4,
                         first, p.len, page, lane);
        }
        load_q(p.t0, 0);                                   // (the keys are of this group of copies)
        const float old = tid < 128 ? weight_old(a, p, tid) : 0.f;
        float4 kf[2][U];
        float sum[2] = {0.f, 0.f};
        for (int t = p.t0; t < p.t1; ++t) {
            const int buf = (t - p.t0) & 1;
            load_q(t + 1, buf ^ 1);
            cp_async_wait<1>();
            __syncthreads();
            if (t == p.t0)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        kf[k][u] = reinterpret_cast<const float4*>(smem)[(half * 2 + k) * 32 * U + tile_unit<U>(lane, u)];
            const float4* q4 = reinterpret_cast<const float4*>(sQ + buf * C::Q_BYTES);
            const int j0 = p.kt * 128 + half * 64 + lane;
#pragma unroll 2
            for (int r = rg; r < RT; r += 4) {
                float2 s[2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) s[k][0] = s[k][1] = make_float2(0.f, 0.f);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float4 qv = q4[r * U + u];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        s[k][0] = __ffma2_rn(make_float2(kf[k][u].x, kf[k][u].y), make_float2(qv.x, qv.y), s[k][0]);
                        s[k][1] = __ffma2_rn(make_float2(kf[k][u].z, kf[k][u].w), make_float2(qv.z, qv.w), s[k][1]);
                    }
                }
                const float nl = s_nl[buf][r];
                const int lim = s_lim[buf][r];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x = (s[k][0].x + s[k][0].y) + (s[k][1].x + s[k][1].y);
                    const float e = ex2(fmaf(x, a.scale_log2, nl));
                    sum[k] += j0 + 32 * k < lim ? e : 0.f;
                }
            }
            __syncthreads();                               // the buffer is read before it is filled again
        }
        cp_async_wait<0>();
        s_sum[rg][half * 64 + lane] = sum[0];
        s_sum[rg][half * 64 + 32 + lane] = sum[1];
        __syncthreads();
        if (tid < 128) weight_put(a, p, tid, (s_sum[0][tid] + s_sum[1][tid]) + (s_sum[2][tid] + s_sum[3][tid]), old);
    }
}

template <int D, int RC, bool F32>
cudaError_t launch_few_t(const WeightArgs& a, cudaStream_t st) {
    using C = FewCfg<D, RC, F32>;
    static_assert(C::CTAS * (C::SMEM + 4096) <= 227 * 1024, "shared memory");
    auto kfn = weights_few_kernel<D, RC, F32>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kfn, C::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(C::CTAS * kWeightCtas), dim3(kFewThreads), C::SMEM, st, a);
}

template <int D>
cudaError_t launch_many_t(const CUtensorMap& tq, const CUtensorMap& tk, const WeightArgs& a, cudaStream_t st) {
    using C = ManyCfg<D>;
    static_assert(C::SMEM + 12 * 1024 <= 227 * 1024, "shared memory");
    auto kfn = weights_many_kernel<D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kfn, C::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(kWeightCtas), dim3(C::THREADS), C::SMEM, st, tq, tk, a);
}

template <int D>
cudaError_t launch_many_f32_t(const WeightArgs& a, cudaStream_t st) {
    using C = ManyF32Cfg<D>;
    auto kfn = weights_many_f32_kernel<D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kfn, C::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(kWeightCtas), dim3(C::THREADS), C::SMEM, st, a);
}

}  // namespace

WeightKind weight_kind(bool f32, int G, int max_new) {
    const long long rows = (long long)G * max_new;
    if (rows > 32) return f32 ? WEIGHTS_MANY_F32 : WEIGHTS_MANY;
    return rows <= 4 ? WEIGHTS_FEW4 : rows <= 8 ? WEIGHTS_FEW8 : rows <= 16 ? WEIGHTS_FEW16 : WEIGHTS_FEW32;
}

void weight_split(WeightKind kind, WeightArgs& a) {
    const int rt = kind == WEIGHTS_MANY_F32 ? 64 : 128;
    a.gs = a.G < rt ? a.G : rt;
    a.ngrp = (a.G + a.gs - 1) / a.gs;
    a.sub = rt / a.gs;
    a.ovh = 2 * a.sub;                                     // the ends of a unit, in tokens
    a.key_shift = kind == WEIGHTS_MANY_F32 ? 7 : 8;
}

cudaError_t launch_paged_weights(WeightKind kind, bool f32, int D, const CUtensorMap& tq, const CUtensorMap& tk,
                                 const WeightArgs& a, cudaStream_t st) {
    cudaError_t e = cudaErrorInvalidValue;
    if (kind == WEIGHTS_MANY) e = D == 128 ? launch_many_t<128>(tq, tk, a, st) : launch_many_t<64>(tq, tk, a, st);
    else if (kind == WEIGHTS_MANY_F32) e = D == 64 ? launch_many_f32_t<64>(a, st) : launch_many_f32_t<32>(a, st);
    else if (f32) {                                        // (eight rows at a time; K is read again from shared memory)
        if (D == 32) e = kind == WEIGHTS_FEW4 ? launch_few_t<32, 4, true>(a, st) : launch_few_t<32, 8, true>(a, st);
        if (D == 64) e = kind == WEIGHTS_FEW4 ? launch_few_t<64, 4, true>(a, st) : launch_few_t<64, 8, true>(a, st);
    } else {
        const int rc = kind == WEIGHTS_FEW32 ? 32 : kind == WEIGHTS_FEW16 ? 16 : 8;
        if (D == 32) e = rc == 8 ? launch_few_t<32, 8, false>(a, st) : rc == 16 ? launch_few_t<32, 16, false>(a, st) : launch_few_t<32, 32, false>(a, st);
        if (D == 64) e = rc == 8 ? launch_few_t<64, 8, false>(a, st) : rc == 16 ? launch_few_t<64, 16, false>(a, st) : launch_few_t<64, 32, false>(a, st);
        if (D == 128) e = rc == 8 ? launch_few_t<128, 8, false>(a, st) : rc == 16 ? launch_few_t<128, 16, false>(a, st) : launch_few_t<128, 32, false>(a, st);
    }
    if (e != cudaSuccess || (kind != WEIGHTS_MANY && kind != WEIGHTS_MANY_F32)) return e;
    return launch_k(weights_join_kernel, dim3(kWeightCtas), dim3(kWeightKeys), 0, st, a);
}

}  // namespace ne
