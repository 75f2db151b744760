// paged_tiles.cu -- attention of chunks of new tokens over the paged cache on tcgen05
// tensor cores, bf16, head_dim 64 and 128.
//
// The query heads of a kv head read the same keys, so a tile's 128 rows are (token, head)
// pairs: 128 / G tokens times G heads, token first, as TMA lays a [tokens, heads, 64] box
// down.  A work unit holds two such subtiles (u = 0, 1), which share every K and V tile:
// 128 keys, fetched page by page (one TMA box per page and 64 columns, one lane per page).
// The keys are rotated already, so between TMA and the tensor cores nothing touches them.
// Units and their shares of the key axis: paged_sched.cuh.
//
// Per unit and key tile, 4 * 256 * 128 * D flops against 512 D bytes: 16 D cycles of the tensor
// core (8192 dense bf16 flops a cycle) and 1024 of the exponential units (32 results a cycle),
// so products bound D 128 and exponentials come close to them at D 64.  The two subtiles
// alternate: while the softmax warps of one work on its S tile, the tensor core runs the other's
// PV and next S.  Roles (12 warps):
//   warp 0       producer: Q pair of the unit, then K and V tiles through an NS-slot ring.
//   warp 1       UMMA issuer (owns the 512 TMEM columns); at D 64 one of two, warp 2 the other, each
//                for a subtile.  Per tile t: O_u += P_u(t) V(t) once P_u(t) is there, and S_u(t + 1) =
//                Q_u K(t + 1)^T.  At D 64, where P has columns of its own, S(t + 1) goes first, as soon
//                as S(t) is in registers.  At D 128 P lies over S, and S(t + 1) goes right behind the PV
//                (one thread's UMMAs run in order, so it cannot overtake it, and S(t + 1) complete means
//                PV(t) complete).
//   warp 2       zeroes the V rows behind a sequence's length in the tile that holds it (P is 0
//                there, but 0 x NaN is not).
//   warp 3       finds the CTA's parts (paged_sched.cuh) and queues them for the others.
//   warps 4-11   softmax: thread r of subtile u owns row r (TMEM lane r).
// TMEM: S_u at 128 u, O_u behind both; P_u (bf16) over S_u's first half at D 128, where TMEM
// is full, in columns of its own at D 64.
// Weights are rounded to bf16 for the product (half a step, 2^-8 of each weight, as the
// training forward does); maximum and sum stay fp32, and the sum is of the unrounded weights.
// Measured (GB300): 2048 new tokens over 16384 positions, 16/4 heads of 128, pages of 64: 185 us
// with the join, 1.39 PFLOP/s (73% of the 1.89 measured for a bf16 GEMM; 182 us with the cache in
// the L2, 192 with pages of 16, where a tile takes 8 boxes of each kind), the tensor pipe 63% busy:
// a subtile's chain, PV + S on the tensor core (0.54 us) and its softmax (0.7 us, then waits), takes 1.45 us per
// tile, longer than both subtiles' tensor work.  12/4 heads of 64: 102 us, 0.94 PFLOP/s (100 in
// the L2; pages of 16: 110).  With one
// issuer for both subtiles that took 122 us: waiting for one subtile's P it could not start the
// other's S, which tied the two softmaxes to the same phase.  At D 128 two issuers are slower (196
// us): the tensor core is the longer half there, and two streams of UMMAs delay each other.
// Tried and left out: two threads per row in 16 softmax warps (chunk 199 us), PV in two halves
// (0.4% at D 128), the second subtile started half a tile late (no change), weights taken before
// the tile's maximum is known (the scores stay live: 2 KB of spills).
// Every wait is bounded; a CTA that gives up reports, drains its copies and UMMAs, frees its
// TMEM and ends.
#include <cuda_bf16.h>
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kSegs = 4;               // parts in the queue from warp 3 to the others
constexpr int kSegReaders = 11;        // warps 0, 1, 2 and 4-11

template <int D>
struct TileCfg {
    static constexpr int BN = 128;                         // keys of a tile
    static constexpr int ROWB = D * 2;
    static constexpr int NCH = ROWB / 128;                 // 64-column chunks
    static constexpr int CHUNK = 128 * 128;                // bytes of a chunk of 128 rows
    static constexpr int TILE = NCH * CHUNK;               // one Q subtile, or one K or V tile
    static constexpr int NS = D == 128 ? 5 : 12;           // ring slots
    static constexpr int SMEM = 1024 + 2 * TILE + NS * TILE;
    static constexpr int THREADS = 384;
    static constexpr int O_COL = 256;                      // O_u at O_COL + u D
    // P in columns of its own where TMEM has them left (D 64): the next S then starts as soon as
    // this one has been read into registers, instead of after its PV.
    static constexpr bool SEP = D == 64;
    static constexpr int P_COL = SEP ? O_COL + 2 * D : 0;  // P_u at P_COL + u P_STEP
    static constexpr int P_STEP = SEP ? 64 : 128;
    static constexpr int ISSUERS = SEP ? 2 : 1;
    static_assert(SMEM + 1536 <= 227 * 1024, "shared memory (with the static part)");
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint4 shfl_xor4(const uint4& v, int m) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, v.x, m), __shfl_xor_sync(0xffffffffu, v.y, m),
                      __shfl_xor_sync(0xffffffffu, v.z, m), __shfl_xor_sync(0xffffffffu, v.w, m));
}
// Transposes a 4 x 4 block of 16-byte units held by four neighbouring lanes: afterwards lane l
// of the four holds unit l of each of them.
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int l) {
    const uint4 a = shfl_xor4(l & 1 ? v[0] : v[1], 1), b = shfl_xor4(l & 1 ? v[2] : v[3], 1);
    if (l & 1) {
        v[0] = a;
        v[2] = b;
    } else {
        v[1] = a;
        v[3] = b;
    }
    const uint4 c = shfl_xor4(l & 2 ? v[0] : v[2], 2), d = shfl_xor4(l & 2 ? v[1] : v[3], 2);
    if (l & 2) {
        v[0] = c;
        v[1] = d;
    } else {
        v[2] = c;
        v[3] = d;
    }
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const PagedAttnArgs a) {
    using C = TileCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;                                    // two subtiles
    uint8_t* sRing = smem + 2 * C::TILE;
    __shared__ __align__(8) uint64_t bar_q_full, bar_q_empty, bar_vfix[2], bar_final;
    __shared__ __align__(8) uint64_t bar_full[C::NS], bar_empty[C::NS];
    __shared__ __align__(8) uint64_t bar_s_full[2], bar_p_ready[2], bar_o_full[2], bar_s_free[2];
    __shared__ __align__(8) uint64_t bar_seg_full[kSegs], bar_seg_empty[kSegs];
    __shared__ PagedLocate loc;
    __shared__ PagedSeg s_seg[kSegs];                      // the CTA's parts in order (b < 0: the end)
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(smem_u32(&bar_q_full), 1);
        mbar_init(smem_u32(&bar_q_empty), C::ISSUERS);     // their commits after a unit's last S
        mbar_init(smem_u32(&bar_final), C::ISSUERS);
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(smem_u32(&bar_full[s]), 1);
            mbar_init(smem_u32(&bar_empty[s]), 2);         // warps 1 and 2, by a commit where they multiply
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(smem_u32(&bar_s_full[u]), 1);
            mbar_init(smem_u32(&bar_p_ready[u]), 128);
            mbar_init(smem_u32(&bar_o_full[u]), 1);        // a part's last PV; SEP: every PV
            mbar_init(smem_u32(&bar_s_free[u]), 128);      // SEP: S is in registers
            mbar_init(smem_u32(&bar_vfix[u]), 32);         // the k-th fix arrives on k % 2: warp 2 can be one
                                                           // fix ahead of the issuer (one part, by its Q), not two
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(smem_u32(&bar_seg_full[s]), 1);
            mbar_init(smem_u32(&bar_seg_empty[s]), kSegReaders);
        }
        abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();                           // after the TMEM allocation
    griddep_wait();
    const uint32_t tm = tmem_slot;
    const WaitCtx w{a.err, &abort_flag, a.timeout_ns};
    const int sub = a.p.sub;                               // tokens of a subtile
    PagedSeg g;
    int nseg = 0;
    // The CTA's next part, from the queue; false at its end (or when a wait ran out).  One warp
    // finds the parts for all: the arithmetic has long latencies and a copy of it in every role
    // cost each of them microseconds of instruction fetches at the start.
    auto next_part = [&]() -> bool {
        const int s = nseg % kSegs;
        if (!mbar_wait_warp(smem_u32(&bar_seg_full[s]), (nseg / kSegs) & 1, w, SITE_PAGED_SEG)) return false;
        ++nseg;
        g = s_seg[s];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_seg_empty[s]));
        return g.b >= 0;
    };
    // Where the CTA's share begins, warp 3 finds alone among up to 32 sequences, all warps among more.
    if (a.s.B > 32) paged_locate<C::THREADS>(a, blockIdx.x, loc, blockIdx.x == 0);
    // A part's K tile t sits at ring index 2 i, its V tile at 2 i + 1, i counting the CTA's tiles.
    // Zeros for the rows of the V tile at ring index i (keys of tile t) that lie behind the length.
    auto zero_v = [&](int i, int t) {
        uint8_t* v = sRing + (i % C::NS) * C::TILE;
        const int r0 = g.len - t * C::BN;
        for (int x = lane; x < (C::BN - r0) * C::NCH * 8; x += 32) {
            const int r = r0 + x / (C::NCH * 8), e = x % (C::NCH * 8);
            *reinterpret_cast<uint4*>(v + (e >> 3) * C::CHUNK + sw128_offset(r, e & 7)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        int seg = 0, item = 0;
        bool ok = true;
        const int mask = (1 << a.c.ps_shift) - 1;
        const int npg = a.c.ps_shift >= 7 ? 1 : 128 >> a.c.ps_shift;   // pages of a tile
        const int rows = 128 / npg;
        while (ok && next_part()) {
            if (g.t0 == g.t1) continue;                    // no keys: the softmax warps write the rows
            const int* trow = a.s.table + (size_t)g.b * a.s.W;
            auto page = [&](int t) -> int {                // page of this lane's part of tile t
                const int pos = t * C::BN + lane * rows;
                return lane < npg && pos < g.kv ? __ldg(trow + (pos >> a.c.ps_shift)) : -1;
            };
            int next = page(g.t0), next1 = g.t0 + 1 < g.t1 ? page(g.t0 + 1) : 0;   // two tiles ahead
            if (seg > 0 && !(ok = mbar_wait_warp(smem_u32(&bar_q_empty), (seg - 1) & 1, w, SITE_PAGED_Q))) break;
            const int n_sub = g.ntok > sub ? 2 : 1;
            if (lane == 0) {
                const uint32_t qf = smem_u32(&bar_q_full);
                mbar_arrive_expect_tx(qf, n_sub * C::NCH * sub * a.G * 128);
                for (int u = 0; u < n_sub; ++u)
                    for (int c = 0; c < C::NCH; ++c)
                        tma_load_3d(smem_u32(sQ + u * C::TILE + c * C::CHUNK), &tm_q, qf, c * 64, g.hg * a.G,
                                    g.tok0 + g.tok + u * sub);
            }
            ++seg;
            for (int t = g.t0; ok && t < g.t1; ++t) {
                // (Looked at only now: a branch on the id at its load would wait for it.)  An id
                // outside the pool reads as zeros: TMA fills what lies behind the last page.
                int p = next;
                if ((unsigned)p >= (unsigned)a.c.n_pages) {
                    if (lane < npg && t * C::BN + lane * rows < g.kv) report_error(a.err, SITE_PAGED_PAGE);
                    p = a.c.n_pages;
                }
                next = next1;
                if (t + 2 < g.t1) next1 = page(t + 2);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++item) {
                    const int s = item % C::NS;
                    if (item >= C::NS &&
                        !(ok = mbar_wait_warp(smem_u32(&bar_empty[s]), (item / C::NS - 1) & 1, w, SITE_PAGED_KV_EMPTY)))
                        break;
                    const uint32_t full = smem_u32(&bar_full[s]);
                    if (lane == 0) mbar_arrive_expect_tx(full, C::TILE);
                    __syncwarp();
                    if (lane < npg)
#pragma unroll
                        for (int c = 0; c < C::NCH; ++c)
                            tma_load_4d(smem_u32(sRing + s * C::TILE + c * C::CHUNK + lane * rows * 128), kv ? &tm_v : &tm_k,
                                        full, c * 64, g.hg, (t * C::BN) & mask, p);
                }
            }
        }
        // Every copy this CTA started has landed before it ends.
        __syncwarp();
        if (lane == 0) {
            if (seg > 0) mbar_wait_drain(smem_u32(&bar_q_full), (seg - 1) & 1, w, SITE_PAGED_DRAIN);
            for (int i = max(0, item - C::NS); i < item; ++i)
                mbar_wait_drain(smem_u32(&bar_full[i % C::NS]), (i / C::NS) & 1, w, SITE_PAGED_DRAIN);
        }
    } else if (warp == 1 || (C::SEP && warp == 2)) {
        // ------------------------------------------------------------ UMMA issuers
        constexpr int NU = C::SEP ? 1 : 2;                 // subtiles of this warp: u0 .. u0 + NU-1
        const int u0 = C::SEP ? warp - 1 : 0;
        constexpr uint32_t id_s = idesc_make(FMT_BF16, 128, C::BN, false, false);
        constexpr uint32_t id_o = idesc_make(FMT_BF16, 128, D, false, true);
        const uint64_t dq0 = sdesc(smem_u32(sQ) + u0 * C::TILE, 16, 1024);
        const uint64_t dk0 = sdesc(smem_u32(sRing), 16, 1024);
        const uint64_t dv0 = sdesc(smem_u32(sRing), C::CHUNK, 1024);
        int seg = 0, item = 0, tiles[NU] = {}, s_tiles = 0, fixes = 0;
        bool ok = true;
        auto s_mmas = [&](int i, int k_item) {             // S of subtile u0 + i
            const uint64_t dq = sdesc_add(dq0, i * C::TILE), dk = sdesc_add(dk0, (k_item % C::NS) * C::TILE);
#pragma unroll
            for (int ks = 0; ks < C::ROWB / 32; ++ks) {
                const uint32_t off = ((ks * 32) >> 7) * C::CHUNK + ((ks * 32) & 127);
                umma_ss<false>(tm + (u0 + i) * 128, sdesc_add(dq, off), sdesc_add(dk, off), id_s, ks > 0);
            }
            umma_commit(smem_u32(&bar_s_full[u0 + i]));
        };
        // After this warp's last S of a K tile: its slot, and after the part's last S the Q.
        auto s_done = [&](int k_item, bool last) {
            umma_commit(smem_u32(&bar_empty[k_item % C::NS]));
            if (last) umma_commit(smem_u32(&bar_q_empty));
        };
        auto full = [&](int i) {
            const bool r = mbar_wait_warp(smem_u32(&bar_full[i % C::NS]), (i / C::NS) & 1, w, SITE_PAGED_KV_FULL);
            tc_fence_after();
            return r;
        };
        // S's columns hold no S that is still to be read (SEP; otherwise the PV in front of the
        // next S, on this same thread, says so).
        auto s_free = [&]() -> bool {
            if (!C::SEP || s_tiles == 0) return true;
            const bool r = mbar_wait_warp(smem_u32(&bar_s_free[u0]), (s_tiles - 1) & 1, w, SITE_PAGED_S_FULL);
            tc_fence_after();
            return r;
        };
        // The V tile at ring index i, with zeros behind the length.
        auto v_tile = [&](int i, int t) -> bool {
            if (!full(i)) return false;
            if ((t + 1) * C::BN <= g.len) return true;
            const int k = fixes++;
            if (!C::SEP || u0 == 0) return mbar_wait_warp(smem_u32(&bar_vfix[k & 1]), (k >> 1) & 1, w, SITE_PAGED_KV_FULL);
            zero_v(i, t);
            mbar_arrive(smem_u32(&bar_vfix[k & 1]));
            __syncwarp();
            return true;
        };
        while (ok && next_part()) {
            if (g.t0 == g.t1) continue;
            const int nt = g.t1 - g.t0;
            const int mine = C::SEP ? (g.ntok > u0 * sub ? 1 : 0) : (g.ntok > sub ? 2 : 1);
            // (SEP: a warp without a subtile in this part waits for its Q too, or it could take the
            // next part's wait for this one's.)
            if (!(ok = mbar_wait_warp(smem_u32(&bar_q_full), seg & 1, w, SITE_PAGED_Q))) break;
            if (C::SEP && mine == 0) {                     // nothing to multiply: it zeroes V and lets go
                for (int i = 0; ok && i < 2 * nt; ++i) {
                    if (!(ok = i & 1 ? v_tile(item + i, g.t0 + (i >> 1)) : full(item + i))) break;
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&bar_empty[(item + i) % C::NS]));
                        if (i == 0) mbar_arrive(smem_u32(&bar_q_empty));
                    }
                    __syncwarp();
                }
                item += 2 * nt;
                ++seg;
                continue;
            }
            if (!(ok = full(item) && s_free())) break;
            ++s_tiles;
            if (elect_one()) {
                s_mmas(0, item);
                if (NU == 2 && mine == 2) s_mmas(NU - 1, item);
                s_done(item, nt == 1);
            }
            __syncwarp();
            for (int t = 0; ok && t < nt; ++t) {
                const int vi = item + 2 * t + 1, kn = item + 2 * t + 2;
                const bool more = t + 1 < nt;
                const uint64_t dv = sdesc_add(dv0, (vi % C::NS) * C::TILE);
                if (C::SEP && more) {
                    if (!(ok = full(kn) && s_free())) break;
                    ++s_tiles;
                    if (elect_one()) {
                        s_mmas(0, kn);
                        s_done(kn, t + 2 == nt);
                    }
                    __syncwarp();
                }
                if (!(ok = v_tile(vi, g.t0 + t))) break;
                if (!C::SEP && more && !(ok = full(kn))) break;
#pragma unroll
                for (int i = 0; i < NU; ++i) {
                    if (i >= mine) break;
                    const int u = u0 + i;
                    if (!(ok = mbar_wait_warp(smem_u32(&bar_p_ready[u]), tiles[i] & 1, w, SITE_PAGED_P_READY))) break;
                    ++tiles[i];
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < C::BN / 16; ++ks)
                            umma_ts<false>(tm + C::O_COL + u * D, tm + C::P_COL + u * C::P_STEP + ks * 8,
                                           sdesc_add(dv, ks * 16 * 128), id_o, (t > 0 || ks > 0) ? 1u : 0u);
                        if (C::SEP || !more) umma_commit(smem_u32(&bar_o_full[u]));
                        if (!C::SEP && more) s_mmas(i, kn);
                        if (i == mine - 1) {
                            umma_commit(smem_u32(&bar_empty[vi % C::NS]));
                            if (!C::SEP && more) s_done(kn, t + 2 == nt);
                        }
                    }
                    __syncwarp();
                }
            }
            item += 2 * nt;
            ++seg;
        }
        umma_commit_e(smem_u32(&bar_final));
    } else if (warp == 2) {
        // ------------------------------------------------------------ V rows behind the length (D 128)
        // It follows every slot's phases and releases each along with the issuer, so neither can
        // fall a phase behind the other.
        int item = 0, fixes = 0;
        bool ok = true;
        while (ok && next_part()) {
            for (int i = 0; ok && i < 2 * (g.t1 - g.t0); ++i, ++item) {
                const int s = item % C::NS, t = g.t0 + (i >> 1);
                if (!(ok = mbar_wait_warp(smem_u32(&bar_full[s]), (item / C::NS) & 1, w, SITE_PAGED_KV_FULL))) break;
                if ((i & 1) && (t + 1) * C::BN > g.len) {
                    zero_v(item, t);
                    mbar_arrive(smem_u32(&bar_vfix[fixes++ & 1]));
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_empty[s]));
            }
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ the CTA's parts
        if (lane < 2) a.part_info[blockIdx.x * 2 + lane] = make_int4(0, 0, 0, 0);
        __syncwarp();                                      // both in front of lane 0's arrivals, and so of any record
        PagedWalk walk;
        if (a.s.B <= 32) paged_locate_warp(a, blockIdx.x, walk, blockIdx.x == 0);
        else walk.init(a, loc.w0, loc.w1, loc.snap, loc.b, loc.start);
        bool more = true;
        for (int k = 0; more; ++k) {
            const int s = k % kSegs;
            more = walk.next(a, g);
            if (!more) g.b = -1;
            if (k >= kSegs &&
                !mbar_wait_warp(smem_u32(&bar_seg_empty[s]), (k / kSegs - 1) & 1, w, SITE_PAGED_SEG))
                break;
            if (lane == 0) {
                s_seg[s] = g;
                mbar_arrive(smem_u32(&bar_seg_full[s]));
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ softmax of subtile u
        const int u = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;              // row = TMEM lane
        const uint32_t lt = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t sc = lt + u * 128, oc = lt + C::O_COL + u * D, pc = lt + C::P_COL + u * C::P_STEP;
        const float sl2 = a.scale_log2;
        int tiles = 0, parts = 0;
        bool ok = true;
        while (ok && next_part()) {
            const int ntok = min(sub, g.ntok - u * sub);   // tokens of this subtile
            const int live_rows = ntok * a.G;
            if (ntok <= 0) continue;
            const bool live = r < live_rows;
            const int tok = g.tok + u * sub + r / a.G;
            const long long orow = (long long)(g.tok0 + tok) * a.Hq + g.hg * a.G + r % a.G;
            if (g.t0 == g.t1) {                            // nothing to attend to
                if (live) {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + orow * D);
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
                    a.lse[orow] = -INFINITY;
                }
                continue;
            }
            const int first_lim = g.base + g.tok + u * sub + 1;        // keys that the subtile's first token sees
            const int lim = live ? g.base + tok + 1 : 0;
            const bool warp_live = (warp & 3) * 32 < live_rows;
            float m = -INFINITY, l = 0.f;
            for (int t = g.t0; t < g.t1; ++t, ++tiles) {
                if (!(ok = mbar_wait_warp(smem_u32(&bar_s_full[u]), tiles & 1, w, SITE_PAGED_S_FULL))) break;
                // SEP: P(t - 1) is read and O_u at rest once PV(t - 1) is complete.  (Every warp waits
                // for it, so that none arrives for a tile while others still owe the one before.)
                auto pv_before = [&]() {
                    return !C::SEP || tiles == 0 ||
                           mbar_wait_warp(smem_u32(&bar_o_full[u]), (tiles - 1) & 1, w, SITE_PAGED_O_FULL);
                };
                if (!warp_live) {                          // rows of nobody: their P may be anything
                    if (C::SEP) mbar_arrive(smem_u32(&bar_s_free[u]));
                    ok = pv_before();
                    if (!ok) break;
                    mbar_arrive(smem_u32(&bar_p_ready[u]));
                    continue;
                }
                tc_fence_after();
                uint32_t s[128];
                tmem_ld_cols<4>(sc, s);
                const int kv0 = t * C::BN;
                if (kv0 + C::BN > first_lim) {
#pragma unroll
                    for (int e = 0; e < C::BN; ++e)
                        if (kv0 + e >= lim) s[e] = 0xff800000u;        // -inf
                }
                float m4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(s[k]);
#pragma unroll
                for (int e = 4; e + 8 <= C::BN; e += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) m4[k] = fmax3(m4[k], __uint_as_float(s[e + k]), __uint_as_float(s[e + 4 + k]));
#pragma unroll
                for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], __uint_as_float(s[C::BN - 4 + k]));
                const float m_tile = __fmul_rn(fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]), sl2);
                // A row whose maximum grew by more than 2^8 rescales its sum and output; the
                // others keep the old reference (weights up to 2^8 lose nothing).  PV(t - 1) is
                // complete: waited for (SEP), or S(t) was issued behind it.
                if (C::SEP) {
                    tc_fence_before();
                    mbar_arrive(smem_u32(&bar_s_free[u]));
                }
                ok = pv_before();
                if (!ok) break;
                if (C::SEP) tc_fence_after();
                const bool need = t > g.t0 && m_tile > m + 8.f;
                if (t == g.t0) m = m_tile;
                if (__any_sync(0xffffffffu, need)) {
                    const float alpha = need ? ex2(m - m_tile) : 1.f;
                    if (need) {
                        l *= alpha;
                        m = m_tile;
                    }
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(oc + c, o);
                        tmem_wait_ld16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st16(oc + c, o);
                    }
                }
                const float neg = m == -INFINITY ? 0.f : -m;
                float2 s2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < C::BN; c += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[c + e]), __uint_as_float(s[c + e + 1])),
                                                    make_float2(sl2, sl2), make_float2(neg, neg));
                        const float2 p = make_float2(ex2(x.x), ex2(x.y));
                        s2[(e >> 1) & 3] = __fadd2_rn(s2[(e >> 1) & 3], p);
                        pk[e >> 1] = pack2(p.x, p.y);
                    }
                    tmem_st16(pc + (c >> 1), pk);
                }
                l += ((s2[0].x + s2[0].y) + (s2[1].x + s2[1].y)) + ((s2[2].x + s2[2].y) + (s2[3].x + s2[3].y));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&bar_p_ready[u]));
            }
            if (!ok) break;
            if (!(ok = mbar_wait_warp(smem_u32(&bar_o_full[u]), (C::SEP ? tiles - 1 : parts) & 1, w, SITE_PAGED_O_FULL))) break;
            ++parts;
            if (!warp_live) continue;
            tc_fence_after();
            const bool whole = g.whole();
            const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            // A thread holds a row's columns; four neighbours exchange 16-byte units, so that a store
            // writes 64 bytes of each of eight rows instead of 16 of each of 32 (at D 128 the
            // scattered stores took 4 us a part).
            const int prow = (blockIdx.x * 2 + g.slot()) * a.p.rows + u * 128 + r;
            const int q0 = r & ~3, ql = lane & 3;
            int row4[4];                                   // rows q0 .. q0 + 3 of the output (or the part)
#pragma unroll
            for (int k = 0; k < 4; ++k) row4[k] = whole ? __shfl_sync(0xffffffffu, (int)orow, (lane & ~3) + k) : prow - ql + k;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld_cols<1>(oc + c, o);
                if (whole) {
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t pk[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            pk[i] = pack2(__uint_as_float(o[8 * k + 2 * i]) * inv, __uint_as_float(o[8 * k + 2 * i + 1]) * inv);
                        v[k] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    }
                    transpose4(v, ql);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (q0 + k < live_rows)
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + (long long)row4[k] * D + c + 8 * ql) = v[k];
                } else {
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = make_uint4(o[h + 4 * k], o[h + 4 * k + 1], o[h + 4 * k + 2], o[h + 4 * k + 3]);
                        transpose4(v, ql);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (q0 + k < live_rows)
                                *reinterpret_cast<uint4*>(a.part_o + (size_t)row4[k] * D + c + h + 4 * ql) = v[k];
                    }
                }
            }
            __syncwarp();
            tc_fence_before();
            if (live) {
                if (whole) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                else a.part_ml[prow] = make_float2(m, l);
            }
            if (!whole && u == 0 && r == 0) a.part_info[blockIdx.x * 2 + g.slot()] = paged_record(g);
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

template <int D>
cudaError_t launch_tiles_t(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a,
                           cudaStream_t st) {
    using C = TileCfg<D>;
    auto kfn = paged_tiles_kernel<D>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kfn, C::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_k(kfn, dim3(a.p.C), dim3(C::THREADS), C::SMEM, st, tq, tk, tv, a);
}

}  // namespace

cudaError_t launch_paged_tiles(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, cudaStream_t st) {
    if (D == 64) return launch_tiles_t<64>(tq, tk, tv, a, st);
    if (D == 128) return launch_tiles_t<128>(tq, tk, tv, a, st);
    return cudaErrorInvalidValue;
}

}  // namespace ne
