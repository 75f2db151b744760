// paged_append.cu -- new tokens into the paged cache: rotate the key (and query) rows at
// their positions, store keys and values into their pages.
//
// y = R(p) x on the first rot elements of a row: pair i turns by the angle p f_i, given as
// the fraction of a turn (p * turns_i mod 2^64) / 2^64, which is exact for every position
// (a product of fp32, or a table, would lose the angle of far positions); sincospi takes
// it from there.  A token's angles are formed once per CTA in shared memory and serve all
// its heads.  Bound: every row is read once and written once, 2 (Hq + 2 Hkv) D elements
// per token at the copy bandwidth; a step of a few tokens is latency (find the token's
// sequence, its page, then one load and one store).
#include <cuda_bf16.h>
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kThreads = 256;
constexpr int kTok = 8;                                    // most tokens per CTA

template <typename T>
struct Vec;                                                // 16 bytes of a row
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void get(const uint4& u, float (&f)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 put(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static void get(const uint4& u, float (&f)[4]) {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 put(const float (&f)[4]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ static float one(const float* p) { return *p; }
};

// Sequence that row t belongs to (the last b with cu[b] <= t), found by a warp, 32
// candidates at a time; -1 outside [cu[0], cu[B]).
__device__ __forceinline__ int find_seq(const int* cu, int B, int t, int lane) {
    int lo = 0, hi = B + 1;                                // the answer's index in cu[0 .. B], half open
    if (t < __ldg(cu)) return -1;
    while (hi - lo > 1) {                                  // cu[lo] <= t, and cu[hi] > t or hi == B + 1
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < hi && __ldg(cu + i) <= t);
        const int last = 31 - __clz(m | 1u);               // (lane 0's entry is at or before t)
        const int nlo = lo + last * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo < B ? lo : -1;
}

// 16-byte unit `u` at element e0 of a row, rotated; `pair` holds the other elements of its
// pairs (half layout with whole units per half; elsewhere they come from the row itself).
template <typename T>
__device__ __forceinline__ uint4 rotated(const uint4& u, const uint4& pair, const T* row, int e0, const float2* cs, int rot,
                                         int layout) {
    constexpr int N = Vec<T>::N;
    if (e0 >= rot) return u;
    float x[N], y[N];
    Vec<T>::get(u, x);
    if (layout == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if (e0 + i < rot) {
                const float2 c = cs[(e0 + i) >> 1];
                y[i] = x[i] * c.x - x[i + 1] * c.y;
                y[i + 1] = x[i] * c.y + x[i + 1] * c.x;
            } else {
                y[i] = x[i];
                y[i + 1] = x[i + 1];
            }
        }
        return Vec<T>::put(y);
    }
    const int half = rot >> 1;
    float z[N];
    if (half % N == 0) {
        Vec<T>::get(pair, z);
        const bool first = e0 < half;
        const float4* c4 = reinterpret_cast<const float4*>(cs + (first ? e0 : e0 - half));
        const float sign = first ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float4 c = c4[i >> 1];                   // (cos, sin) of two pairs
            y[i] = x[i] * c.x + sign * (z[i] * c.y);
            y[i + 1] = x[i + 1] * c.z + sign * (z[i + 1] * c.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = e0 + i;
            if (e >= rot) {
                y[i] = x[i];
            } else {
                const bool first = e < half;
                const float o = Vec<T>::one(row + (first ? e + half : e - half));
                const float2 c = cs[first ? e : e - half];
                y[i] = first ? x[i] * c.x - o * c.y : x[i] * c.x + o * c.y;
            }
        }
    }
    return Vec<T>::put(y);
}

// Units in flight per thread.  Their loads need no position, so the first ones go out before
// the CTA has looked its tokens up.
constexpr int kUnits = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
    constexpr int N = Vec<T>::N;
    __shared__ __align__(16) float2 s_cs[kTok][64];
    __shared__ int s_pos[kTok];                            // position, -1: not stored, -2: not a row of the call
    __shared__ long long s_slot[kTok];                     // the slot's offset in the pools (elements), -1: none
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * a.tpc, nt = min(a.tpc, a.s.N - t0);

    // Unit i of the CTA: token i / per, head, 16-byte unit of the head.  A head's units are
    // neighbours within one warp (at most 32 of them), and a warp reads a batch of units
    // before it writes any of them, so q_out may be q itself.
    const int vshift = a.vec_shift, qh = a.q ? a.Hq : 0;
    const int per = (qh + 2 * a.Hkv) << vshift, total = nt * per;
    struct Unit {
        int t, h, e0;
        const T* row;
    };
    auto unit = [&](int i) {
        Unit x;
        x.t = (int)fast_div((uint32_t)i, a.div_per);
        const int r = i - x.t * per;
        x.h = r >> vshift;
        x.e0 = (r & ((1 << vshift) - 1)) * N;
        const long long row = t0 + x.t;
        x.row = x.h < qh ? static_cast<const T*>(a.q) + row * a.q_ld + (long long)x.h * a.D
                : x.h < qh + a.Hkv ? static_cast<const T*>(a.k_in) + row * a.k_ld + (long long)(x.h - qh) * a.D
                                   : static_cast<const T*>(a.v_in) + row * a.v_ld + (long long)(x.h - qh - a.Hkv) * a.D;
        return x;
    };
    uint4 raw[kUnits];
    auto fetch = [&](int base) {
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int i = base + k * kThreads + lane;
            raw[k] = make_uint4(0u, 0u, 0u, 0u);
            if (i < total) {
                const Unit x = unit(i);
                raw[k] = *reinterpret_cast<const uint4*>(x.row + x.e0);
            }
        }
    };
    fetch(warp * 32);

    if (warp < nt) {
        const int t = t0 + warp;
        const int b = a.s.cu ? find_seq(a.s.cu, a.s.B, t, lane) : t;
        int pos = -2;
        long long slot = -1;
        if (b >= 0) {
            int bad = 0;
            const PagedSeq q = paged_seq(a.s, b, bad);
            if (t >= q.tok0 && t < q.tok0 + q.n) {
                pos = q.len - q.n + (t - q.tok0);
                if (pos < 0) {
                    pos = -1;
                } else {
                    const int page = __ldg(a.s.table + (size_t)b * a.s.W + (pos >> a.c.ps_shift));
                    if ((unsigned)page < (unsigned)a.c.n_pages)
                        slot = (long long)page * a.c.page_stride +
                               (long long)(pos & ((1 << a.c.ps_shift) - 1)) * a.c.tok_stride;
                    else if (lane == 0)
                        report_error(a.err, SITE_PAGED_PAGE);
                }
            }
            if (bad && lane == 0) report_error(a.err, bad);
        }
        if (lane == 0) {
            s_pos[warp] = pos;
            s_slot[warp] = slot;
        }
        if (pos >= 0)
            for (int p = lane; p < a.rot >> 1; p += 32) {
                // Fraction of a turn in [-1/2, 1/2), as a signed 64-bit number over 2^64.
                const long long f = (long long)((unsigned long long)(pos + a.pos_offset) * turns.t[p]);
                float s, c;
                sincospif((float)f * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
                s_cs[warp][p] = make_float2(c * a.mscale, s * a.mscale);
            }
    }
    // Sequences without rows are looked at too, or a bad entry of theirs would go unnoticed.
    if (blockIdx.x == gridDim.x - 1) {
        int bad = 0;
        for (int b = tid; b < a.s.B; b += kThreads) paged_seq(a.s, b, bad);
        if (bad) report_error(a.err, bad);
    }
    __syncthreads();

    const int pair_lanes = (a.rot >> 1) / N;               // half layout: lanes between the units of a pair
    for (int base = warp * 32; base < total; base += kUnits * kThreads) {
        uint4 val[kUnits];
        T* dst[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int i = base + k * kThreads + lane;
            const Unit x = unit(min(i, total - 1));
            uint4 pair = raw[k];
            if (a.layout == 1) {
                const int from = (lane + (x.e0 < a.rot >> 1 ? pair_lanes : -pair_lanes)) & 31;
                pair.x = __shfl_sync(0xffffffffu, raw[k].x, from);
                pair.y = __shfl_sync(0xffffffffu, raw[k].y, from);
                pair.z = __shfl_sync(0xffffffffu, raw[k].z, from);
                pair.w = __shfl_sync(0xffffffffu, raw[k].w, from);
            }
            dst[k] = nullptr;
            val[k] = raw[k];
            const int pos = s_pos[x.t];
            const long long slot = s_slot[x.t];
            if (i < total) {
                if (x.h < qh) {
                    if (pos != -2) dst[k] = static_cast<T*>(a.q_out) + (long long)(t0 + x.t) * a.qo_ld + (long long)x.h * a.D + x.e0;
                } else if (slot >= 0) {
                    const bool key = x.h - qh < a.Hkv;
                    dst[k] = static_cast<T*>(const_cast<void*>(key ? a.c.k : a.c.v)) + slot +
                             (long long)(key ? x.h - qh : x.h - qh - a.Hkv) * a.c.head_stride + x.e0;
                }
                if (pos < 0) val[k] = make_uint4(0u, 0u, 0u, 0u);
                else if (x.h < qh + a.Hkv) val[k] = rotated<T>(raw[k], pair, x.row, x.e0, s_cs[x.t], a.rot, a.layout);
            }
        }
        __syncwarp();                                      // every read of this batch is done
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
            if (dst[k]) *reinterpret_cast<uint4*>(dst[k]) = val[k];
        fetch(base + kUnits * kThreads);
    }
}

}  // namespace

cudaError_t launch_paged_append(bool f32, const AppendArgs& a0, const RopeTurns& t, cudaStream_t st) {
    AppendArgs a = a0;
    // A CTA per token while there are no more than four per SM, then up to eight tokens each.
    a.tpc = a.s.N <= 4 * 152 ? 1 : (a.s.N <= 16 * 152 ? 4 : kTok);
    const int vecs = a.D / (f32 ? 4 : 8);
    while ((1 << a.vec_shift) < vecs) ++a.vec_shift;
    a.div_per = make_fastdiv((uint32_t)(((a.q ? a.Hq : 0) + 2 * a.Hkv) * vecs));
    const dim3 grid((a.s.N + a.tpc - 1) / a.tpc);
    return f32 ? launch_k(paged_append_kernel<float>, grid, dim3(kThreads), 0, st, a, t)
               : launch_k(paged_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a, t);
}

}  // namespace ne
