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

// One 16-byte unit at element e0 of a row, rotated.
template <typename T>
__device__ __forceinline__ uint4 rotated(const T* row, int e0, const float2* cs, int rot, int layout) {
    constexpr int N = Vec<T>::N;
    uint4 u = *reinterpret_cast<const uint4*>(row + e0);
    if (e0 >= rot) return u;
    float x[N], y[N];
    Vec<T>::get(u, x);
    if (layout == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const bool in = e0 + i < rot;
            const float2 c = in ? cs[(e0 + i) >> 1] : make_float2(1.f, 0.f);
            y[i] = x[i] * c.x - x[i + 1] * c.y;
            y[i + 1] = x[i] * c.y + x[i + 1] * c.x;
            if (!in) {
                y[i] = x[i];
                y[i + 1] = x[i + 1];
            }
        }
    } else {
        const int half = rot >> 1;
        float z[N];                                        // the other element of every pair
        if (half % N == 0) {
            const int p0 = e0 < half ? e0 + half : e0 - half;
            Vec<T>::get(*reinterpret_cast<const uint4*>(row + p0), z);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = e0 + i;
                z[i] = e < rot ? Vec<T>::one(row + (e < half ? e + half : e - half)) : 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = e0 + i;
            if (e >= rot) {
                y[i] = x[i];
            } else {
                const float2 c = cs[e < half ? e : e - half];
                y[i] = e < half ? x[i] * c.x - z[i] * c.y : z[i] * c.y + x[i] * c.x;
            }
        }
    }
    return Vec<T>::put(y);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
    constexpr int N = Vec<T>::N;
    __shared__ float2 s_cs[kTok][64];
    __shared__ int s_pos[kTok];                            // position, -1: not stored, -2: not a row of the call
    __shared__ long long s_slot[kTok];                     // the slot's offset in the pools (elements), -1: none
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * a.tpc, nt = min(a.tpc, a.s.N - t0);
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
    }
    // Sequences without rows are looked at too, or a bad entry of theirs would go unnoticed.
    if (blockIdx.x == 0) {
        int bad = 0;
        for (int b = tid; b < a.s.B; b += kThreads) paged_seq(a.s, b, bad);
        if (bad) report_error(a.err, bad);
    }
    __syncthreads();
    const int pairs = a.rot >> 1;
    for (int i = tid; i < nt * pairs; i += kThreads) {
        const int t = i / pairs, p = i - t * pairs;
        if (s_pos[t] < 0) continue;
        // Fraction of a turn in [-1/2, 1/2), as a signed 64-bit number over 2^64.
        const long long f = (long long)((unsigned long long)(s_pos[t] + a.pos_offset) * turns.t[p]);
        float s, c;
        sincospif((float)f * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
        s_cs[t][p] = make_float2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();
    // A head's units are neighbours within one warp (at most 32 of them): the warp reads its
    // rows before it writes any, so q_out may be q itself.
    const int vecs = a.D / N;
    const int qh = a.q ? a.Hq : 0;
    const int per = (qh + 2 * a.Hkv) * vecs;
    for (int base = warp * 32; base < nt * per; base += kThreads) {
        const int i = base + lane;
        uint4 val = make_uint4(0u, 0u, 0u, 0u);
        T* dst = nullptr;
        if (i < nt * per) {
            const int t = i / per, r = i - t * per;
            const int h = r / vecs, e0 = (r - h * vecs) * N;
            const int pos = s_pos[t];
            const long long row = t0 + t, slot = s_slot[t];
            if (h < qh) {
                if (pos != -2) {
                    dst = static_cast<T*>(a.q_out) + row * a.qo_ld + (long long)h * a.D + e0;
                    if (pos >= 0)
                        val = rotated<T>(static_cast<const T*>(a.q) + row * a.q_ld + (long long)h * a.D, e0, s_cs[t], a.rot,
                                         a.layout);
                }
            } else if (slot >= 0) {
                const bool key = h - qh < a.Hkv;
                const int hh = key ? h - qh : h - qh - a.Hkv;
                dst = static_cast<T*>(const_cast<void*>(key ? a.c.k : a.c.v)) + slot + (long long)hh * a.c.head_stride + e0;
                if (key)
                    val = rotated<T>(static_cast<const T*>(a.k_in) + row * a.k_ld + (long long)hh * a.D, e0, s_cs[t], a.rot,
                                     a.layout);
                else
                    val = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v_in) + row * a.v_ld +
                                                          (long long)hh * a.D + e0);
            }
        }
        __syncwarp();
        if (dst) *reinterpret_cast<uint4*>(dst) = val;
    }
}

}  // namespace

cudaError_t launch_paged_append(bool f32, const AppendArgs& a0, const RopeTurns& t, cudaStream_t st) {
    AppendArgs a = a0;
    // A CTA per token while there are no more than four per SM, then up to eight tokens each.
    a.tpc = a.s.N <= 4 * 152 ? 1 : (a.s.N <= 16 * 152 ? 4 : kTok);
    const dim3 grid((a.s.N + a.tpc - 1) / a.tpc);
    return f32 ? launch_k(paged_append_kernel<float>, grid, dim3(kThreads), 0, st, a, t)
               : launch_k(paged_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, a, t);
}

}  // namespace ne
