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
// Measured (GB300): 6250 tokens, 16 + 2 x 4 heads of 128, half of each head rotated: 17.8 us,
// 4.3 TB/s (64% of the copy rate; 40% of the issue slots, the rest the latency of the lookups);
// 16 tokens of 12 + 2 x 4 heads of 64: 3.6 us.
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

// What a lane needs to rotate its unit (elements e0 .. e0 + N-1) of every head of a token:
// the (cos, sin) of its pairs, fetched once.  HALF: pairs (i, i + rot/2), one per element;
// else pairs (2i, 2i+1), one per two elements.
template <typename T, bool HALF>
struct Turn {
    static constexpr int N = Vec<T>::N;
    static constexpr int P = HALF ? N : N / 2;
    float2 cs[P];
    __device__ __forceinline__ void load(const float2* s, int e0, int rot) {
        const int half = rot >> 1;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int e = HALF ? e0 + i : e0 + 2 * i;
            const int p = HALF ? (e < half ? e : e - half) : e >> 1;
            cs[i] = e < rot ? s[p] : make_float2(1.f, 0.f);
        }
    }
    // `pair`: the unit that holds the other elements of the pairs (whole units per half);
    // otherwise they are read from the row.
    __device__ __forceinline__ uint4 apply(const uint4& u, const uint4& pair, const T* row, int e0, int rot) const {
        float x[N], y[N];
        Vec<T>::get(u, x);
        if constexpr (!HALF) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float2 c = cs[i >> 1];
                const bool in = e0 + i < rot;              // (the rest passes, infinities too)
                y[i] = in ? x[i] * c.x - x[i + 1] * c.y : x[i];
                y[i + 1] = in ? x[i] * c.y + x[i + 1] * c.x : x[i + 1];
            }
        } else {
            const int half = rot >> 1;
            if (half % N == 0) {
                float z[N];
                Vec<T>::get(pair, z);
                const float sign = e0 < half ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < N; ++i) y[i] = x[i] * cs[i].x + (sign * z[i]) * cs[i].y;
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int e = e0 + i;
                    if (e >= rot) {
                        y[i] = x[i];
                    } else {
                        const float o = Vec<T>::one(row + (e < half ? e + half : e - half));
                        y[i] = x[i] * cs[i].x + (e < half ? -o : o) * cs[i].y;
                    }
                }
            }
        }
        return Vec<T>::put(y);
    }
};

// Heads in flight per lane.  Their loads need no position, so the first ones go out before
// the CTA has looked its tokens up.
constexpr int kBatch = 4;

// A lane keeps one 16-byte unit of a head and walks over the heads of one token: 32 / vecs heads
// to a warp, kThreads / 32 / tpc warps to a token.  (Units dealt out flat cost 250 instructions
// each for indices and angles, and bound the kernel by its instructions.)  A warp holds whole
// heads and reads a batch of them before it writes any, so q_out may be q itself.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
    constexpr int N = Vec<T>::N;
    __shared__ __align__(16) float2 s_cs[kTok][64];
    __shared__ int s_pos[kTok];                            // position, -1: not stored, -2: not a row of the call
    __shared__ long long s_slot[kTok];                     // the slot's offset in the pools (elements), -1: none
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * a.tpc, nt = min(a.tpc, a.s.N - t0);
    const int wpt = (kThreads / 32) / a.tpc;               // warps of a token
    const int t = warp / wpt;
    const long long row = t0 + t;
    const int e0 = (lane & ((1 << a.vec_shift) - 1)) * N;  // this lane's unit
    const int hpw = 32 >> a.vec_shift;                     // heads of a warp's pass
    const int qh = a.q ? a.Hq : 0, heads = t < nt ? qh + 2 * a.Hkv : 0;
    const int step = wpt * hpw;
    const int h0 = (warp - t * wpt) * hpw + (lane >> a.vec_shift);
    const T* qrow = static_cast<const T*>(a.q) + row * a.q_ld + e0;
    const T* krow = static_cast<const T*>(a.k_in) + row * a.k_ld + e0;
    const T* vrow = static_cast<const T*>(a.v_in) + row * a.v_ld + e0;
    auto source = [&](int h) { return h < qh ? qrow + h * a.D : h < qh + a.Hkv ? krow + (h - qh) * a.D : vrow + (h - qh - a.Hkv) * a.D; };
    uint4 raw[kBatch];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k, h += step)
            raw[k] = h < heads ? *reinterpret_cast<const uint4*>(source(h)) : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch(h0);

    if (t < nt && warp == t * wpt) {
        const int r = t0 + t;
        const int b = a.s.cu ? find_seq(a.s.cu, a.s.B, r, lane) : r;
        int pos = -2;
        long long slot = -1;
        if (b >= 0) {
            int bad = 0;
            const PagedSeq q = paged_seq(a.s, b, bad);
            if (r >= q.tok0 && r < q.tok0 + q.n) {
                pos = q.len - q.n + (r - q.tok0);
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
            s_pos[t] = pos;
            s_slot[t] = slot;
        }
        if (pos >= 0)
            for (int p = lane; p < a.rot >> 1; p += 32) {
                // Fraction of a turn in [-1/2, 1/2), as a signed 64-bit number over 2^64.
                const long long f = (long long)((unsigned long long)(pos + a.pos_offset) * turns.t[p]);
                float s, c;
                sincospif((float)f * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
                s_cs[t][p] = make_float2(c * a.mscale, s * a.mscale);
            }
    }
    // Sequences without rows are looked at too, or a bad entry of theirs would go unnoticed.
    if (blockIdx.x == gridDim.x - 1) {
        int bad = 0;
        for (int b = tid; b < a.s.B; b += kThreads) paged_seq(a.s, b, bad);
        if (bad) report_error(a.err, bad);
    }
    __syncthreads();
    if (t >= nt) return;

    const int pos = s_pos[t];
    const long long slot = s_slot[t];
    const bool turned = e0 < a.rot && pos >= 0;
    Turn<T, HALF> turn;
    if (turned) turn.load(s_cs[t], e0, a.rot);
    // HALF: the lane that holds the other elements of this one's pairs.
    const int other = HALF ? lane + (e0 < a.rot >> 1 ? (a.rot >> 1) / N : -((a.rot >> 1) / N)) : 0;
    T* qdst = pos != -2 && a.q ? static_cast<T*>(a.q_out) + row * a.qo_ld + e0 : nullptr;
    T* kdst = slot >= 0 ? static_cast<T*>(const_cast<void*>(a.c.k)) + slot + e0 : nullptr;
    T* vdst = slot >= 0 ? static_cast<T*>(const_cast<void*>(a.c.v)) + slot + e0 : nullptr;
    // (The loop runs on the warp's first head, so that every lane takes the same passes.)
    for (int hw = h0 - (lane >> a.vec_shift); hw < heads; hw += kBatch * step) {
        const int h = hw + (lane >> a.vec_shift);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            uint4 pair = raw[k];
            if (HALF) {
                pair.x = __shfl_sync(0xffffffffu, raw[k].x, other & 31);
                pair.y = __shfl_sync(0xffffffffu, raw[k].y, other & 31);
                pair.z = __shfl_sync(0xffffffffu, raw[k].z, other & 31);
                pair.w = __shfl_sync(0xffffffffu, raw[k].w, other & 31);
            }
            const int hk = h + k * step;
            if (hk < qh + a.Hkv && hk < heads && turned)
                raw[k] = turn.apply(raw[k], pair, source(hk) - e0, e0, a.rot);
        }
        __syncwarp();                                      // every read of this batch is done
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int hk = h + k * step;
            if (hk >= heads) continue;
            T* dst;
            if (hk < qh) dst = qdst ? qdst + hk * a.D : nullptr;
            else if (hk < qh + a.Hkv) dst = kdst ? kdst + (hk - qh) * a.c.head_stride : nullptr;
            else dst = vdst ? vdst + (hk - qh - a.Hkv) * a.c.head_stride : nullptr;
            if (dst) *reinterpret_cast<uint4*>(dst) = pos < 0 ? make_uint4(0u, 0u, 0u, 0u) : raw[k];
        }
        fetch(h + kBatch * step);
    }
}

}  // namespace

cudaError_t launch_paged_append(bool f32, const AppendArgs& a0, const RopeTurns& t, cudaStream_t st) {
    AppendArgs a = a0;
    // A CTA per token while there are no more than four per SM; then a warp or two per token:
    // the lookups of a CTA's tokens take as long as two batches of heads, whatever their number.
    a.tpc = a.s.N <= 4 * 152 ? 1 : a.s.N <= 16 * 152 ? 4 : kTok;
    const int vecs = a.D / (f32 ? 4 : 8);
    while ((1 << a.vec_shift) < vecs) ++a.vec_shift;
    const dim3 grid((a.s.N + a.tpc - 1) / a.tpc), block(kThreads);
    if (a.layout == 1)
        return f32 ? launch_k(paged_append_kernel<float, true>, grid, block, 0, st, a, t)
                   : launch_k(paged_append_kernel<__nv_bfloat16, true>, grid, block, 0, st, a, t);
    return f32 ? launch_k(paged_append_kernel<float, false>, grid, block, 0, st, a, t)
               : launch_k(paged_append_kernel<__nv_bfloat16, false>, grid, block, 0, st, a, t);
}

}  // namespace ne
