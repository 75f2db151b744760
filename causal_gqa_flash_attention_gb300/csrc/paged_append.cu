// paged_append.cu -- new tokens into the paged cache: rotate the key (and query) rows at
// their positions, store keys and values into their pages.
//
// y = R(p) x on the first rot elements of a row: pair i turns by the angle p f_i, given as
// the fraction of a turn (p * turns_i mod 2^64) / 2^64, which is exact for every position
// (a product of fp32, or a table, would lose the angle of far positions); sincospi takes
// it from there.  A token's angles are formed once by each of its warps and serve all the
// warp's heads.  Bound: every row is read once and written once, 2 (Hq + 2 Hkv) D elements
// per token at the copy bandwidth; a step of a few tokens is latency (find the token's
// sequence, its page, then one load and one store).
// Measured (GB300), inputs and pages from DRAM: 6250 tokens, 16 + 2 x 4 heads of 128, half of each
// head rotated in halves: 18.6 us, 4.1 TB/s (61% of the copy rate: 1.3 waves of one warp per token,
// each of which loads its next heads only when it has stored the last; 14 us where the L2 holds
// everything); 2048 tokens 8.1 us (3.7 at the copy rate); 32768 tokens 65 us (91%).  fp32, heads of
// 64: 17.0 and 62 us (6250 and 32768 tokens, 67% and 96%).  16 tokens of 12 + 2 x 4 heads of 64: 3.2 us.
#include <cuda_bf16.h>
#include "paged_sched.cuh"

namespace ne {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSms = 152;

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

// What a lane needs to rotate its two units (elements ea .. ea+N-1 and eb .. eb+N-1) of every
// head of a token: the (cos, sin) of their pairs, fetched once.  Interleaved, pairs (2i, 2i+1)
// lie in a unit; half-split, pairs (i, i + rot/2), unit b holds the partners of unit a.  Where
// half of rot is no whole number of units the half-split partners are read from the row.
template <typename T, bool HALF>
struct Turn {
    static constexpr int N = Vec<T>::N;
    float2 cs[N];
    __device__ __forceinline__ void load(const float2* s, int ea, int eb, int rot) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = HALF ? ea + i : i < N / 2 ? ea + 2 * i : eb + 2 * i - N;
            cs[i] = e < rot ? s[HALF ? e : e >> 1] : make_float2(1.f, 0.f);
        }
    }
    __device__ __forceinline__ void apply(uint4& ua, uint4& ub, int ea, int eb, int rot) const {
        float x[N], z[N];
        Vec<T>::get(ua, x);
        Vec<T>::get(ub, z);
        if constexpr (HALF) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float u = x[i] * cs[i].x - z[i] * cs[i].y;
                z[i] = z[i] * cs[i].x + x[i] * cs[i].y;
                x[i] = u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) {               // (what lies behind rot passes, infinities too)
                const float2 c = cs[i >> 1], d = cs[(i + N) >> 1];
                const float u = x[i] * c.x - x[i + 1] * c.y, w = z[i] * d.x - z[i + 1] * d.y;
                if (ea + i < rot) {
                    x[i + 1] = x[i] * c.y + x[i + 1] * c.x;
                    x[i] = u;
                }
                if (eb + i < rot) {
                    z[i + 1] = z[i] * d.y + z[i + 1] * d.x;
                    z[i] = w;
                }
            }
        }
        ua = Vec<T>::put(x);
        ub = Vec<T>::put(z);
    }
    __device__ static uint4 odd(const uint4& u, const T* head, const float2* s, int e0, int rot) {
        const int half = rot >> 1;
        float x[N];
        Vec<T>::get(u, x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = e0 + i;
            if (e >= rot) break;
            const float2 c = s[e < half ? e : e - half];
            const float o = Vec<T>::one(head + (e < half ? e + half : e - half));
            x[i] = x[i] * c.x + (e < half ? -o : o) * c.y;
        }
        return Vec<T>::put(x);
    }
};

// Heads in flight per lane, two units each (one: 2 to 9% slower on long chunks; three need a
// CTA less per SM and lose a quarter on short ones).  Their loads need no position, so the first ones go out before
// the warp has looked its token up.
constexpr int kBatch = 2;

// A warp serves one token, or 1 / wpt of its heads.  A lane keeps two 16-byte units of a head
// and walks over the heads: 64 / vecs of them to a pass.  (Units dealt out flat cost 250
// instructions each for indices and angles, and bound the kernel by its instructions; with one
// unit per lane the half-split partners came by shuffles, 17.8 us for the chunk below.)  A warp
// holds whole heads and reads a batch of them before it writes any, so q_out may be q itself.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns turns) {
    constexpr int N = Vec<T>::N;
    __shared__ __align__(16) float2 s_cs[kWarps][64];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    griddep_wait();
    // Sequences without rows are looked at too, or a bad entry of theirs would go unnoticed.
    if (blockIdx.x == gridDim.x - 1) {
        int bad = 0;
        for (int b = tid; b < a.s.B; b += kThreads) paged_seq(a.s, b, bad);
        if (bad) report_error(a.err, bad);
    }
    const long long item = (long long)blockIdx.x * kWarps + warp;
    const int part = (int)item & ((1 << a.wpt_shift) - 1);
    const long long row = item >> a.wpt_shift;
    if (row >= a.s.N) return;
    const int lph = 1 << (a.vec_shift - 1);                // lanes per head
    const int j = lane & (lph - 1);
    // Whole units per half: the partners' distance, and the lanes that turn.
    const bool whole = HALF && (a.rot >> 1) % N == 0;
    const int turning = whole ? (a.rot >> 1) / N : 0;
    const int ea = N * (j < turning ? j : j + turning);
    const int eb = ea + N * (j < turning ? turning : lph - turning);
    const int qh = a.q ? a.Hq : 0, heads = qh + 2 * a.Hkv;
    const int hpw = 32 / lph, step = hpw << a.wpt_shift;
    const T* qrow = static_cast<const T*>(a.q) + row * a.q_ld;
    const T* krow = static_cast<const T*>(a.k_in) + row * a.k_ld;
    const T* vrow = static_cast<const T*>(a.v_in) + row * a.v_ld;
    auto source = [&](int h) { return h < qh ? qrow + h * a.D : h < qh + a.Hkv ? krow + (h - qh) * a.D : vrow + (h - qh - a.Hkv) * a.D; };
    uint4 ua[kBatch], ub[kBatch];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k, h += step) {
            ua[k] = ub[k] = make_uint4(0u, 0u, 0u, 0u);
            if (h < heads) {
                const T* s = source(h);
                ua[k] = *reinterpret_cast<const uint4*>(s + ea);
                ub[k] = *reinterpret_cast<const uint4*>(s + eb);
            }
        }
    };
    const int first = part * hpw;                          // the warp's first head
    fetch(first + lane / lph);

    const int r = (int)row;
    const int b = a.s.cu ? find_seq(a.s.cu, a.s.B, r, lane) : r;
    int pos = -2;                                          // -1: not stored, -2: not a row of the call
    int shift = a.pos_offset;                              // the rotation's position behind the slot's
    long long slot = -1;                                   // the slot's offset in the pools (elements), -1: none
    if (b >= 0) {
        int bad = 0;
        const PagedSeq q = paged_seq(a.s, b, bad);
        if (a.pos_offsets) {
            const int o = __ldg(a.pos_offsets + b);
            if ((unsigned)o >= 1u << 30) bad = SITE_PAGED_LEN;
            shift = min(max(o, 0), (1 << 30) - 1);
        }
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
    Turn<T, HALF> turn;
    if (pos >= 0 && a.rot) {
        for (int p = lane; p < a.rot >> 1; p += 32) {
            // Fraction of a turn in [-1/2, 1/2), as a signed 64-bit number over 2^64.
            const long long f = (long long)((unsigned long long)(pos + shift) * turns.t[p]);
            float s, c;
            sincospif((float)f * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
            s_cs[warp][p] = make_float2(c * a.mscale, s * a.mscale);
        }
        __syncwarp();
        if (!HALF || j < turning) turn.load(s_cs[warp], ea, eb, a.rot);
    }
    const bool turned = pos >= 0 && (whole ? j < turning : ea < a.rot);
    T* qdst = pos != -2 && a.q ? static_cast<T*>(a.q_out) + row * a.qo_ld : nullptr;
    T* kdst = slot >= 0 ? static_cast<T*>(const_cast<void*>(a.c.k)) + slot : nullptr;
    T* vdst = slot >= 0 ? static_cast<T*>(const_cast<void*>(a.c.v)) + slot : nullptr;
    // (The loop runs on the warp's first head, so that every lane takes the same passes.)
    for (int hw = first; hw < heads; hw += kBatch * step) {
        const int h = hw + lane / lph;
        if (turned) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int hk = h + k * step;
                if (hk >= qh + a.Hkv) continue;
                if (!HALF || whole) {
                    turn.apply(ua[k], ub[k], ea, eb, a.rot);
                } else {
                    ua[k] = turn.odd(ua[k], source(hk), s_cs[warp], ea, a.rot);
                    ub[k] = turn.odd(ub[k], source(hk), s_cs[warp], eb, a.rot);
                }
            }
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
            if (dst) {
                *reinterpret_cast<uint4*>(dst + ea) = pos < 0 ? make_uint4(0u, 0u, 0u, 0u) : ua[k];
                *reinterpret_cast<uint4*>(dst + eb) = pos < 0 ? make_uint4(0u, 0u, 0u, 0u) : ub[k];
            }
        }
        fetch(h + kBatch * step);
    }
}

}  // namespace

cudaError_t launch_paged_append(bool f32, const AppendArgs& a0, const RopeTurns& t, cudaStream_t st) {
    AppendArgs a = a0;
    // Several warps per token while all of them are resident at once (four CTAs per SM); 2048
    // tokens: 6.3 us with two warps each.  From there on a second look-up costs more than it hides.
    const int slots = 4 * kSms * kWarps;
    a.wpt_shift = a.s.N <= slots / 8 ? 3 : a.s.N <= slots / 4 ? 2 : a.s.N <= slots / 2 ? 1 : 0;
    const int vecs = a.D / (f32 ? 4 : 8);
    while ((1 << a.vec_shift) < vecs) ++a.vec_shift;
    const dim3 grid((unsigned)((((long long)a.s.N << a.wpt_shift) + kWarps - 1) / kWarps)), block(kThreads);
    if (a.layout == 1)
        return f32 ? launch_k(paged_append_kernel<float, true>, grid, block, 0, st, a, t)
                   : launch_k(paged_append_kernel<__nv_bfloat16, true>, grid, block, 0, st, a, t);
    return f32 ? launch_k(paged_append_kernel<float, false>, grid, block, 0, st, a, t)
               : launch_k(paged_append_kernel<__nv_bfloat16, false>, grid, block, 0, st, a, t);
}

}  // namespace ne
