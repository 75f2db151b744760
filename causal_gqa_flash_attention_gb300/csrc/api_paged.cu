// api_paged.cu -- the paged-cache entry points of include/neattn.h: argument validation,
// kernel choice and launches.  Every step runs in the kernels.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "api.h"
#include "kernels.h"
#include "neattn.h"
#include "paged.h"

using namespace ne::api;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 39;
constexpr double kTwoPi = 6.283185307179586476925286766559;

bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Half-open byte ranges [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

// Rows of `w` bytes, n of them, ld bytes apart at p, against rows of wq bytes, ldq apart, at
// q.  Slices of one buffer (the parts of a fused projection) interleave without sharing.
bool rows_overlap(const void* p, int64_t w, int64_t ld, const void* q, int64_t wq, int64_t ldq, int64_t n) {
    if (!p || !q || !overlap(p, (size_t)(ld * (n - 1) + w), q, (size_t)(ldq * (n - 1) + wq))) return false;
    if (n == 1 || ld != ldq) return true;
    const int64_t d = ((reinterpret_cast<intptr_t>(q) - reinterpret_cast<intptr_t>(p)) % ld + ld) % ld;
    return d < w || d + wq > ld;
}

ne_status check_cache(const ne_paged_cache* c, int want_bytes, bool attn) {
    if (!c) return fail(NE_ERR_INVALID_ARG, "null cache");
    if (c->elem_bytes != 2 && c->elem_bytes != 4)
        return fail(NE_ERR_INVALID_ARG, "cache elem_bytes must be 2 (bf16) or 4 (f32), got %d", c->elem_bytes);
    if (want_bytes && c->elem_bytes != want_bytes)
        return fail(NE_ERR_INVALID_ARG, "the cache holds %d-byte elements, the call takes %d-byte ones", c->elem_bytes,
                    want_bytes);
    if (c->layers < 1 || c->layers > 4096 || c->n_pages < 1 || c->n_pages >= (1 << 24) || c->Hkv < 1 || c->Hkv > 1024)
        return fail(NE_ERR_INVALID_ARG,
                    "need 1 <= layers <= 4096, 1 <= n_pages < 2^24, 1 <= Hkv <= 1024 (layers=%d n_pages=%d Hkv=%d)", c->layers,
                    c->n_pages, c->Hkv);
    if (attn && c->layers != 1)
        return fail(NE_ERR_INVALID_ARG, "the call works on one layer: pass that layer's pools with layers = 1");
    if (c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return fail(NE_ERR_UNSUPPORTED, "page_size must be a power of two from 8 to 256 (page_size=%d)", c->page_size);
    if (!(c->D == 32 || c->D == 64 || (c->D == 128 && c->elem_bytes == 2)))
        return fail(NE_ERR_UNSUPPORTED, "head_dim D=%d is not supported for %s (supported: %s)", c->D,
                    c->elem_bytes == 4 ? "f32" : "bf16", c->elem_bytes == 4 ? "32, 64" : "32, 64, 128");
    ne_status s = check_ptrs({c->k, c->v});
    if (s != NE_OK) return s;
    const int64_t strides[4] = {c->layer_stride, c->page_stride, c->tok_stride, c->head_stride};
    const int extent[4] = {c->layers, c->n_pages, c->page_size, c->Hkv};
    for (int i = 0; i < 4; ++i) {
        if (extent[i] == 1) continue;
        if (strides[i] < c->D || strides[i] >= kMaxStride || strides[i] * c->elem_bytes % 16 != 0)
            return fail(NE_ERR_INVALID_ARG,
                        "cache strides must be at least D, below 2^39 elements and multiples of 16 bytes (stride %lld)",
                        (long long)strides[i]);
    }
    return NE_OK;
}

ne_status check_rows(const char* what, const void* p, int64_t ld, int64_t heads, const ne_paged_cache* c) {
    if (!p || !aligned16(p)) return fail(NE_ERR_INVALID_ARG, "%s must be non-null and 16-byte aligned", what);
    if (ld < heads * c->D || ld >= kMaxStride || ld * c->elem_bytes % 16 != 0)
        return fail(NE_ERR_INVALID_ARG, "%s rows must be at least %lld elements apart, in multiples of 16 bytes (%lld)", what,
                    (long long)(heads * c->D), (long long)ld);
    return NE_OK;
}

ne_status check_batch(const ne_paged_cache* c, const int* table, const int* lens, const int* cu, int B, int N, int heads,
                      int max_pages) {
    if (B < 0 || N < 0) return fail(NE_ERR_INVALID_ARG, "B and N must be >= 0 (B=%d N=%d)", B, N);
    if (heads < 1 || heads > (1 << 20)) return fail(NE_ERR_INVALID_ARG, "need 1 <= Hq <= 2^20 (Hq=%d)", heads);
    if ((long long)N * std::max(heads, c->Hkv) * c->D >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "N * max(Hq, Hkv) * D must be < 2^31");
    if (B == 0 || N == 0) return NE_OK;
    if (!cu && N != B) return fail(NE_ERR_INVALID_ARG, "without cu_new every sequence has one row: N == B (N=%d B=%d)", N, B);
    if (max_pages < 1 || (long long)max_pages * c->page_size > (1 << 30) || (long long)B * max_pages >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "need max_pages >= 1, max_pages * page_size <= 2^30 and B * max_pages < 2^31 (max_pages=%d)",
                    max_pages);
    if (!aligned4(table) || !aligned4(lens) || (cu && !aligned4(cu)))
        return fail(NE_ERR_INVALID_ARG, "page_table, seq_lens and cu_new must be non-null, 4-byte aligned device pointers");
    return NE_OK;
}

int log2_of(int x) {
    int s = 0;
    while ((1 << s) < x) ++s;
    return s;
}

// Strides of an extent of one are never used; a plain value keeps the tensor maps valid.
ne::PagedView view_of(const ne_paged_cache* c) {
    ne::PagedView v;
    v.k = c->k;
    v.v = c->v;
    v.n_pages = c->n_pages;
    v.ps_shift = log2_of(c->page_size);
    v.page_stride = c->n_pages > 1 ? c->page_stride : c->D;
    v.tok_stride = c->tok_stride;
    v.head_stride = c->Hkv > 1 ? c->head_stride : c->D;
    return v;
}

ne::PagedBatch batch_of(const ne_paged_cache* c, const int* table, const int* lens, const int* cu, int B, int N, int W) {
    ne::PagedBatch s;
    s.table = table;
    s.lens = lens;
    s.cu = cu;
    s.B = B;
    s.N = N;
    s.W = W;
    s.cap = W * c->page_size;
    return s;
}

// The device error word.  Its first use allocates, which a capture does not allow.
ne_status ready(cudaStream_t st, int** err) {
    int dev;
    ne_status s = current_device(&dev);
    if (s != NE_OK) return s;
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (!have_error_word(dev) && cudaStreamIsCapturing(st, &cap) == cudaSuccess && cap != cudaStreamCaptureStatusNone)
        return fail(NE_ERR_UNSUPPORTED,
                    "first call on this device happened inside stream capture; make one call before capturing");
    return error_word(dev, err);
}

ne_status append_impl(int eb, const void* q, const void* k, const void* v, const ne_paged_cache* c, const int* table,
                      const int* lens, const int* cu, const ne_rope_spec* spec, int pos_offset, const int* pos_offsets, void* q_out,
                      int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t qo_ld, int B, int N, int Hq, int W, ne_stream_t stream) {
    clear_error();
    ne_status s = check_cache(c, eb, true);
    if (s != NE_OK) return s;
    if ((q == nullptr) != (q_out == nullptr)) return fail(NE_ERR_INVALID_ARG, "q and q_out go together");
    if ((s = check_batch(c, table, lens, cu, B, N, q ? Hq : c->Hkv, W)) != NE_OK) return s;
    if (spec && (spec->D != c->D || spec->rot_dim < 2 || spec->rot_dim > c->D || spec->rot_dim % 2 ||
                 (spec->layout != 0 && spec->layout != 1)))
        return fail(NE_ERR_INVALID_ARG, "the rope spec is not one of ne_rope_spec_init for D=%d", c->D);
    if (pos_offset < 0 || pos_offset >= (1 << 30)) return fail(NE_ERR_INVALID_ARG, "need 0 <= pos_offset < 2^30");
    if (B == 0 || N == 0) return NE_OK;
    if ((s = check_rows("k", k, k_ld, c->Hkv, c)) != NE_OK) return s;
    if ((s = check_rows("v", v, v_ld, c->Hkv, c)) != NE_OK) return s;
    if (q) {
        if ((s = check_rows("q", q, q_ld, Hq, c)) != NE_OK) return s;
        if ((s = check_rows("q_out", q_out, qo_ld, Hq, c)) != NE_OK) return s;
        const int64_t e = c->elem_bytes, qw = (int64_t)Hq * c->D * e, kw = (int64_t)c->Hkv * c->D * e;
        if (q == q_out ? q_ld != qo_ld : rows_overlap(q_out, qw, qo_ld * e, q, qw, q_ld * e, N))
            return fail(NE_ERR_INVALID_ARG, "q_out must be q itself, with the same row stride, or not overlap it");
        if (rows_overlap(q_out, qw, qo_ld * e, k, kw, k_ld * e, N) || rows_overlap(q_out, qw, qo_ld * e, v, kw, v_ld * e, N))
            return fail(NE_ERR_INVALID_ARG, "q_out must not overlap k or v");
    }
    ne::AppendArgs a = {};
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    a.c = view_of(c);
    a.s = batch_of(c, table, lens, cu, B, N, W);
    a.q = q;
    a.k_in = k;
    a.v_in = v;
    a.q_out = q_out;
    a.q_ld = q_ld;
    a.k_ld = k_ld;
    a.v_ld = v_ld;
    a.qo_ld = qo_ld;
    a.Hq = Hq;
    a.Hkv = c->Hkv;
    a.D = c->D;
    a.rot = spec ? spec->rot_dim : 0;
    a.layout = spec ? spec->layout : 0;
    a.mscale = spec ? spec->mscale : 1.f;
    a.pos_offset = pos_offset;
    a.pos_offsets = pos_offsets;
    ne::RopeTurns turns = {};
    if (spec)
        for (int i = 0; i < spec->rot_dim / 2; ++i) turns.t[i] = spec->turns[i];
    cudaError_t e = ne::launch_paged_append(eb == 4, a, turns, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged_append launch");
    return NE_OK;
}

// Tensor maps of the tile kernels: a query box is (64 columns, `heads` heads, `sub` tokens), a
// key or value box (64 columns, one head, the rows of a page that fall into one tile).  tv null: keys alone.
ne_status tile_maps(CUtensorMap* tq, CUtensorMap* tk, CUtensorMap* tv, const ne_paged_cache* c, const ne::PagedView& v, const void* q,
                    int64_t q_ld, int Hq, int N, int heads, int sub) {
    EncodeTiledFn enc;
    ne_status s = encode_fn(&enc);
    if (s != NE_OK) return s;
    auto encode = [&](CUtensorMap* m, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                      const cuuint32_t* box) -> ne_status {
        const cuuint32_t one[4] = {1, 1, 1, 1};
        CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(p), dims, strides, box, one,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        return r == CUDA_SUCCESS ? NE_OK : fail(NE_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    };
    const cuuint64_t qd[3] = {(cuuint64_t)c->D, (cuuint64_t)Hq, (cuuint64_t)N};
    const cuuint64_t qs[2] = {(cuuint64_t)c->D * 2, (cuuint64_t)q_ld * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)heads, (cuuint32_t)sub};
    if ((s = encode(tq, q, 3, qd, qs, qb)) != NE_OK) return s;
    const cuuint64_t kd[4] = {(cuuint64_t)c->D, (cuuint64_t)c->Hkv, (cuuint64_t)c->page_size, (cuuint64_t)c->n_pages};
    const cuuint64_t ks[3] = {(cuuint64_t)v.head_stride * 2, (cuuint64_t)v.tok_stride * 2, (cuuint64_t)v.page_stride * 2};
    const cuuint32_t kb[4] = {64, 1, (cuuint32_t)std::min(c->page_size, 128), 1};
    if ((s = encode(tk, v.k, 4, kd, ks, kb)) != NE_OK || !tv) return s;
    return encode(tv, v.v, 4, kd, ks, kb);
}

// Bytes of a call's workspace: the largest over the kernels that its head_dim and heads may run.
size_t attn_ws_bytes(int D, int Hkv, int G) {
    static thread_local struct {
        int D, Hkv, G;
        size_t bytes;
    } last = {0, 0, 0, 0};                     // (twenty splits to look through: a loop over layers asks for one shape)
    if (D == last.D && Hkv == last.Hkv && G == last.G) return last.bytes;
    size_t most = 0;
    for (int f32 = 0; f32 < 2; ++f32)
        for (int rows : {1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 1 << 20}) {
            if (f32 && D > 64) continue;
            const ne::PagedKind kind = ne::paged_kind(f32 != 0, D, G, rows);
            most = std::max(most, ne::paged_part_bytes(ne::paged_split(kind, D, Hkv, G, 1 << 30), D));
        }
    last = {D, Hkv, G, round_up(most, 256)};
    return last.bytes;
}

// Checks of a call of ne_paged_attn but for its workspace.
ne_status attn_check(int eb, const void* q, const ne_paged_cache* c, const int* table, const int* lens, const int* cu,
                     const void* o, const float* lse, int64_t q_ld, int B, int N, int Hq, int W, int max_new) {
    ne_status s = check_cache(c, eb, true);
    if (s != NE_OK) return s;
    if (Hq < 1 || Hq % c->Hkv != 0)
        return fail(NE_ERR_INVALID_ARG, "need Hq > 0 and Hq %% Hkv == 0 (Hq=%d Hkv=%d)", Hq, c->Hkv);
    if ((s = check_batch(c, table, lens, cu, B, N, Hq, W)) != NE_OK) return s;
    if (max_new < 1) return fail(NE_ERR_INVALID_ARG, "max_new must be >= 1 (max_new=%d)", max_new);
    if (B == 0 || N == 0) return NE_OK;
    if ((s = check_rows("q", q, q_ld, Hq, c)) != NE_OK) return s;
    if ((s = check_ptrs({o, lse})) != NE_OK) return s;
    const int64_t row = (int64_t)Hq * c->D * eb;
    if (rows_overlap(o, row, row, q, row, q_ld * eb, N) || rows_overlap(lse, Hq * 4, Hq * 4, q, row, q_ld * eb, N) ||
        overlap(o, (size_t)(row * N), lse, (size_t)N * Hq * 4))
        return fail(NE_ERR_INVALID_ARG, "o, lse and q must not overlap");
    return NE_OK;
}

ne_status attn_ws_check(const void* ws, size_t ws_bytes, size_t need) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return fail(NE_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned (%zu bytes needed)", need);
    if (ws_bytes < need)
        return fail(NE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
    return NE_OK;
}

// What the kernels of a call are told; `ws` holds the parts.
ne_status attn_args(ne::PagedAttnArgs* out, ne::PagedKind kind, const void* q, const ne_paged_cache* c, const int* table,
                    const int* lens, const int* cu, void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int W, void* ws,
                    ne_stream_t stream) {
    ne::PagedAttnArgs& a = *out;
    a = ne::PagedAttnArgs();
    const ne_status s = ready((cudaStream_t)stream, &a.err);
    if (s != NE_OK) return s;
    a.c = view_of(c);
    a.s = batch_of(c, table, lens, cu, B, N, W);
    a.G = Hq / c->Hkv;
    a.p = ne::paged_split(kind, c->D, c->Hkv, a.G, a.s.cap);
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.q_ld = q_ld;
    a.Hq = Hq;
    a.Hkv = c->Hkv;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->D));
    const size_t parts = 2 * (size_t)a.p.C;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + parts * a.p.rows * c->D);
    a.part_info = reinterpret_cast<int4*>(a.part_ml + parts * a.p.rows);
    a.timeout_ns = timeout_ns();
    return NE_OK;
}

// The call behind its checks.
ne_status attn_run(int eb, const void* q, const ne_paged_cache* c, const int* table, const int* lens, const int* cu,
                   void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int W, int max_new, void* ws, ne_stream_t stream) {
    const int G = Hq / c->Hkv;
    ne_status s;
    const bool f32 = eb == 4;
    const ne::PagedKind kind = ne::paged_kind(f32, c->D, G, cu ? std::min(max_new, N) : 1);
    ne::PagedAttnArgs a;
    if ((s = attn_args(&a, kind, q, c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, ws, stream)) != NE_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (kind == ne::PAGED_TILES) {
        CUtensorMap tq, tk, tv;
        if ((s = tile_maps(&tq, &tk, &tv, c, a.c, q, q_ld, Hq, N, a.G, a.p.sub)) != NE_OK) return s;
        e = ne::launch_paged_tiles(c->D, tq, tk, tv, a, st);
    } else if (f32) e = ne::launch_paged_f32(kind, c->D, a, st);
    else e = ne::launch_paged_short(kind, c->D, a, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged_attn launch");
    if (a.p.nocut) return NE_OK;
    e = ne::launch_paged_join(f32, c->D, a, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged_attn join launch");
    return NE_OK;
}

ne_status attn_impl(int eb, const void* q, const ne_paged_cache* c, const int* table, const int* lens, const int* cu,
                    void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int W, int max_new, void* ws,
                    size_t ws_bytes, ne_stream_t stream) {
    clear_error();
    ne_status s = attn_check(eb, q, c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, max_new);
    if (s != NE_OK || B == 0 || N == 0) return s;
    if ((s = attn_ws_check(ws, ws_bytes, attn_ws_bytes(c->D, c->Hkv, Hq / c->Hkv))) != NE_OK) return s;
    return attn_run(eb, q, c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, max_new, ws, stream);
}

// ---------------------------------------------------------------- shared prefixes
// Where a call runs as ne_paged_attn.
// (1) While all sequences' caches, as large as their tables, take no more bytes than this, reading them all beats a
// join of two lines: bf16, 33 MB 14.5 us against 16.5, 65 MB 18.1 against 17.1, 132 MB 25.8 against 19.3; fp32
// with up to 32 rows a sequence 134 MB 22 against 32, 537 MB 59 against 54 (its products take as long either way).
constexpr long long kSharedBytes = 64LL << 20, kSharedBytesF32 = 256LL << 20;
// (2) With more than 32 rows a sequence ne_paged_attn has tiles of 256 rows (fp32: 64), too: shared, the tiles of a
// prefix are full, but every sequence has a part more.  It pays where the part of the tiles that would be empty, times
// the positions of a table, reaches this.
// bf16, 16 sequences, 12/4 heads of 64: 192 rows each (a quarter empty) over 4096 alone 30.1 us, shared 32.6, over
// 16384 75 and 71; 240 rows 77 and 109; up to 768 rows over 8192 83 and 73.  200 shapes (lengths alike and different, 2048
// to 16384 positions, head_dims 64 and 128): 7.6% faster than never sharing, 7.8 by the better of both each time.
// fp32, the same with 4 heads: 80 rows (three eighths empty) over 1024 93 and 79, over 4096 297 and 203; 64 rows over
// 4096 154 and 170; up to 64 rows over 1024 50 and 50, over 4096 148 and 107.
constexpr double kSharedEmpty = 1200., kSharedEmptyF32 = 600.;
// (3) The same in bf16 at head_dim 32, where ne_paged_attn takes 32 rows at a time: from so many rows times positions of
// all sequences on (12/4 heads: 4 sequences of 64 over 2300 19.5 us against 26.1 shared, 4 of 200 over 600 21.5 and 19.5, 16
// of 64 over 2100 41 and 27, 16 of up to 256 over 8192 179 and 92.  85 shapes, 2 to 32 sequences, 12/4, 8/1 and 4/2 heads: 1.4%
// slower than the better of both each time; never sharing 8.1%, always 16%).
constexpr double kSharedWork = 9e6;

// (2) and (3): whether sharing pays.
bool shared_pays(bool f32, int D, int G, int Hq, int most, int N, int B, long long cap) {
    const double mean = (double)N / B;
    if (!f32 && D == 32) return (double)N * Hq * (double)cap >= kSharedWork;
    // Row tiles of a sequence (bf16: one with half its rows or fewer takes 0.8 of the time), and how many its rows fill.
    const int sub = f32 ? std::max(64 / G, 1) : 128 / G, tpt = f32 ? sub : 2 * sub, rem = most % tpt;
    const double full = mean / tpt, half = f32 ? 1. : 0.8;
    double tiles;
    if (N == (long long)B * most) tiles = most / tpt + (rem == 0 ? 0. : rem <= sub ? half : 1.);
    else tiles = most <= sub ? half : most <= tpt ? 0.9 : full + 0.5 * half;   // (lengths differ: half a tile is empty)
    return (tiles - full) * (double)cap >= (f32 ? kSharedEmptyF32 : kSharedEmpty) * tiles;
}

struct SharedWs {
    size_t parts, row_o, row_ml, rec, total;   // parts, row_o, row_ml and records of one of the two lines; both
};
SharedWs shared_ws(int N, int Hq, int Hkv, int D) {
    const int G = Hq / Hkv;
    SharedWs w;
    w.parts = attn_ws_bytes(D, Hkv, G);
    if (G <= 128) w.parts = std::max(w.parts, round_up(ne::paged_part_bytes(ne::paged_split(ne::PAGED_TILES, D, Hkv, G, 1 << 30), D), 256));
    const size_t rows = (size_t)N * Hq;
    w.row_o = round_up(rows * D * 4, 256);
    w.row_ml = round_up(rows * 8, 256);
    w.rec = round_up(rows * 8, 256);           // (a head group has at least one head)
    w.total = 2 * (w.parts + w.row_o + w.row_ml + w.rec);
    return w;
}

ne_status shared_impl(int eb, const void* q, const ne_paged_cache* c, const int* table, const int* lens, const int* cu,
                      const int* groups, const int* shared, int R, void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int W,
                      int max_new, void* ws, size_t ws_bytes, ne_stream_t stream) {
    clear_error();
    ne_status s = attn_check(eb, q, c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, max_new);
    if (s != NE_OK) return s;
    if (R < 0 || R > B || (long long)R + B >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "need 0 <= R <= B groups and R + B < 2^31 (R=%d B=%d)", R, B);
    if (B == 0 || N == 0) return NE_OK;
    if (!aligned4(groups) || (R > 0 && !aligned4(shared)))
        return fail(NE_ERR_INVALID_ARG, "groups and shared must be non-null, 4-byte aligned device pointers");
    const SharedWs w = shared_ws(N, Hq, c->Hkv, c->D);
    if ((s = attn_ws_check(ws, ws_bytes, w.total)) != NE_OK) return s;
    const int G = Hq / c->Hkv, most = cu ? std::min(max_new, N) : 1;
    const bool f32 = eb == 4;
    const long long bytes = (long long)B * W * c->page_size * c->Hkv * 2 * c->D * eb;
    const long long rows_each = (long long)most * G;
    bool alone = R == 0 || (!f32 && G > 128);
    if (rows_each <= 32 || (!f32 && c->D != 32)) alone |= bytes <= (f32 ? kSharedBytesF32 : kSharedBytes);
    if (!alone && rows_each > 32) alone = !shared_pays(f32, c->D, G, Hq, most, N, B, (long long)W * c->page_size);
    if (alone)
        return attn_run(eb, q, c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, max_new, ws, stream);
    // bf16: one line of prefixes and own positions, tiles for all.  fp32: a line and a kernel for each,
    // chosen by the rows of a group and of a sequence.
    const int lines = f32 ? 2 : 1;
    ne::PagedAttnArgs a[2];                    // prefixes (and own positions), own positions
    ne::PagedKind kind[2] = {f32 ? ne::paged_kind(true, c->D, G, N) : ne::PAGED_TILES, ne::paged_kind(true, c->D, G, most)};
    char* rows = static_cast<char*>(ws) + 2 * w.parts;
    for (int i = 0; i < lines; ++i) {
        if ((s = attn_args(&a[i], kind[i], q, c, table, lens, cu, o, lse, q_ld, lines == 1 ? R + B : i ? B : R, N, Hq, W,
                           static_cast<char*>(ws) + i * w.parts, stream)) != NE_OK)
            return s;
        // A part's ends with its fp32 rows: less than two tiles where few of them are live (35 shapes, geometric mean: 21.0
        // us with 896, 20.3 with 1024, 20.8 with 1152, 20.6 with 1280 and 1408), nearly three where all are, and then a part of
        // one subtile waits as long per key tile (138 shapes: 66.7 us as with few, 64.8 as here).
        if (!f32) {
            a[i].p.ovh = rows_each > 32 ? 1792 : 1024;
            if (rows_each > 32) a[i].p.w_part = a[i].p.w_full;
        }
        a[i].s.groups = groups;
        a[i].s.shared = shared;
        a[i].s.R = R;
        a[i].s.seqs = B;
        a[i].s.pre = i ? 0 : R;
        a[i].s.err = a[i].err;
        for (int k = 0; k < 2; ++k) {
            char* base = rows + k * (w.row_o + w.row_ml + w.rec);
            a[i].row_o[k] = reinterpret_cast<float*>(base);
            a[i].row_ml[k] = reinterpret_cast<float2*>(base + w.row_o);
            a[i].rec_first[k] = reinterpret_cast<int*>(base + w.row_o + w.row_ml);
            a[i].rec_last[k] = a[i].rec_first[k] + (size_t)N * Hq;
        }
    }
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (!f32) {
        CUtensorMap tq, tk, tv;
        if ((s = tile_maps(&tq, &tk, &tv, c, a[0].c, q, q_ld, Hq, N, G, a[0].p.sub)) != NE_OK) return s;
        // The bits of a weight are those of ne_paged_attn: its kernels for few rows, which take head_dim 32 whatever the
        // rows, keep two bf16 terms.
        e = ne::launch_shared_tiles(c->D, rows_each <= 32 || c->D == 32 ? 2 : 1, tq, tk, tv, a[0], st);
    } else {
        e = ne::launch_shared_f32(kind[0], c->D, a[0], st);
        if (e == cudaSuccess) e = ne::launch_shared_f32(kind[1], c->D, a[1], st);
    }
    if (e == cudaSuccess) e = ne::launch_shared_join(f32, c->D, a[0], a[lines - 1], st);
    return e == cudaSuccess ? NE_OK : cuda_fail(e, "paged_attn_shared launch");
}

// ---------------------------------------------------------------- accumulated weights
constexpr size_t kWeightParts = 2 * (size_t)ne::kWeightCtas;
constexpr size_t kWeightWs = kWeightParts * (ne::kWeightKeys * sizeof(float) + sizeof(int4));

ne_status weights_impl(int eb, const void* q, const float* lse, const ne_paged_cache* c, const int* table, const int* lens,
                       const int* cu, const float* weights, float* weights_out, int64_t q_ld, int B, int N, int Hq, int W,
                       int max_new, void* ws, size_t ws_bytes, ne_stream_t stream) {
    clear_error();
    ne_status s = check_cache(c, eb, true);
    if (s != NE_OK) return s;
    if (Hq < 1 || Hq % c->Hkv != 0)
        return fail(NE_ERR_INVALID_ARG, "need Hq > 0 and Hq %% Hkv == 0 (Hq=%d Hkv=%d)", Hq, c->Hkv);
    if (B < 0 || N < 0) return fail(NE_ERR_INVALID_ARG, "B and N must be >= 0 (B=%d N=%d)", B, N);
    if (max_new < 1) return fail(NE_ERR_INVALID_ARG, "max_new must be >= 1 (max_new=%d)", max_new);
    if (B == 0) return NE_OK;
    // (Without new tokens the weights are still copied: the batch is checked as if it had one.)
    if (!cu && N != B) return fail(NE_ERR_INVALID_ARG, "without cu_new every sequence has one row: N == B (N=%d B=%d)", N, B);
    if ((s = check_batch(c, table, lens, N > 0 ? cu : lens, B, std::max(N, 1), Hq, W)) != NE_OK) return s;
    if (N == 0 && cu && !aligned4(cu)) return fail(NE_ERR_INVALID_ARG, "cu_new must be a 4-byte aligned device pointer");
    const size_t row = (size_t)Hq * c->D * eb, wb = (size_t)B * c->Hkv * W * c->page_size * 4;
    if (!aligned4(weights_out) || (weights && !aligned4(weights)))
        return fail(NE_ERR_INVALID_ARG, "weights and weights_out must be 4-byte aligned device pointers, weights_out non-null");
    if (weights && weights != weights_out && overlap(weights, wb, weights_out, wb))
        return fail(NE_ERR_INVALID_ARG, "weights_out must be weights itself or not overlap it");
    if (N > 0) {
        if ((s = check_rows("q", q, q_ld, Hq, c)) != NE_OK) return s;
        if (!aligned4(lse)) return fail(NE_ERR_INVALID_ARG, "lse must be a non-null, 4-byte aligned device pointer");
        if (overlap(weights_out, wb, q, (size_t)(q_ld * eb * (N - 1)) + row) || overlap(weights_out, wb, lse, (size_t)N * Hq * 4))
            return fail(NE_ERR_INVALID_ARG, "weights_out must not overlap q or lse");
    }
    const ne::WeightKind kind = N == 0 ? ne::WEIGHTS_FEW4 : ne::weight_kind(eb == 4, Hq / c->Hkv, cu ? std::min(max_new, N) : 1);
    if (kind >= ne::WEIGHTS_MANY) {
        if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
            return fail(NE_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned (%zu bytes needed)", kWeightWs);
        if (ws_bytes < kWeightWs)
            return fail(NE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", ws_bytes, kWeightWs);
    }
    ne::WeightArgs a = {};
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    a.c = view_of(c);
    a.s = batch_of(c, table, lens, cu, B, N, W);
    a.q = q;
    a.lse = lse;
    a.w = weights;
    a.w_out = weights_out;
    a.q_ld = q_ld;
    a.Hq = Hq;
    a.Hkv = c->Hkv;
    a.G = Hq / c->Hkv;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->D));
    a.part = static_cast<float*>(ws);
    a.part_info = reinterpret_cast<int4*>(a.part + kWeightParts * ne::kWeightKeys);
    a.timeout_ns = timeout_ns();
    ne::weight_split(kind, a);
    CUtensorMap tq = {}, tk = {};
    if (kind == ne::WEIGHTS_MANY && (s = tile_maps(&tq, &tk, nullptr, c, a.c, q, q_ld, Hq, N, a.gs, a.sub)) != NE_OK) return s;
    const cudaError_t e = ne::launch_paged_weights(kind, eb == 4, c->D, tq, tk, a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged_weights launch");
    return NE_OK;
}

// ---------------------------------------------------------------- pages
struct PagesWs {
    size_t off, free_ids, list, total;
};
PagesWs pages_ws(int n_pages, int n, int W) {
    // Listed pages: those taken (at most one per table entry and one per page), or those a
    // compaction moves (at most half of the pool).
    const size_t taken = std::min((size_t)n_pages, (size_t)n * W);
    const size_t most = std::max(taken, (size_t)n_pages / 2 + 1);
    PagesWs w;
    w.off = 256;
    w.free_ids = w.off + round_up((size_t)n * 8, 256);
    w.list = w.free_ids + round_up(most * 4, 256);
    w.total = w.list + round_up(most * 16, 256);
    return w;
}

// Everything the three calls share.  n: sequences that take pages; more_out [more_n]: child
// lengths or remap; same_ok: table_out may be page_table.
ne_status pages_args(ne::PagesArgs* a, const ne_paged_cache* c, const int* ref, const int* table, const int* lens,
                     const int* other, int* ref_out, int* table_out, int* more_out, size_t more_n, int* one_out, int B, int W,
                     int n, bool same_ok, void* ws, size_t ws_bytes) {
    clear_error();
    ne_status s = check_cache(c, 0, false);
    if (s != NE_OK) return s;
    if (B < 0 || n < 0) return fail(NE_ERR_INVALID_ARG, "sequence counts must be >= 0 (%d, %d)", B, n);
    if (W < 1 || (long long)W * c->page_size > (1 << 30) || (long long)std::max(B, n) * W >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "need max_pages >= 1, max_pages * page_size <= 2^30 and sequences * max_pages < 2^31 "
                    "(max_pages=%d)", W);
    if ((s = check_ptrs({ref, ref_out})) != NE_OK) return s;
    // The int arrays: inputs first, then outputs.  No output overlaps anything but the input it
    // may be itself.
    struct Ints {
        const int* p;
        size_t n;
        const char* name;
    };
    const size_t P = c->n_pages;
    const Ints in[4] = {{ref, P, "refcount"}, {table, (size_t)B * W, "page_table"}, {lens, lens ? (size_t)B : 0, "seq_lens"},
                        {other, other ? (size_t)n : 0, "parents or new_lens"}};
    const Ints out[4] = {{ref_out, P, "refcount_out"}, {table_out, (size_t)n * W, "table_out"}, {more_out, more_n, "child_lens or remap"},
                         {one_out, 1, "short_out or n_live"}};
    for (int i = 0; i < 4; ++i)
        for (const Ints* a1 : {&in[i], &out[i]})
            if (a1->n > 0 && !aligned4(a1->p))
                return fail(NE_ERR_INVALID_ARG, "%s must be a non-null, 4-byte aligned device pointer", a1->name);
    for (int i = 0; i < 4; ++i) {
        for (int k = 0; k < 4; ++k) {
            const bool itself = out[i].p == in[k].p && i == k && (i == 0 || (i == 1 && same_ok));
            if (out[i].n > 0 && in[k].n > 0 && !itself && overlap(out[i].p, out[i].n * 4, in[k].p, in[k].n * 4))
                return fail(NE_ERR_INVALID_ARG, "%s must not overlap %s", out[i].name, in[k].name);
        }
        for (int k = 0; k < i; ++k)
            if (out[i].n > 0 && out[k].n > 0 && overlap(out[i].p, out[i].n * 4, out[k].p, out[k].n * 4))
                return fail(NE_ERR_INVALID_ARG, "%s must not overlap %s", out[i].name, out[k].name);
    }
    const PagesWs w = pages_ws(c->n_pages, n, W);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return fail(NE_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned (%zu bytes needed)", w.total);
    if (ws_bytes < w.total)
        return fail(NE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", ws_bytes, w.total);
    *a = ne::PagesArgs();
    const int e = c->elem_bytes;
    a->k = static_cast<char*>(c->k);
    a->v = static_cast<char*>(c->v);
    a->layers = c->layers;
    a->n_pages = c->n_pages;
    a->ps = c->page_size;
    a->ps_shift = log2_of(c->page_size);
    a->Hkv = c->Hkv;
    a->row_vecs = c->D * e / 16;
    a->row_shift = log2_of(a->row_vecs);
    a->layer_stride = c->layers > 1 ? c->layer_stride * e : 0;
    a->page_stride = c->n_pages > 1 ? c->page_stride * e : 0;
    a->tok_stride = c->tok_stride * e;
    a->head_stride = c->Hkv > 1 ? c->head_stride * e : 0;
    a->ref = ref;
    a->table = table;
    a->ref_out = ref_out;
    a->table_out = table_out;
    a->short_out = one_out;
    a->B = B;
    a->W = W;
    a->n = n;
    a->cap = W * c->page_size;
    char* base = static_cast<char*>(ws);
    a->head = reinterpret_cast<int*>(base);
    a->off = reinterpret_cast<int2*>(base + w.off);
    a->free_ids = reinterpret_cast<int*>(base + w.free_ids);
    a->list = reinterpret_cast<int4*>(base + w.list);
    return NE_OK;
}

// ---------------------------------------------------------------- cuts by weight
struct EvictWs {
    size_t list, total;
};
EvictWs evict_ws(size_t rows, size_t T) {
    EvictWs w;
    w.list = round_up(rows * 4, 256);
    w.total = w.list + round_up(rows * T * 4, 256);
    return w;
}

// Arrays of a call: no output overlaps anything but the input that it may be itself (same: its
// index among the inputs, -1 for none).
struct CallArray {
    const void* p;
    size_t bytes;
    const char* name;
    int same;
};
ne_status check_arrays(std::initializer_list<CallArray> in, std::initializer_list<CallArray> out) {
    for (const auto* list : {&in, &out})
        for (const CallArray& x : *list)
            if (x.bytes > 0 && !aligned4(x.p))
                return fail(NE_ERR_INVALID_ARG, "%s must be a non-null, 4-byte aligned device pointer", x.name);
    for (const CallArray& o : out) {
        int k = 0;
        for (const CallArray& i : in) {
            const bool itself = k++ == o.same && o.p == i.p;
            if (o.bytes > 0 && i.bytes > 0 && !itself && overlap(o.p, o.bytes, i.p, i.bytes))
                return fail(NE_ERR_INVALID_ARG, "%s must not overlap %s", o.name, i.name);
        }
        for (const CallArray& i : out)
            if (&i < &o && o.bytes > 0 && i.bytes > 0 && overlap(o.p, o.bytes, i.p, i.bytes))
                return fail(NE_ERR_INVALID_ARG, "%s must not overlap %s", o.name, i.name);
    }
    return NE_OK;
}

}  // namespace

extern "C" {

ne_status ne_rope_spec_init(ne_rope_spec* out, int D, int rot_dim, int layout, double theta, int scaling, double factor,
                            int orig_len, double beta_fast, double beta_slow, double mscale) {
    clear_error();
    if (!out) return fail(NE_ERR_INVALID_ARG, "null output");
    if (D <= 0 || D > 128 || D % 2 != 0) return fail(NE_ERR_INVALID_ARG, "D must be even, 2 to 128 (D=%d)", D);
    if (rot_dim < 2 || rot_dim > D || rot_dim % 2 != 0)
        return fail(NE_ERR_INVALID_ARG, "rot_dim must be even, 2 to D (rot_dim=%d D=%d)", rot_dim, D);
    if (layout != 0 && layout != 1) return fail(NE_ERR_INVALID_ARG, "layout must be 0 (interleaved) or 1 (half)");
    if (!(theta > 0.0) || !std::isfinite(theta)) return fail(NE_ERR_INVALID_ARG, "theta must be finite and > 0");
    if (!(std::fabs(mscale) <= FLT_MAX)) return fail(NE_ERR_INVALID_ARG, "mscale must be finite in fp32");
    if (scaling < NE_ROPE_NONE || scaling > NE_ROPE_PARTS) return fail(NE_ERR_INVALID_ARG, "unknown scaling %d", scaling);
    if (scaling != NE_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor)))
        return fail(NE_ERR_INVALID_ARG, "factor must be finite and > 0");
    if (scaling == NE_ROPE_BASE && rot_dim < 4) return fail(NE_ERR_INVALID_ARG, "base scaling needs rot_dim >= 4");
    if (scaling == NE_ROPE_PARTS && (orig_len < 1 || !(beta_fast > beta_slow) || !std::isfinite(beta_fast) ||
                                     !std::isfinite(beta_slow)))
        return fail(NE_ERR_INVALID_ARG, "scaling by parts needs orig_len >= 1 and finite beta_fast > beta_slow");
    double base = theta;
    if (scaling == NE_ROPE_BASE) base = theta * std::pow(factor, rot_dim / (rot_dim - 2.0));
    if (!(base > 0.0) || !std::isfinite(base))
        return fail(NE_ERR_INVALID_ARG, "the scaled base theta * factor^(rot_dim / (rot_dim - 2)) must be finite and > 0 (%g)", base);
    ne_rope_spec spec = ne_rope_spec();
    spec.D = D;
    spec.rot_dim = rot_dim;
    spec.layout = layout;
    spec.mscale = (float)mscale;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == NE_ROPE_LINEAR) f /= factor;
        if (scaling == NE_ROPE_PARTS) {
            const double n = orig_len * f / kTwoPi;
            const double g = std::min(1.0, std::max(0.0, (n - beta_slow) / (beta_fast - beta_slow)));
            f *= g + (1.0 - g) / factor;
        }
        if (!std::isfinite(f)) return fail(NE_ERR_INVALID_ARG, "the frequency of pair %d is not finite (%g)", i, f);
        // Turns per position, whole turns dropped, in units of 2^-64.
        double t = f / kTwoPi;
        t -= std::floor(t);
        const double hi = std::floor(t * 4294967296.0);    // two exact halves of the 64-bit fraction
        const double lo = std::floor((t * 4294967296.0 - hi) * 4294967296.0 + 0.5);
        spec.turns[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
    }
    *out = spec;
    return NE_OK;
}

ne_status ne_paged_append(const void* q, const void* k, const void* v, const ne_paged_cache* cache, const int* page_table,
                          const int* seq_lens, const int* cu_new, const ne_rope_spec* spec, int pos_offset, void* q_out,
                          int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t q_out_ld, int B, int N, int Hq, int max_pages,
                          ne_stream_t stream) {
    return append_impl(2, q, k, v, cache, page_table, seq_lens, cu_new, spec, pos_offset, nullptr, q_out, q_ld, k_ld, v_ld,
                       q_out_ld, B, N, Hq, max_pages, stream);
}

ne_status ne_paged_append_f32(const float* q, const float* k, const float* v, const ne_paged_cache* cache,
                              const int* page_table, const int* seq_lens, const int* cu_new, const ne_rope_spec* spec,
                              int pos_offset, float* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t q_out_ld,
                              int B, int N, int Hq, int max_pages, ne_stream_t stream) {
    return append_impl(4, q, k, v, cache, page_table, seq_lens, cu_new, spec, pos_offset, nullptr, q_out, q_ld, k_ld, v_ld,
                       q_out_ld, B, N, Hq, max_pages, stream);
}

ne_status ne_paged_append_at(const void* q, const void* k, const void* v, const ne_paged_cache* cache, const int* page_table,
                             const int* seq_lens, const int* cu_new, const ne_rope_spec* spec, const int* pos_offsets,
                             void* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t q_out_ld, int B, int N, int Hq,
                             int max_pages, ne_stream_t stream) {
    clear_error();
    if (B > 0 && N > 0 && !aligned4(pos_offsets)) return fail(NE_ERR_INVALID_ARG, "pos_offsets must be a non-null, 4-byte aligned device pointer");
    return append_impl(2, q, k, v, cache, page_table, seq_lens, cu_new, spec, 0, pos_offsets, q_out, q_ld, k_ld, v_ld, q_out_ld,
                       B, N, Hq, max_pages, stream);
}

ne_status ne_paged_append_at_f32(const float* q, const float* k, const float* v, const ne_paged_cache* cache,
                                 const int* page_table, const int* seq_lens, const int* cu_new, const ne_rope_spec* spec,
                                 const int* pos_offsets, float* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                                 int64_t q_out_ld, int B, int N, int Hq, int max_pages, ne_stream_t stream) {
    clear_error();
    if (B > 0 && N > 0 && !aligned4(pos_offsets)) return fail(NE_ERR_INVALID_ARG, "pos_offsets must be a non-null, 4-byte aligned device pointer");
    return append_impl(4, q, k, v, cache, page_table, seq_lens, cu_new, spec, 0, pos_offsets, q_out, q_ld, k_ld, v_ld, q_out_ld,
                       B, N, Hq, max_pages, stream);
}

size_t ne_paged_attn_workspace_size(int B, int N, int Hq, int Hkv, int D) {
    if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 32 && D != 64 && D != 128)) return 0;
    return attn_ws_bytes(D, Hkv, Hq / Hkv);
}

ne_status ne_paged_attn(const void* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                        const int* cu_new, void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int max_pages,
                        int max_new, void* workspace, size_t workspace_bytes, ne_stream_t stream) {
    return attn_impl(2, q, cache, page_table, seq_lens, cu_new, o, lse, q_ld, B, N, Hq, max_pages, max_new, workspace,
                     workspace_bytes, stream);
}

ne_status ne_paged_attn_f32(const float* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                            const int* cu_new, float* o, float* lse, int64_t q_ld, int B, int N, int Hq, int max_pages,
                            int max_new, void* workspace, size_t workspace_bytes, ne_stream_t stream) {
    return attn_impl(4, q, cache, page_table, seq_lens, cu_new, o, lse, q_ld, B, N, Hq, max_pages, max_new, workspace,
                     workspace_bytes, stream);
}

size_t ne_paged_attn_shared_workspace_size(int B, int N, int Hq, int Hkv, int D) {
    if (B < 0 || N < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (D != 32 && D != 64 && D != 128)) return 0;
    return shared_ws(N, Hq, Hkv, D).total;
}

ne_status ne_paged_attn_shared(const void* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                               const int* cu_new, const int* groups, const int* shared, int R, void* o, float* lse,
                               int64_t q_ld, int B, int N, int Hq, int max_pages, int max_new, void* workspace,
                               size_t workspace_bytes, ne_stream_t stream) {
    return shared_impl(2, q, cache, page_table, seq_lens, cu_new, groups, shared, R, o, lse, q_ld, B, N, Hq, max_pages, max_new,
                       workspace, workspace_bytes, stream);
}

ne_status ne_paged_attn_shared_f32(const float* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                                   const int* cu_new, const int* groups, const int* shared, int R, float* o, float* lse,
                                   int64_t q_ld, int B, int N, int Hq, int max_pages, int max_new, void* workspace,
                                   size_t workspace_bytes, ne_stream_t stream) {
    return shared_impl(4, q, cache, page_table, seq_lens, cu_new, groups, shared, R, o, lse, q_ld, B, N, Hq, max_pages, max_new,
                       workspace, workspace_bytes, stream);
}

size_t ne_paged_weights_workspace_size(void) { return kWeightWs; }

ne_status ne_paged_weights(const void* q, const float* lse, const ne_paged_cache* cache, const int* page_table,
                           const int* seq_lens, const int* cu_new, const float* weights, float* weights_out, int64_t q_ld,
                           int B, int N, int Hq, int max_pages, int max_new, void* workspace, size_t workspace_bytes,
                           ne_stream_t stream) {
    return weights_impl(2, q, lse, cache, page_table, seq_lens, cu_new, weights, weights_out, q_ld, B, N, Hq, max_pages, max_new,
                        workspace, workspace_bytes, stream);
}

ne_status ne_paged_weights_f32(const float* q, const float* lse, const ne_paged_cache* cache, const int* page_table,
                               const int* seq_lens, const int* cu_new, const float* weights, float* weights_out, int64_t q_ld,
                               int B, int N, int Hq, int max_pages, int max_new, void* workspace, size_t workspace_bytes,
                               ne_stream_t stream) {
    return weights_impl(4, q, lse, cache, page_table, seq_lens, cu_new, weights, weights_out, q_ld, B, N, Hq, max_pages, max_new,
                        workspace, workspace_bytes, stream);
}

size_t ne_pages_workspace_size(int n_pages, int n, int max_pages) {
    if (n_pages < 1 || n < 0 || max_pages < 1) return 0;
    return pages_ws(n_pages, n, max_pages).total;
}

ne_status ne_pages_fork(const ne_paged_cache* cache, const int* refcount, const int* page_table, const int* seq_lens,
                        const int* parents, int deep, int* refcount_out, int* child_table, int* child_lens,
                        int* short_out, int B, int C, int max_pages, void* workspace, size_t workspace_bytes,
                        ne_stream_t stream) {
    ne::PagesArgs a;
    clear_error();
    if ((B > 0 && !seq_lens) || (C > 0 && !parents)) return fail(NE_ERR_INVALID_ARG, "null seq_lens or parents");
    ne_status s = pages_args(&a, cache, refcount, page_table, seq_lens, parents, refcount_out, child_table, child_lens,
                             C > 0 ? (size_t)C : 0, short_out, B, max_pages, C, false, workspace, workspace_bytes);
    if (s != NE_OK) return s;
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    a.lens = seq_lens;
    a.other = parents;
    a.deep = deep != 0;
    a.lens_out = child_lens;
    cudaError_t e = ne::launch_pages(ne::PAGES_FORK, a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "pages_fork launch");
    return NE_OK;
}

ne_status ne_pages_resize(const ne_paged_cache* cache, const int* refcount, const int* page_table, const int* seq_lens,
                          const int* new_lens, int* refcount_out, int* table_out, int* short_out, int B, int max_pages,
                          void* workspace, size_t workspace_bytes, ne_stream_t stream) {
    ne::PagesArgs a;
    clear_error();
    if (B > 0 && (!seq_lens || !new_lens)) return fail(NE_ERR_INVALID_ARG, "null seq_lens or new_lens");
    ne_status s = pages_args(&a, cache, refcount, page_table, seq_lens, new_lens, refcount_out, table_out, nullptr, 0,
                             short_out, B, max_pages, B, true, workspace, workspace_bytes);
    if (s != NE_OK) return s;
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    a.lens = seq_lens;
    a.other = new_lens;
    cudaError_t e = ne::launch_pages(ne::PAGES_RESIZE, a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "pages_resize launch");
    return NE_OK;
}

ne_status ne_pages_compact(const ne_paged_cache* cache, const int* refcount, const int* page_table, int* refcount_out,
                           int* table_out, int* remap, int* n_live, int B, int max_pages, void* workspace,
                           size_t workspace_bytes, ne_stream_t stream) {
    ne::PagesArgs a;
    ne_status s = pages_args(&a, cache, refcount, page_table, nullptr, nullptr, refcount_out, table_out, remap,
                             cache && cache->n_pages > 0 ? (size_t)cache->n_pages : 0, n_live, B, max_pages, B, true, workspace,
                             workspace_bytes);
    if (s != NE_OK) return s;
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    a.lens_out = remap;
    cudaError_t e = ne::launch_pages(ne::PAGES_COMPACT, a, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "pages_compact launch");
    return NE_OK;
}

size_t ne_pages_evict_workspace_size(int layers, int B, int Hkv, int T) {
    if (layers < 1 || B < 0 || Hkv < 1 || T < 1 || (long long)layers * B * Hkv >= (1LL << 31)) return 0;
    return evict_ws((size_t)layers * B * Hkv, T).total;
}

ne_status ne_pages_evict(const ne_paged_cache* cache, const float* weights, const int* positions, const int* pos_offset,
                         const int* page_table, const int* seq_lens, const int* new_lens, int sink, int recent,
                         float* weights_out, int* positions_out, int* pos_offset_out, int B, int max_pages, void* workspace,
                         size_t workspace_bytes, ne_stream_t stream) {
    clear_error();
    ne_status s = check_cache(cache, 0, false);
    if (s != NE_OK) return s;
    if (B < 0 || (long long)cache->layers * B * cache->Hkv >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "need B >= 0 and layers * B * Hkv < 2^31 (B=%d)", B);
    if (max_pages < 1 || (long long)max_pages * cache->page_size > (1 << 30) || (long long)B * max_pages >= (1LL << 31))
        return fail(NE_ERR_INVALID_ARG, "need max_pages >= 1, max_pages * page_size <= 2^30 and B * max_pages < 2^31 (max_pages=%d)",
                    max_pages);
    if (sink < 0 || recent < 0 || sink > (1 << 30) || recent > (1 << 30))
        return fail(NE_ERR_INVALID_ARG, "sink and recent must be 0 to 2^30 (sink=%d recent=%d)", sink, recent);
    if (B == 0) return NE_OK;
    const size_t rows = (size_t)cache->layers * B * cache->Hkv, T = (size_t)max_pages * cache->page_size;
    const EvictWs w = evict_ws(rows, T);
    s = check_arrays({{weights, rows * T * 4, "weights", -1}, {positions, rows * T * 4, "positions", -1},
                      {pos_offset, (size_t)B * 4, "pos_offset", -1}, {page_table, (size_t)B * max_pages * 4, "page_table", -1},
                      {seq_lens, (size_t)B * 4, "seq_lens", -1}, {new_lens, (size_t)B * 4, "new_lens", -1}},
                     {{weights_out, rows * T * 4, "weights_out", 0}, {positions_out, rows * T * 4, "positions_out", 1},
                      {pos_offset_out, (size_t)B * 4, "pos_offset_out", 2}, {workspace, w.total, "workspace", -1}});
    if (s == NE_OK) s = check_ptrs({weights, positions, weights_out, positions_out});
    if (s != NE_OK) return s;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(NE_ERR_INVALID_ARG, "workspace must be 256-byte aligned (%zu bytes needed)", w.total);
    if (workspace_bytes < w.total)
        return fail(NE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, w.total);
    if (cache->k == cache->v)
        return fail(NE_ERR_INVALID_ARG, "k and v are one pool: the rows of both are moved, so they must be two");
    ne::EvictArgs a = {};
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    const int e = cache->elem_bytes;
    a.k = static_cast<char*>(cache->k);
    a.v = static_cast<char*>(cache->v);
    a.layers = cache->layers;
    a.n_pages = cache->n_pages;
    a.ps_shift = log2_of(cache->page_size);
    a.Hkv = cache->Hkv;
    a.row_vecs = cache->D * e / 16;
    a.row_shift = log2_of(a.row_vecs);
    a.layer_stride = cache->layers > 1 ? cache->layer_stride * e : 0;
    a.page_stride = cache->n_pages > 1 ? cache->page_stride * e : 0;
    a.tok_stride = cache->tok_stride * e;
    a.head_stride = cache->Hkv > 1 ? cache->head_stride * e : 0;
    a.w = weights;
    a.pos = positions;
    a.off = pos_offset;
    a.table = page_table;
    a.lens = seq_lens;
    a.new_lens = new_lens;
    a.w_out = weights_out;
    a.pos_out = positions_out;
    a.off_out = pos_offset_out;
    a.B = B;
    a.W = max_pages;
    a.T = (int)T;
    a.sink = sink;
    a.recent = recent;
    a.moves = static_cast<int*>(workspace);
    a.list = reinterpret_cast<int*>(static_cast<char*>(workspace) + w.list);
    cudaError_t err = ne::launch_evict(a, (cudaStream_t)stream);
    if (err != cudaSuccess) return cuda_fail(err, "pages_evict launch");
    return NE_OK;
}

}  // extern "C"
