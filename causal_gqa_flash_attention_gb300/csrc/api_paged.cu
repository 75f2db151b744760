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
                      const int* lens, const int* cu, const ne_rope_spec* spec, int pos_offset, void* q_out, int64_t q_ld,
                      int64_t k_ld, int64_t v_ld, int64_t qo_ld, int B, int N, int Hq, int W, ne_stream_t stream) {
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
    ne::RopeTurns turns = {};
    if (spec)
        for (int i = 0; i < spec->rot_dim / 2; ++i) turns.t[i] = spec->turns[i];
    cudaError_t e = ne::launch_paged_append(eb == 4, a, turns, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "paged_append launch");
    return NE_OK;
}

// Tensor maps of the tile kernel: a query box is (64 columns, G heads, `sub` tokens), a
// key or value box (64 columns, one head, the rows of a page that fall into one tile).
ne_status tile_maps(CUtensorMap* tq, CUtensorMap* tk, CUtensorMap* tv, const ne_paged_cache* c, const ne::PagedAttnArgs& a) {
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
    const cuuint64_t qd[3] = {(cuuint64_t)c->D, (cuuint64_t)a.Hq, (cuuint64_t)a.s.N};
    const cuuint64_t qs[2] = {(cuuint64_t)c->D * 2, (cuuint64_t)a.q_ld * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)a.G, (cuuint32_t)a.p.sub};
    if ((s = encode(tq, a.q, 3, qd, qs, qb)) != NE_OK) return s;
    const cuuint64_t kd[4] = {(cuuint64_t)c->D, (cuuint64_t)c->Hkv, (cuuint64_t)c->page_size, (cuuint64_t)c->n_pages};
    const cuuint64_t ks[3] = {(cuuint64_t)a.c.head_stride * 2, (cuuint64_t)a.c.tok_stride * 2, (cuuint64_t)a.c.page_stride * 2};
    const cuuint32_t kb[4] = {64, 1, (cuuint32_t)std::min(c->page_size, 128), 1};
    if ((s = encode(tk, a.c.k, 4, kd, ks, kb)) != NE_OK) return s;
    return encode(tv, a.c.v, 4, kd, ks, kb);
}

// Bytes of a call's workspace: the largest over the kernels that its head_dim and heads may run.
size_t attn_ws_bytes(int D, int Hkv, int G) {
    size_t most = 0;
    for (int f32 = 0; f32 < 2; ++f32)
        for (int rows : {1, 2, 4, 5, 8, 9, 16, 17, 32, 33, 1 << 20}) {
            if (f32 && D > 64) continue;
            const ne::PagedKind kind = ne::paged_kind(f32 != 0, D, G, rows);
            most = std::max(most, ne::paged_part_bytes(ne::paged_split(kind, D, Hkv, G, 1 << 30), D));
        }
    return round_up(most, 256);
}

ne_status attn_impl(int eb, const void* q, const ne_paged_cache* c, const int* table, const int* lens, const int* cu,
                    void* o, float* lse, int64_t q_ld, int B, int N, int Hq, int W, int max_new, void* ws,
                    size_t ws_bytes, ne_stream_t stream) {
    clear_error();
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
    const int G = Hq / c->Hkv;
    const size_t need = attn_ws_bytes(c->D, c->Hkv, G);
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return fail(NE_ERR_INVALID_ARG, "workspace must be non-null and 256-byte aligned (%zu bytes needed)", need);
    if (ws_bytes < need)
        return fail(NE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", ws_bytes, need);
    ne::PagedAttnArgs a = {};
    if ((s = ready((cudaStream_t)stream, &a.err)) != NE_OK) return s;
    const bool f32 = eb == 4;
    const ne::PagedKind kind = ne::paged_kind(f32, c->D, G, cu ? std::min(max_new, N) : 1);
    a.c = view_of(c);
    a.s = batch_of(c, table, lens, cu, B, N, W);
    a.p = ne::paged_split(kind, c->D, c->Hkv, G, a.s.cap);
    a.q = q;
    a.o = o;
    a.lse = lse;
    a.q_ld = q_ld;
    a.Hq = Hq;
    a.Hkv = c->Hkv;
    a.G = G;
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->D));
    const size_t parts = 2 * (size_t)a.p.C;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + parts * a.p.rows * c->D);
    a.part_info = reinterpret_cast<int4*>(a.part_ml + parts * a.p.rows);
    a.timeout_ns = timeout_ns();
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (kind == ne::PAGED_TILES) {
        CUtensorMap tq, tk, tv;
        if ((s = tile_maps(&tq, &tk, &tv, c, a)) != NE_OK) return s;
        e = ne::launch_paged_tiles(c->D, tq, tk, tv, a, st);
    } else if (f32) e = ne::launch_paged_f32(kind, c->D, a, st);
    else e = ne::launch_paged_short(kind, c->D, a, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged_attn launch");
    if (a.p.nocut) return NE_OK;
    e = ne::launch_paged_join(f32, c->D, a, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged_attn join launch");
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
    return append_impl(2, q, k, v, cache, page_table, seq_lens, cu_new, spec, pos_offset, q_out, q_ld, k_ld, v_ld, q_out_ld,
                       B, N, Hq, max_pages, stream);
}

ne_status ne_paged_append_f32(const float* q, const float* k, const float* v, const ne_paged_cache* cache,
                              const int* page_table, const int* seq_lens, const int* cu_new, const ne_rope_spec* spec,
                              int pos_offset, float* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t q_out_ld,
                              int B, int N, int Hq, int max_pages, ne_stream_t stream) {
    return append_impl(4, q, k, v, cache, page_table, seq_lens, cu_new, spec, pos_offset, q_out, q_ld, k_ld, v_ld, q_out_ld,
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

}  // extern "C"
