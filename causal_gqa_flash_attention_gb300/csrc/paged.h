// paged.h -- internal interface between api_paged.cu and the paged-cache kernels.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"

namespace ne {

// One layer of the cache as the kernels see it (strides in elements).
struct PagedView {
    const void* k;
    const void* v;
    int n_pages, ps_shift;            // page_size = 1 << ps_shift
    long long page_stride, tok_stride, head_stride;
};

// Row offsets and lengths of a call, as the device reads them.
struct PagedBatch {
    const int* table;                 // [B, W]
    const int* lens;                  // [B]
    const int* cu;                    // [B + 1], or null: one row per sequence
    int B, N, W;
    int cap;                          // W * page_size: the longest length a table row can hold
    // Sequences that share a prefix (the kernels' SHARED form; otherwise unused).
    const int* groups;                // [R + 1]
    const int* shared;                // [R]
    int R, seqs;                      // groups; sequences
    int pre;                          // the line's first `pre` members are the groups' prefixes (R or 0), the others the
                                      // sequences' own positions
    int* err;
};
// Shared positions count in whole steps of this (a multiple of every page and key tile), so that a
// sequence's own positions begin on a page; the rest is read by every sequence for itself.
constexpr int kSharedStep = 256;

struct AppendArgs {
    PagedView c;
    PagedBatch s;
    const void* q;
    const void* k_in;
    const void* v_in;
    void* q_out;
    long long q_ld, k_ld, v_ld, qo_ld;
    int Hq, Hkv, D;
    int rot, layout, pos_offset;      // rot 0: no rotation
    const int* pos_offsets;           // [B], or null: pos_offset for all
    float mscale;
    int wpt_shift;                    // log2 of the warps per token
    int vec_shift;                    // log2 of the 16-byte units of a head
    int* err;
};
struct RopeTurns {
    unsigned long long t[64];
};

// Split of the attention over CTAs (paged_sched.cuh).
struct PagedSplit {
    int C;                            // CTAs of the main kernel
    unsigned long long inv_C;         // 2^64 / C, rounded down
    int tpt;                          // tokens per work unit
    int hg;                           // head groups: Hkv * ceil(G / rows) (rows < G only in the short kernels)
    int gs;                           // query heads of a group
    int bn_shift;                     // log2 of the keys per tile: what a unit may be cut into
    FastDiv div_tpt;                  // by tpt
    int ovh;                          // fixed cost of a unit
    int w_full, w_part;               // cost of a key of a unit with more than `sub` tokens, and with fewer
    int min_shift;                    // log2 of a CTA's least work
    int snap, snap_shift;             // cuts near a unit's end (paged_snap)
    int nocut;                        // units are not cut (short contexts): no join
    int rows;                         // rows of a unit (partials are stored at this pitch)
    int sub;                          // tokens of a unit's first 128-row subtile (0: rows are contiguous)
};

struct PagedAttnArgs {
    PagedView c;
    PagedBatch s;
    PagedSplit p;
    const void* q;
    void* o;
    float* lse;
    long long q_ld;
    int Hq, Hkv, G;
    float scale_log2;                 // log2(e) / sqrt(D)
    float* part_o;                    // [2C, rows, D] unnormalised outputs of cut units
    float2* part_ml;                  // [2C, rows] (running max in log2 units, sum)
    int4* part_info;                  // [2C] (state: 0 none, 1, 2 the unit's last; first row, tokens, head group)
    // SHARED: uncut units' rows, and for every token and head group the CTAs that hold its unit's first
    // and last part (first: | token within the unit << 16 | kHasPrefix; -1, -2: no keys, without, with a prefix).
    // Own positions' at [0], prefixes' at [1].
    float* row_o[2];                  // [N, Hq, D] unnormalised
    float2* row_ml[2];                // [N, Hq]
    int* rec_first[2];                // [N, hg]
    int* rec_last[2];
    int* err;
    unsigned long long timeout_ns;
};

constexpr int kHasPrefix = 1 << 30;

// Dynamic shared memory of a kernel, set once per device (the first 64).
template <typename F>
cudaError_t allow_smem(F kfn, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Which kernel a call runs, and its split.
enum PagedKind : int { PAGED_SHORT16 = 0, PAGED_SHORT32, PAGED_F32_FEW4, PAGED_F32_FEW8, PAGED_F32_FEW16, PAGED_F32_MANY, PAGED_TILES };
PagedKind paged_kind(bool f32, int D, int G, int max_new);
// cap: the longest length the page tables can hold.
PagedSplit paged_split(PagedKind kind, int D, int Hkv, int G, int cap);
// Bytes of the workspace that a split takes.
size_t paged_part_bytes(const PagedSplit& p, int D);

cudaError_t launch_paged_append(bool f32, const AppendArgs& a, const RopeTurns& t, cudaStream_t st);
cudaError_t launch_paged_short(PagedKind kind, int D, const PagedAttnArgs& a, cudaStream_t st);
cudaError_t launch_paged_f32(PagedKind kind, int D, const PagedAttnArgs& a, cudaStream_t st);
cudaError_t launch_paged_tiles(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, cudaStream_t st);
// The same over prefixes or own positions, results as parts (a.s.groups set).
cudaError_t launch_shared_f32(PagedKind kind, int D, const PagedAttnArgs& a, cudaStream_t st);
// terms: bf16 terms of a softmax weight (head_dim 32: 2).
cudaError_t launch_shared_tiles(int D, int terms, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const PagedAttnArgs& a, cudaStream_t st);
// Puts prefixes' and own positions' parts together (one line of both, or two).
cudaError_t launch_shared_join(bool f32, int D, const PagedAttnArgs& pre, const PagedAttnArgs& own, cudaStream_t st);
// Joins the parts of cut units.
cudaError_t launch_paged_join(bool f32, int D, const PagedAttnArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- accumulated weights
constexpr int kWeightCtas = 152;      // shares of the kernels for many rows
constexpr int kWeightKeys = 256;      // keys of a unit at most
struct WeightArgs {
    PagedView c;
    PagedBatch s;                     // cap: entries of a row of weights
    const void* q;
    const float* lse;
    const float* w;                   // [B, Hkv, cap], or null (zeros)
    float* w_out;
    long long q_ld;
    int Hq, Hkv, G;
    float scale_log2;
    int gs, ngrp, sub;                // heads of a query tile, head groups of a kv head, tokens of a query tile
    int ovh;                          // fixed cost of a unit, in tokens
    int key_shift;                    // log2 of its keys
    float* part;                      // [2 kWeightCtas, kWeightKeys] sums of cut units
    int4* part_info;                  // [2 kWeightCtas] (state: 0 none, 1, 2 the unit's last; sequence, kv head, key tile)
    int* err;
    unsigned long long timeout_ns;
};
enum WeightKind : int { WEIGHTS_FEW4 = 0, WEIGHTS_FEW8, WEIGHTS_FEW16, WEIGHTS_FEW32, WEIGHTS_MANY, WEIGHTS_MANY_F32 };
WeightKind weight_kind(bool f32, int G, int max_new);
void weight_split(WeightKind kind, WeightArgs& a);
cudaError_t launch_paged_weights(WeightKind kind, bool f32, int D, const CUtensorMap& tq, const CUtensorMap& tk,
                                 const WeightArgs& a, cudaStream_t st);

// ---------------------------------------------------------------- pages
struct PagesArgs {
    char* k;
    char* v;
    int layers, n_pages, ps, ps_shift, Hkv, row_vecs;   // row_vecs: 16-byte units of one head's slot (a power of two)
    int row_shift;
    long long layer_stride, page_stride, tok_stride, head_stride;   // bytes
    const int* ref;
    const int* table;
    const int* lens;
    const int* other;                 // parents (fork) or new lengths (resize)
    int* ref_out;
    int* table_out;
    int* lens_out;                    // child lengths (fork) or remap (compact)
    int* short_out;                   // pages missing, or n_live (compact)
    int B, W, n, deep, cap;           // n: sequences that take pages
    // workspace
    int* head;                        // [0] copies, [1] pages missing, [2] pages taken
    int2* off;                        // [n] a sequence's first page in free_ids; its copy in list, or -1
    int* free_ids;                    // free pages in ascending order, as many as are taken
    int4* list;                       // copies: (source page or -1, target page, slots, 0)
    int* err;
    int chunks, pieces;               // pieces of a page and pool; of a copy (all layers, both pools)
    FastDiv div_pieces, div_chunks, div_heads, div_w;
};
// Sequences cut by accumulated weight.
struct EvictArgs {
    char* k;
    char* v;
    int layers, n_pages, ps_shift, Hkv, row_vecs, row_shift;   // row_vecs: 16-byte units of a slot of one head
    long long layer_stride, page_stride, tok_stride, head_stride;   // bytes
    const float* w;                   // [layers, B, Hkv, T]
    const int* pos;
    const int* off;                   // [B]
    const int* table;
    const int* lens;
    const int* new_lens;
    float* w_out;
    int* pos_out;
    int* off_out;
    int B, W, T, sink, recent;
    // workspace
    int* moves;                       // [layers, B, Hkv]
    int* list;                        // [layers, B, Hkv, T]: T / 2 targets, T / 2 sources
    int* err;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st);

enum PagesOp : int { PAGES_FORK = 0, PAGES_RESIZE, PAGES_COMPACT };
cudaError_t launch_pages(PagesOp op, const PagesArgs& a, cudaStream_t st);

}  // namespace ne
