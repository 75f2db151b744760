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
};

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
    int* err;
    unsigned long long timeout_ns;
};

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
// Joins the parts of cut units.
cudaError_t launch_paged_join(bool f32, int D, const PagedAttnArgs& a, cudaStream_t st);

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
enum PagesOp : int { PAGES_FORK = 0, PAGES_RESIZE, PAGES_COMPACT };
cudaError_t launch_pages(PagesOp op, const PagesArgs& a, cudaStream_t st);

}  // namespace ne
