/*
 * neattn.h -- C ABI of libneattn: fused causal grouped-query self-attention with
 * rotary position embeddings (RoPE), forward and backward, on sm_103a tensor cores.
 *
 * What is computed (page title, section):
 *   - causal self-attention, each position attending to itself and earlier
 *     positions ("Tiny hackable CUDA language model implementation", Core Mechanics,
 *     causal self-attention bullet);
 *   - grouped-query attention: Hkv key/value heads, each shared by G = Hq / Hkv
 *     query heads; query head h reads key/value head h / G ("NanoEuler: C와 CUDA로
 *     밑바닥부터 구축한 GPT-2 규모의 LLM", 기술 사양, GQA bullet, and 모델 구성);
 *   - RoPE on queries and keys (same page, 기술 사양, RoPE bullet): adjacent pairs
 *     (2i, 2i+1) of a row at position t are rotated by the angle t * theta^(-2i/D),
 *     (x0, x1) -> (x0 cos - x1 sin, x0 sin + x1 cos), positions t = 0 .. T-1;
 *   - FlashAttention-style tiling with an online softmax, so the T x T score matrix
 *     is never stored (same page, 커널 구현);
 *   - the hand-written backward pass (same page, 검증 및 안정성).
 *   O = softmax(s * Q' K'^T + causal mask) V with s = 1/sqrt(D), Q' = R Q, K' = R K.
 *   LSE[b,h,t] = natural log of sum_j exp(s * q'_t . k'_j) over j <= t.
 *
 * Layouts (all row-major, dense, no padding):
 *   q, o, dO, dq : [B, T, Hq,  D]      k, v, dk, dv : [B, T, Hkv, D]
 *   lse          : [B, Hq, T] fp32     rope tables  : [T, D/2] fp32
 * The bf16 entry points take __nv_bfloat16 tensors and compute with bf16 tensor-core
 * inputs and fp32 accumulation; the *_f32 entry points take fp32 tensors and use TF32
 * tensor cores with fp32 accumulation.  Outputs have the input dtype, lse is fp32.
 *
 * Supported shapes: B >= 0, T >= 0 (any T, ragged tails included), Hq % Hkv == 0,
 * D in {32, 64, 128} for bf16 and {32, 64} for f32 (others return NE_ERR_UNSUPPORTED;
 * bf16 32 runs on the head_dim-64 kernels with zero-padded columns; fp32 128 does not
 * fit the kernels' shared memory: a 128-row fp32 tile of 128 columns is 64 KB),
 * B * T * max(Hq, 1) * D < 2^31.  Every tensor pointer must be 16-byte aligned.
 *
 * Ownership: the caller owns every tensor and the backward workspace.  The library
 * owns only small per-device caches (RoPE tables per (D, theta), one device error
 * word), created on first use and released by ne_shutdown().  A table serves every T up
 * to its length; a call with a longer T builds one of twice the length (or T's), and the
 * shorter table is kept until ne_shutdown() (kernels in flight may still read it), so a
 * caller whose T grows step by step (a growing KV cache) holds at most about twice the
 * largest table (T * D/2 * 8 bytes).  All pointers are device
 * pointers unless stated otherwise.
 *
 * Streams: every call enqueues its kernels on `stream` (NULL = legacy default stream)
 * and returns without synchronising, except that a call that needs a new or longer RoPE
 * table for its (device, D, theta) builds it and synchronises `stream` once; make such
 * a call (the longest T) before any stream capture.  Argument errors return before anything
 * is enqueued.  Device-side failures (a bounded wait inside a kernel that ran out,
 * see ne_get_device_error) are reported asynchronously.
 *
 * Threading: calls are thread-safe; ne_last_error() is per thread.
 */
#ifndef NEATTN_H
#define NEATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t / CUstream. */
typedef struct CUstream_st* ne_stream_t;

typedef enum {
    NE_OK = 0,
    NE_ERR_INVALID_ARG = 1,     /* bad pointer, shape or size; nothing was enqueued */
    NE_ERR_UNSUPPORTED = 2,     /* valid but not implemented (e.g. head_dim) */
    NE_ERR_CUDA = 3,            /* a CUDA runtime/driver call failed; see ne_last_error() */
    NE_ERR_DEVICE_TIMEOUT = 4,  /* a kernel's bounded wait ran out (ne_get_device_error) */
    NE_ERR_NO_DEVICE = 5        /* no CUDA device, or not an sm_103 device */
} ne_status;

/* RoPE cos/sin table (the rotation of the RoPE bullet, same page): for t < T and
 * i < D/2, cos_out[t*(D/2)+i] = cos(t * theta^(-2i/D)) and likewise sin_out.  Angles
 * are formed in fp64 on the device and stored as fp32.  cos_out/sin_out: device
 * pointers to T*D/2 floats each.  D must be even and > 0, theta > 0. */
ne_status ne_rope_table(float* cos_out, float* sin_out, int T, int D, double theta,
                        ne_stream_t stream);

/* Forward (커널 구현: tiling + online softmax).  q [B,T,Hq,D], k and v [B,T,Hkv,D] in,
 * o [B,T,Hq,D] and lse [B,Hq,T] (fp32) out.  bf16 tensors. */
ne_status ne_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                      int B, int T, int Hq, int Hkv, int D, double rope_theta,
                      ne_stream_t stream);
/* Same with fp32 tensors on TF32 tensor cores. */
ne_status ne_attn_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse,
                          int B, int T, int Hq, int Hkv, int D, double rope_theta,
                          ne_stream_t stream);

/* Bytes of device workspace ne_attn_bwd needs for this shape (0 on a bad shape).
 * Layout: Delta fp32 [B,Hq,T] at offset 0, then (256-byte aligned) the fp32 dQ
 * accumulator [B,T,Hq,D], then (256-byte aligned) the rotated queries R Q as fp16
 * [B,T,Hq,D] (used by the bf16 head_dim-64 kernel).  All are rewritten by every call. */
size_t ne_attn_bwd_workspace_size(int B, int T, int Hq, int Hkv, int D);

/* Backward (검증 및 안정성: the hand-written backward), the vector-Jacobian product of
 * <dO, O> for the forward above.  Inputs q, k, v, o, lse, dO as the forward wrote or
 * read them; outputs dq [B,T,Hq,D], dk and dv [B,T,Hkv,D] in the input dtype.  The
 * gradient of every kv head is summed over its G query heads.  `workspace` must hold
 * ne_attn_bwd_workspace_size() bytes (256-byte aligned); it is caller-owned scratch. */
ne_status ne_attn_bwd(const void* q, const void* k, const void* v, const void* o,
                      const float* lse, const void* dO, void* dq, void* dk, void* dv,
                      int B, int T, int Hq, int Hkv, int D, double rope_theta,
                      void* workspace, size_t workspace_bytes, ne_stream_t stream);
ne_status ne_attn_bwd_f32(const float* q, const float* k, const float* v, const float* o,
                          const float* lse, const float* dO, float* dq, float* dk, float* dv,
                          int B, int T, int Hq, int Hkv, int D, double rope_theta,
                          void* workspace, size_t workspace_bytes, ne_stream_t stream);

/* Training pair: the forward and backward of one layer sharing that layer's backward
 * workspace (the pages train with the forward and backward kernels of 커널 구현 and
 * 검증 및 안정성, same page).  ne_attn_fwd_train computes what ne_attn_fwd computes and,
 * for bf16 head_dim 32 and 64, also fills the workspace for the later backward: the
 * rotated queries R Q as fp16 and a zeroed fp32 dQ accumulator (the forward rotates the
 * queries anyway, and its HBM is mostly idle).  ne_attn_bwd_train then computes what
 * ne_attn_bwd computes while skipping that work, so its preprocess pass only forms Delta.
 * Same arguments as ne_attn_fwd / ne_attn_bwd plus the workspace (as for ne_attn_bwd:
 * ne_attn_bwd_workspace_size() bytes, 256-byte aligned, caller-owned).  Contract: the
 * backward must get the same workspace, the same q, k, v, shape and theta, and nothing
 * may write the workspace between the two calls (one workspace per layer in flight).
 * For f32 tensors and head_dim 128 the pair is exactly ne_attn_fwd + ne_attn_bwd (the
 * forward leaves the workspace alone and the backward fills it itself). */
ne_status ne_attn_fwd_train(const void* q, const void* k, const void* v, void* o, float* lse,
                            void* workspace, size_t workspace_bytes, int B, int T, int Hq, int Hkv, int D,
                            double rope_theta, ne_stream_t stream);
ne_status ne_attn_fwd_train_f32(const float* q, const float* k, const float* v, float* o, float* lse,
                                void* workspace, size_t workspace_bytes, int B, int T, int Hq, int Hkv,
                                int D, double rope_theta, ne_stream_t stream);
ne_status ne_attn_bwd_train(const void* q, const void* k, const void* v, const void* o,
                            const float* lse, const void* dO, void* dq, void* dk, void* dv,
                            int B, int T, int Hq, int Hkv, int D, double rope_theta,
                            void* workspace, size_t workspace_bytes, ne_stream_t stream);
ne_status ne_attn_bwd_train_f32(const float* q, const float* k, const float* v, const float* o,
                                const float* lse, const float* dO, float* dq, float* dk, float* dv,
                                int B, int T, int Hq, int Hkv, int D, double rope_theta,
                                void* workspace, size_t workspace_bytes, ne_stream_t stream);

/* Variable-length sequences in a padded batch: the supervised fine-tuning data of
 * "NanoEuler: C와 CUDA로 밑바닥부터 구축한 GPT-2 규모의 LLM" (2단계 학습 프로세스, SFT bullet)
 * pads sequences of different lengths to one T, and the padding must not take part.
 * Same tensors and layouts as ne_attn_fwd / ne_attn_bwd, plus
 *   seq_lens [B] int32 (device memory, 4-byte aligned): sequence b occupies positions
 *            0 .. seq_lens[b]-1 of row b; positions seq_lens[b] .. T-1 are padding.
 * The valid positions of sequence b get the results of the same call on that sequence
 * alone with T = seq_lens[b] (RoPE positions start at 0 in every row).
 * Padding never takes part: no valid query attends to a padding key, padding queries
 * and keys get zero outputs and gradients (o, dq, dk, dv = 0) and lse = -inf (the log of
 * an empty sum).  Padding entries of q and k are not read as values (the kernels zero
 * them before any MMA); padding entries of v and dO must be finite (e.g. zeros, as
 * padding usually is): they meet zero weights inside tensor-core products, where a NaN
 * or infinity would still propagate.  A length outside [0, T] is clamped on the device
 * and reported by ne_get_device_error() as NE_ERR_INVALID_ARG; a length of 0 is an
 * empty sequence.  The backward takes the workspace of ne_attn_bwd. */
ne_status ne_attn_fwd_varlen(const void* q, const void* k, const void* v, const int* seq_lens, void* o,
                             float* lse, int B, int T, int Hq, int Hkv, int D, double rope_theta,
                             ne_stream_t stream);
ne_status ne_attn_fwd_varlen_f32(const float* q, const float* k, const float* v, const int* seq_lens,
                                 float* o, float* lse, int B, int T, int Hq, int Hkv, int D,
                                 double rope_theta, ne_stream_t stream);
ne_status ne_attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o,
                             const float* lse, const void* dO, const int* seq_lens, void* dq, void* dk,
                             void* dv, int B, int T, int Hq, int Hkv, int D, double rope_theta,
                             void* workspace, size_t workspace_bytes, ne_stream_t stream);
ne_status ne_attn_bwd_varlen_f32(const float* q, const float* k, const float* v, const float* o,
                                 const float* lse, const float* dO, const int* seq_lens, float* dq,
                                 float* dk, float* dv, int B, int T, int Hq, int Hkv, int D,
                                 double rope_theta, void* workspace, size_t workspace_bytes,
                                 ne_stream_t stream);

/* Backward that allocates nothing (there is no counterpart of this call on the
 * pages: it is a deployment convenience).  Same computation, arguments and outputs
 * as ne_attn_bwd for bf16 tensors, but without a workspace argument: its scratch
 * (RoPE table, Delta, fp32 dQ accumulator, rotated queries) lives in one file-scope
 * device array of 48 MiB that every GPU loading the library keeps until the process exits.  It is for
 * callers that cannot call cudaMalloc at this point: code that runs while a stream
 * is being captured into a CUDA graph (allocation is not allowed there), runtimes
 * whose own allocator already owns the device's free memory, or real-time loops that
 * forbid allocation after start-up.  It calls no cudaMalloc, cudaFree or allocating
 * library routine.
 *  - Limit: round256(max(T,64)*P*8) + round256(B*Hq*T*4) + round256(B*T*Hq*D*4)
 *    + (D <= 64 ? B*T*Hq*D*2 : 0) <= 50331648 bytes, P = max(D,64)/2 (the GPU-pipeline shape B=16 T=512
 *    Hq=12 D=64 uses 38.3 MB); larger shapes
 *    return NE_ERR_INVALID_ARG before anything is enqueued.
 *  - The first call on a device looks up the array's device address (once per
 *    device, with that device current); make that first call before any stream
 *    capture.
 *  - All calls share the one array, which keeps the last call's contents; every call
 *    rewrites what it reads.  Calls whose kernels overlap on the GPU (two streams, or
 *    two threads) race on the scratch and produce wrong gradients: serialise them.
 *  - Device-side errors (a bounded wait that ran out, or an MMA operand beyond the
 *    fp16 range: a rotated q or k, or dS) are recorded in a second file-scope device
 *    word beside the scratch, not in the allocated word ne_get_device_error() reads;
 *    read them with ne_noalloc_get_device_error(). */
ne_status ne_attn_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, const void* dO, void* dq, void* dk, void* dv,
                              int B, int T, int Hq, int Hkv, int D, double rope_theta,
                              ne_stream_t stream);
/* The error report of the allocation-free calls (no counterpart on the pages).
 * Synchronises `stream`, then reads and clears the current device's static error word
 * of ne_attn_bwd_noalloc; allocates nothing.  Returns NE_ERR_INVALID_ARG when an MMA
 * operand left the fp16 range (the outputs of that call are invalid),
 * NE_ERR_DEVICE_TIMEOUT when a bounded wait ran out, NE_ERR_CUDA when the
 * synchronisation failed, else NE_OK.  Like the scratch, the word is shared by all
 * calls on a device. */
ne_status ne_noalloc_get_device_error(ne_stream_t stream);

/* Decode step over a key/value cache: the newest token of every sequence attends to
 * all cached positions of its sequence.  For sequence b with len = seq_lens[b] the
 * newest token sits at position len - 1, and the result is row len - 1 of the causal
 * attention above over positions 0 .. len - 1: the same RoPE, grouped heads, scale and
 * LSE convention.  The CUDA engine of "NanoEuler: C와 CUDA로 밑바닥부터 구축한 GPT-2 규모의
 * LLM" (CUDA 엔진 및 성능) runs inference as well as training, and its chat command
 * generates token by token ("NanoEuler – 순수 C/CUDA로 처음부터 만든 GPT-2 규모 언어
 * 모델", Code Example).
 *   q        [B, Hq, D]        query rows of the newest tokens, unrotated (in)
 *   k_cache  [B, T_max, Hkv, D] keys, unrotated, positions 0 .. len-1 valid; the newest
 *                              token's key must already be written at len - 1 (in)
 *   v_cache  [B, T_max, Hkv, D] values, same positions (in)
 *   seq_lens [B] int32         1 <= len <= T_max (device memory, 4-byte aligned) (in)
 *   o        [B, Hq, D]        output rows, input dtype (out)
 *   lse      [B, Hq] fp32      natural log of the softmax denominator (out)
 * Rows at positions >= len are never read.  `workspace` holds
 * ne_attn_decode_workspace_size() bytes (256-byte aligned, caller-owned, rewritten by
 * every call); it may be NULL when that size is 0.  A seq_lens entry outside
 * [1, T_max] is clamped on the device and reported by ne_get_device_error() as
 * NE_ERR_INVALID_ARG; that sequence's outputs are then invalid.
 * Supported: D in {64, 128} (bf16) or {32, 64} (f32), Hq % Hkv == 0, 1 <= B <= 65535,
 * 1 <= T_max <= 2^30; B == 0 is a no-op.  Arithmetic is fp32 throughout (no tensor cores: one
 * query row per head is a matrix-vector product, bound by the read of the cache). */
size_t ne_attn_decode_workspace_size(int B, int T_max, int Hq, int Hkv, int D);
ne_status ne_attn_decode(const void* q, const void* k_cache, const void* v_cache,
                         const int* seq_lens, void* o, float* lse, int B, int T_max, int Hq,
                         int Hkv, int D, double rope_theta, void* workspace,
                         size_t workspace_bytes, ne_stream_t stream);
ne_status ne_attn_decode_f32(const float* q, const float* k_cache, const float* v_cache,
                             const int* seq_lens, float* o, float* lse, int B, int T_max,
                             int Hq, int Hkv, int D, double rope_theta, void* workspace,
                             size_t workspace_bytes, ne_stream_t stream);

/* The steps before attention in every layer, fused into one tensor-core GEMM ("NanoEuler:
 * C와 CUDA로 밑바닥부터 구축한 GPT-2 규모의 LLM", 기술 사양: RMSNorm as pre-normalization
 * without bias, RoPE on queries and keys; the model has no biases): for token row m of x,
 *   r_m = sqrt(mean_c x_mc^2 + eps),   y_m = W (x_m o gamma) / r_m,
 * split into query heads (rows 0 .. Hq*D-1 of W), key heads (next Hkv*D rows) and value
 * heads (last Hkv*D rows).  With rotate != 0 the query and key heads are rotated by the
 * RoPE of the attention calls (position m mod T, theta rope_theta); the attention calls
 * take unrotated q and k (they rotate as their tiles load), so the form they consume is
 * rotate = 0.
 *   x     [B, T, dim] bf16 (in)          gamma [dim] bf16 (in)
 *   w     [(Hq + 2 Hkv) * D, dim] bf16, row-major (in: row n holds output feature n)
 *   q     [B, T, Hq, D] bf16 (out)       k, v  [B, T, Hkv, D] bf16 (out)
 *   workspace: caller-owned device scratch of ne_qkv_prologue_workspace_size(B, T, dim,
 *              Hq, Hkv, D) bytes, 256-byte aligned; each call rewrites it with
 *              W diag(gamma) (bf16) and the reciprocal root-mean-square of every token row
 *              (fp32), formed by two small passes before the GEMM.
 * Arithmetic: bf16 tensor-core products with fp32 accumulation; the gain is folded into
 * the weights (W diag(gamma), rounded to bf16, formed on the device by each call), the
 * root-mean-square is fp32.  Supported: D in {32, 64, 128}, dim a multiple of 8,
 * Hq % Hkv == 0, B*T*dim and B*T*(Hq + 2 Hkv)*D below 2^31, eps >= 0.  Pointers 16-byte
 * aligned.  A call that needs a new or longer RoPE table builds it and synchronises
 * `stream` once (as the attention calls do). */
size_t ne_qkv_prologue_workspace_size(int B, int T, int dim, int Hq, int Hkv, int D);
ne_status ne_qkv_prologue(const void* x, const void* gamma, const void* w, void* q, void* k, void* v,
                          int B, int T, int dim, int Hq, int Hkv, int D, double eps,
                          double rope_theta, int rotate, void* workspace, size_t workspace_bytes,
                          ne_stream_t stream);

/* ------------------------------------------------------------------ paged cache
 * A key/value cache in pages of `page_size` positions, for generation over many sequences
 * of different and growing lengths (generation: "NanoEuler – 순수 C/CUDA로 처음부터 만든
 * GPT-2 규모 언어 모델", Code Example; the pages describe no paged cache: its design is this
 * library's).  Position p of sequence b lies in slot p % page_size of page
 * page_table[b][p / page_size].  Keys are stored ROTATED (ne_paged_append rotates them
 * once; the contiguous cache of ne_attn_decode holds them unrotated), so attention over
 * pages rotates nothing and its queries come rotated from ne_paged_append too.
 *
 * One pool of keys and one of values, over `layers` layers that share the page tables:
 * element d of head h in slot t of page p of layer l lies at
 *   l * layer_stride + p * page_stride + t * tok_stride + h * head_stride + d   (elements).
 * The strides cover [layers, pages, page_size, Hkv, D] as well as head-major pages and
 * pools with keys and values side by side.  ne_paged_append and ne_paged_attn work on one
 * layer (layers = 1, k and v pointing at it); the ne_pages_* calls move page contents of
 * every layer at once.
 * Supported: page_size a power of two from 8 to 256; D in {32, 64, 128} for bf16
 * (elem_bytes 2) and {32, 64} for f32 (elem_bytes 4); k, v 16-byte aligned and strides
 * multiples of 16 bytes, below 2^39 elements, the strides of an extent above 1 at least D; n_pages < 2^24, layers <= 4096,
 * Hkv <= 1024. */
typedef struct {
    void* k;
    void* v;
    int elem_bytes;             /* 2 (bf16) or 4 (f32) */
    int layers, n_pages, page_size, Hkv, D;
    int64_t layer_stride, page_stride, tok_stride, head_stride;
} ne_paged_cache;

/* Rotary positions as a value (host struct; ne_rope_spec_init fills it, the caller keeps
 * it).  Pair i < rot_dim / 2 of a row at position p is rotated by the angle p * f_i; the
 * elements from rot_dim on pass through.  layout 0: pairs (2i, 2i+1), the attention calls'
 * convention; layout 1: pairs (i, i + rot_dim/2).  f_i = theta^(-2i/rot_dim), changed by
 *   NE_ROPE_NONE   nothing;
 *   NE_ROPE_LINEAR f_i / factor (positions interpolated);
 *   NE_ROPE_BASE   theta replaced by theta * factor^(rot_dim / (rot_dim - 2));
 *   NE_ROPE_PARTS  f_i (g + (1 - g) / factor), g = clamp((n_i - beta_slow) / (beta_fast -
 *                  beta_slow), 0, 1), n_i = orig_len * f_i / (2 pi) the turns of the pair over
 *                  the trained context: fast pairs keep their angle, slow ones interpolate.
 * cos and sin are multiplied by mscale.  The angle is kept as a 64-bit fraction of a turn
 * (turns[i] = f_i / (2 pi) * 2^64), so p * turns[i] mod 2^64 is exact for every position:
 * far positions lose nothing and no table is built.  Refused: parameters that leave an angle
 * (or the scaled theta) infinite or no number, and an mscale beyond fp32. */
enum { NE_ROPE_NONE = 0, NE_ROPE_LINEAR = 1, NE_ROPE_BASE = 2, NE_ROPE_PARTS = 3 };
typedef struct {
    int D, rot_dim, layout;
    float mscale;
    uint64_t turns[64];
} ne_rope_spec;
ne_status ne_rope_spec_init(ne_rope_spec* out, int D, int rot_dim, int layout, double theta, int scaling,
                            double factor, int orig_len, double beta_fast, double beta_slow, double mscale);

/* New tokens into the cache: the rows of sequence b are cu_new[b] .. cu_new[b+1]-1 of the
 * packed inputs, n_b of them, and take positions seq_lens[b] - n_b .. seq_lens[b] - 1
 * (seq_lens counts them already).  k rows are rotated (spec at position + pos_offset; a null spec stores
 * them as they are) and stored, v rows are stored; with q, the query rows are rotated into
 * q_out (which may be q itself, with the same row stride).
 *   k, v  [N, Hkv, D] rows k_ld, v_ld elements apart;  q [N, Hq, D] rows q_ld apart
 *   q_out [N, Hq, D] rows q_out_ld apart (both or neither of q, q_out; Hq ignored without)
 *   page_table [B, max_pages] int32, seq_lens [B] int32, cu_new [B+1] int32 or NULL
 *   (one row per sequence, N == B); device memory, 4-byte aligned.
 *   pos_offset: added to every position for the rotation alone (a cache that dropped its
 *   first pages); 0 <= pos_offset < 2^30.
 * Rows outside [cu_new[0], cu_new[B]) have no effect and are not written.  A row whose position
 * is negative (n_b > seq_lens[b]) is not stored and gets q_out = 0.  Bad device-side
 * arguments never reach memory: a cu_new entry outside [0, N] or decreasing, a length
 * outside [0, max_pages * page_size], a page id outside [0, n_pages) are clamped or skipped
 * and reported by ne_get_device_error() as NE_ERR_INVALID_ARG.  No two rows may name one
 * slot (a page to be written belongs to one sequence; ne_pages_fork sees to it).
 * Row strides are multiples of 16 bytes.  N * max(Hq, Hkv) * D < 2^31. */
ne_status ne_paged_append(const void* q, const void* k, const void* v, const ne_paged_cache* cache,
                          const int* page_table, const int* seq_lens, const int* cu_new,
                          const ne_rope_spec* spec, int pos_offset, void* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                          int64_t q_out_ld, int B, int N, int Hq, int max_pages, ne_stream_t stream);
ne_status ne_paged_append_f32(const float* q, const float* k, const float* v, const ne_paged_cache* cache,
                              const int* page_table, const int* seq_lens, const int* cu_new,
                              const ne_rope_spec* spec, int pos_offset, float* q_out, int64_t q_ld, int64_t k_ld, int64_t v_ld,
                              int64_t q_out_ld, int B, int N, int Hq, int max_pages, ne_stream_t stream);

/* The same with an offset per sequence: row i of sequence b is rotated at its slot's position plus
 * pos_offsets[b] (int32 [B], device memory; 0 <= pos_offsets[b] < 2^30, clamped and reported otherwise),
 * for sequences that ne_pages_evict has cut. */
ne_status ne_paged_append_at(const void* q, const void* k, const void* v, const ne_paged_cache* cache,
                             const int* page_table, const int* seq_lens, const int* cu_new,
                             const ne_rope_spec* spec, const int* pos_offsets, void* q_out, int64_t q_ld, int64_t k_ld,
                             int64_t v_ld, int64_t q_out_ld, int B, int N, int Hq, int max_pages, ne_stream_t stream);
ne_status ne_paged_append_at_f32(const float* q, const float* k, const float* v, const ne_paged_cache* cache,
                                 const int* page_table, const int* seq_lens, const int* cu_new,
                                 const ne_rope_spec* spec, const int* pos_offsets, float* q_out, int64_t q_ld,
                                 int64_t k_ld, int64_t v_ld, int64_t q_out_ld, int B, int N, int Hq, int max_pages,
                                 ne_stream_t stream);

/* Attention of the new tokens over the pages: row i of sequence b (packed as above), at
 * position seq_lens[b] - n_b + i, attends to the cached positions up to its own.  n_b = 1 is
 * a generation step, n_b = seq_lens[b] a whole prompt, anything between a chunk; one call
 * mixes them.
 *   q   [N, Hq, D] rotated, rows q_ld elements apart (in)
 *   o   [N, Hq, D] dense (out)        lse [N, Hq] fp32, natural log (out)
 * Rows outside [cu_new[0], cu_new[B]) stay as they were.  A row with nothing to attend to
 * (a negative position) gets o = 0 and lse = -inf.  Slots at or behind a sequence's length
 * may hold anything (NaN included); values in front of it must be finite.
 * max_new: the largest n_b as far as the caller knows (N if not).  It chooses between
 * kernels (a few rows per kv head stream the cache through registers; more use tcgen05
 * tiles) and changes no result beyond rounding: any n_b is right with any max_new >= 1.
 * bf16: tensor-core products of bf16 inputs with fp32 accumulation and fp32 softmax
 * statistics.  The weights of the product with V are rounded: the kernels for a few rows (max_new
 * times Hq / Hkv up to 32; any max_new at D 32 or above 128 heads per kv head) keep two bf16 terms
 * of each, off by at most 2^-16 of it, the tcgen05 tiles one, 2^-8, as the training forward does;
 * so o is off by that much of sum p |v| beside its own rounding.  f32: fp32 throughout (no TF32).  Work is split over the key axis by counted
 * work, so results depend on the shape, lengths and device but never on timing: the same
 * call gives the same bits.  o and lse overlap neither q nor each other.  workspace:
 * ne_paged_attn_workspace_size() bytes (5 to 41 MB by D and Hq / Hkv, whatever B and N), 256-byte
 * aligned, caller-owned, rewritten by every call (two calls that may overlap need two).
 * Device-side arguments are checked as in ne_paged_append; a bad page id reads as zeros.
 * In a bf16 chunk a part may wait for as long as a pass of 256 rows over its keys takes, about 1.5
 * us per 128: beyond some 1.5e8 positions raise the limit of the waits (ne_set_wait_timeout_ms), or
 * the call ends with NE_ERR_DEVICE_TIMEOUT. */
size_t ne_paged_attn_workspace_size(int B, int N, int Hq, int Hkv, int D);
ne_status ne_paged_attn(const void* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                        const int* cu_new, void* o, float* lse, int64_t q_ld, int B, int N, int Hq,
                        int max_pages, int max_new, void* workspace, size_t workspace_bytes, ne_stream_t stream);
ne_status ne_paged_attn_f32(const float* q, const ne_paged_cache* cache, const int* page_table,
                            const int* seq_lens, const int* cu_new, float* o, float* lse, int64_t q_ld, int B,
                            int N, int Hq, int max_pages, int max_new, void* workspace, size_t workspace_bytes,
                            ne_stream_t stream);

/* Attention of sequences that share their first positions (children of one ne_pages_fork, questions
 * about one document): the result of ne_paged_attn, with the shared keys and values read and multiplied once for
 * all rows of a group.
 *   groups [R + 1] int32: group r is sequences groups[r] .. groups[r+1]-1 of the batch (ascending; sequences
 *          in front of groups[0] and from groups[R] on share nothing); 0 <= R <= B
 *   shared [R] int32: the first shared[r] positions hold the same in every sequence of group r (whether
 *          or not in the same pages), all in front of its new tokens: shared[r] <= seq_lens[b] - n_b
 * Both device memory, 4-byte aligned.  They are read through the group's first sequence, up to its length (what
 * shared[r] has above it counts for nothing and is not reported) and in whole steps of 256 positions; what is left of
 * them, and the prefix of a group of one, every sequence reads for itself.
 * Everything else is as in ne_paged_attn (its workspace of another size), the bits that are kept of a weight
 * among it; results are the same up to rounding, and the same bits for the same call.  Groups outside [0, B] or
 * descending, a negative shared[r], and whole steps that so count and reach into a sequence's new tokens or behind its
 * length are reported by ne_get_device_error() (outputs of that group invalid).  A call that has nothing to gain
 * (sequences whose rows fill tiles by themselves, judged by max_new, N, B and max_pages; caches that are small even were
 * every table full; more than 128 bf16 query heads per kv head) runs as ne_paged_attn does, and then looks at neither
 * groups nor shared.
 * workspace: ne_paged_attn_shared_workspace_size() bytes (two workspaces of ne_paged_attn and 8 D + 32 bytes per
 * row and query head). */
size_t ne_paged_attn_shared_workspace_size(int B, int N, int Hq, int Hkv, int D);
ne_status ne_paged_attn_shared(const void* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                               const int* cu_new, const int* groups, const int* shared, int R, void* o, float* lse,
                               int64_t q_ld, int B, int N, int Hq, int max_pages, int max_new, void* workspace,
                               size_t workspace_bytes, ne_stream_t stream);
ne_status ne_paged_attn_shared_f32(const float* q, const ne_paged_cache* cache, const int* page_table, const int* seq_lens,
                                   const int* cu_new, const int* groups, const int* shared, int R, float* o, float* lse,
                                   int64_t q_ld, int B, int N, int Hq, int max_pages, int max_new, void* workspace,
                                   size_t workspace_bytes, ne_stream_t stream);

/* The attention weight that every cached position receives from the new tokens, added to what it had:
 * for sequence b, kv head g and slot j < seq_lens[b]
 *   weights_out[b][g][j] = weights[b][g][j] + sum over the rows i of b at positions t_i >= j and the query
 *                          heads h of g of exp(q_ih . k_j / sqrt(D) - lse_ih),
 * q, lse, cu_new and max_new as ne_paged_attn takes and gives them (one layer).  What ne_pages_evict chooses by;
 * to count a part of the new tokens, pass the last rows of each sequence alone.
 *   weights     [B, Hkv, T] fp32, T = max_pages * page_size, or NULL (zeros)
 *   weights_out [B, Hkv, T] fp32: weights itself, or no overlap with it.  Entries at and behind
 *               seq_lens[b] stay as they were; a sequence without new tokens is copied.
 * bf16: tensor-core products of bf16 inputs, fp32 sums; f32: fp32 throughout.  The order of the sums depends
 * on the shape, lengths and device, never on timing.  cache->v is not read (a valid pointer all the same).  Slots at or
 * behind a length may hold anything, rows outside [cu_new[0], cu_new[B]) too.  Device-side arguments are checked as in
 * ne_paged_attn.  workspace: ne_paged_weights_workspace_size() bytes (316 KB), 256-byte aligned,
 * caller-owned, rewritten by every call; NULL will do where max_new * Hq / Hkv is at most 32. */
size_t ne_paged_weights_workspace_size(void);
ne_status ne_paged_weights(const void* q, const float* lse, const ne_paged_cache* cache, const int* page_table,
                           const int* seq_lens, const int* cu_new, const float* weights, float* weights_out, int64_t q_ld,
                           int B, int N, int Hq, int max_pages, int max_new, void* workspace, size_t workspace_bytes,
                           ne_stream_t stream);
ne_status ne_paged_weights_f32(const float* q, const float* lse, const ne_paged_cache* cache, const int* page_table,
                               const int* seq_lens, const int* cu_new, const float* weights, float* weights_out, int64_t q_ld,
                               int B, int N, int Hq, int max_pages, int max_new, void* workspace, size_t workspace_bytes,
                               ne_stream_t stream);

/* Pages of sequences.  The pool's state is refcount [n_pages] int32 (device memory, owned
 * by the caller, zero at first): a page is free when its count is 0.  New pages are always
 * the lowest free ids, in the order of the sequences, so a call has one result.  Every
 * call is all or nothing: when the pool has too few free pages, short_out[0] is how many
 * are missing, the outputs equal the inputs (for a fork: every child empty) and no page is
 * written; otherwise it is 0.  refcount_out (and, but for a fork, table_out) may be the
 * input itself; any other overlap of an output is refused.  Nothing synchronises: a whole scheduling
 * step can be captured.  page_table entries behind a sequence's pages are -1 on output.
 * workspace: ne_pages_workspace_size(n_pages, n, max_pages) bytes, n the number of
 * sequences (for a fork: of children), 256-byte aligned, caller-owned, rewritten by every call.  refcount
 * and refcount_out are 16-byte aligned, the other int arrays 4-byte.  A table entry in front of a
 * sequence's length (compact: any entry but -1) that is no page of the pool is reported by
 * ne_get_device_error(), whether the call is short or not: it is neither counted nor copied,
 * a resize keeps it as it is, a fork and a compaction write -1 for it.
 *
 * ne_pages_fork: child c continues sequence parents[c] (-1: an empty child).  Shared
 * (deep == 0): whole pages are shared (their counts rise), the partly filled last page is
 * copied to a new page, so a page that is still written belongs to one sequence.  deep:
 * every page is copied.  Only filled slots are copied.
 *   child_table [C, max_pages] (out), child_lens [C] (out) */
size_t ne_pages_workspace_size(int n_pages, int n, int max_pages);
ne_status ne_pages_fork(const ne_paged_cache* cache, const int* refcount, const int* page_table,
                        const int* seq_lens, const int* parents, int deep, int* refcount_out,
                        int* child_table, int* child_lens, int* short_out, int B, int C, int max_pages,
                        void* workspace, size_t workspace_bytes, ne_stream_t stream);
/* ne_pages_resize: sequence b goes from seq_lens[b] to new_lens[b] positions (0 frees it).
 * Pages behind the new length are given back first, then a partly filled last page (of
 * min(old, new) positions) that other sequences still hold is copied to a page of its own,
 * then new pages are taken; a page that only such copies leave behind is free for the
 * next call.  seq_lens itself is left to the caller.  Lengths are clamped to
 * [0, max_pages * page_size] and reported. */
ne_status ne_pages_resize(const ne_paged_cache* cache, const int* refcount, const int* page_table,
                          const int* seq_lens, const int* new_lens, int* refcount_out, int* table_out,
                          int* short_out, int B, int max_pages, void* workspace, size_t workspace_bytes,
                          ne_stream_t stream);
/* ne_pages_compact: moves the live pages into 0 .. n_live - 1: the j-th live page at or
 * behind n_live goes to the j-th free page in front of it, the others stay.
 *   remap [n_pages] (out): a live page's new id, -1 for a free page;  n_live [1] (out)
 * The one table given is rewritten; further tables go through remap.  Never short. */
ne_status ne_pages_compact(const ne_paged_cache* cache, const int* refcount, const int* page_table,
                           int* refcount_out, int* table_out, int* remap, int* n_live, int B, int max_pages,
                           void* workspace, size_t workspace_bytes, ne_stream_t stream);

/* Sequences cut to fewer positions, those with the least accumulated attention weight given up
 * (ne_paged_weights sums it): sequence b keeps m = min(new_lens[b], seq_lens[b]) of its n = seq_lens[b]
 * slots, chosen for every layer and kv head by itself.  Guarded slots stay first: those of positions below
 * `sink`, and of the `recent` newest; then the largest weights, ties to the lowest slot (also among
 * guarded slots where m does not hold them all; -0 counts as 0, NaN below every number).  A kept row
 * stays in its slot, but those in slots m .. n-1 move into the slots below m that were given up, the j-th of
 * them (in slot order) into the j-th: keys, values, weight and position.  Attention over the cut
 * sequence is attention over the kept positions, whose order does not matter to it; new tokens follow in
 * slots m, m+1, ..., rotated at slot + pos_offset_out[b] (ne_paged_append_at).
 *   weights, weights_out      [layers, B, Hkv, T] fp32, T = max_pages * page_size
 *   positions, positions_out  [layers, B, Hkv, T] int32: the position that a slot holds; -1 (what a caller
 *                             fills in at first, and what a cut leaves behind m): slot + pos_offset[b]
 *   pos_offset, pos_offset_out [B] int32: positions given up so far; pos_offset_out = pos_offset + n - m.
 *                             0 <= pos_offset[b] < 2^30
 * weights, positions and their outputs are 16-byte aligned, the other arrays 4.
 * Slots m .. n-1 get weight 0 and position -1; entries at and behind n stay as they were.  Each output
 * may be its input; any other overlap of these arrays and the workspace is refused, and k and v that are one pool
 * (the pools' memory is compared with nothing else).  The pages that hold a sequence's slots must belong to it alone
 * (ne_pages_fork with deep sees to that; a child's rows of these arrays are the caller's to copy, as are a new
 * sequence's to fill in).  ne_pages_resize from seq_lens to m, not to a new_lens above it, which would grow the sequence, then
 * gives back the pages behind m.  Bad lengths, offsets and page ids are clamped or skipped and reported by
 * ne_get_device_error().  workspace: ne_pages_evict_workspace_size() bytes (4 per entry of weights), 256-byte
 * aligned, caller-owned, rewritten by every call.  layers * B * Hkv < 2^31; 0 <= sink, recent <= 2^30. */
size_t ne_pages_evict_workspace_size(int layers, int B, int Hkv, int T);
ne_status ne_pages_evict(const ne_paged_cache* cache, const float* weights, const int* positions, const int* pos_offset,
                         const int* page_table, const int* seq_lens, const int* new_lens, int sink, int recent,
                         float* weights_out, int* positions_out, int* pos_offset_out, int B, int max_pages,
                         void* workspace, size_t workspace_bytes, ne_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* ne_status_string(ne_status s);
/* Detail of the last error on the calling thread ("" if none). */
const char* ne_last_error(void);

/* Synchronises `stream`, then reads and clears the current device's error word.
 * Returns NE_ERR_DEVICE_TIMEOUT if a kernel's bounded wait ran out since the last
 * check (the kernel then skipped the rest of its work and its outputs are invalid),
 * NE_ERR_CUDA if the synchronisation failed, else NE_OK. */
ne_status ne_get_device_error(ne_stream_t stream);

/* Wall-clock limit of every bounded wait inside the kernels (default 2000 ms, or
 * NE_ATTN_TIMEOUT_MS from the environment).  0 restores the default. */
void ne_set_wait_timeout_ms(uint32_t ms);

/* Diagnostic: launches one tiny kernel whose bounded wait can never be satisfied, so
 * it runs out after `timeout_ms` and records NE_ERR_DEVICE_TIMEOUT in the device error
 * word, exactly as a stalled attention kernel would.  Used to test the error path
 * without faulting or hanging the GPU. */
ne_status ne_selftest_wait_timeout(uint32_t timeout_ms, ne_stream_t stream);

/* Diagnostic timing of the kernels behind the calls above.  While enabled (on != 0),
 * every call records a CUDA event before and after each kernel it launches, on the
 * call's stream; ne_profile_totals() synchronises the current device and returns, per
 * phase, the summed milliseconds and the number of launches since enabling:
 * phase 0 forward, 1 backward Delta preprocess, 2 backward main, 3 backward dQ
 * epilogue.  Enabling again restarts the sums and reuses the events already made;
 * disabling (on == 0) frees them.  Not thread-safe; off by default. */
void ne_profile_enable(int on);
ne_status ne_profile_totals(double ms_out[4], int launches_out[4]);

/* Releases the library's per-device caches (RoPE tables, error words). */
void ne_shutdown(void);

#ifdef __cplusplus
}
#endif

#endif /* NEATTN_H */
