/*
 * dflash_attn.h -- C ABI of the GB300 (sm_103a) DFlash draft block-attention
 * library.
 *
 * The operation.  A DFlash draft predicts a whole block of block_size tokens
 * in one non-causal forward whose keys and values are
 * [projected target-hidden context (S tokens) | noise block (Q tokens)]
 * (nemo_automodel.components.speculative.dflash.draft_kimi_k3 page, module
 * docstring).  Queries are the Q noise (draft) tokens: per
 * KimiK3DFlashAttention.forward the query axis has blocks x block_size rows
 * and the key axis the sequence plus those rows.  The backbone is Kimi K3
 * MLA: one K/V per query head with no GQA repeat (KimiK3DFlashAttention), and
 * NoPE: the rope part of the key is one vector per token, shared by all
 * heads, with no rotary embedding (module docstring).  Per head h, query row
 * i and key k:
 *
 *   s(i,k) = ( q_nope(i,h) . k_nope(k,h) + q_rope(i,h) . k_rope(k) ) * scale
 *            [+ mask(i,k) on the dense entry point]
 *   out(i,h) = sum_k softmax_k(s(i,.)) v(k,h)
 *
 * with scale = (d_nope + d_rope)^-0.5 by default
 * (nemo_automodel.components.speculative.dspark.draft_kimi_k3 page,
 * KimiK3DSparkAttention: q_head_dim = qk_nope_head_dim + qk_rope_head_dim,
 * scaling = q_head_dim ** -0.5).
 *
 * Layouts (row-major, contiguous, element type = dtype):
 *   q      [B, Q, H, d_nope + d_rope]   the nope part first, then the rope part
 *   k_nope [B, S+Q, H, d_nope]          keys 0..S-1 context, S..S+Q-1 noise
 *   k_rope [B, S+Q, d_rope]             one per token, shared by every head
 *   v      [B, S+Q, H, d_v]
 *   out    [B, Q, H, d_v]               written in dtype (bf16: round to nearest even)
 *   lse    [B, H, Q] fp32, optional     natural-log log-sum-exp of the scaled scores
 *   mask   [B, 1, Q, S+Q] (dense only)  additive, element type = dtype
 *
 * Ownership and execution.  Every pointer argument of the compute calls is a
 * device pointer owned by the caller; the library allocates no device memory
 * and uses only the caller's workspace.  Calls are asynchronous on the given
 * stream and never synchronise the host.  Errors are status codes; nothing is
 * thrown across the ABI.  Host-side validation happens before any launch, and
 * a call that returns an error launches nothing.  Conditions only the device
 * can see (an anchor outside [0, S], a wait that ran past its time limit) are
 * recorded in a per-device error word read by dflash_last_device_error().
 *
 * Rows that see no key (dense masks whose row is entirely -inf) produce
 * out = 0 and lse = -inf.  Mask entries must be finite or -inf.
 */
#ifndef DFLASH_ATTN_H_
#define DFLASH_ATTN_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define DFLASH_API __attribute__((visibility("default")))
#else
#define DFLASH_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* dflash_stream_t;

typedef enum {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID = 1,     /* null pointer, negative size, bad anchor/offset on the device */
  DFLASH_ERR_SHAPE = 2,       /* inconsistent shapes (nb*block_size != Q, ...) */
  DFLASH_ERR_DTYPE = 3,       /* unknown dtype */
  DFLASH_ERR_ALIGN = 4,       /* a tensor base pointer is not 16-byte aligned */
  DFLASH_ERR_UNSUPPORTED = 5, /* head dims beyond the kernels' limits */
  DFLASH_ERR_WORKSPACE = 6,   /* workspace null, misaligned (256 B) or too small */
  DFLASH_ERR_CUDA = 7,        /* a CUDA runtime call or launch failed */
  DFLASH_ERR_TIMEOUT = 8      /* a bounded device wait gave up (kernel returned early) */
} dflash_status_t;

typedef enum { DFLASH_BF16 = 0, DFLASH_FP32 = 1 } dflash_dtype_t;

typedef struct {
  int B;      /* batch rows */
  int H;      /* heads (one K/V per query head) */
  int S;      /* context tokens */
  int Q;      /* noise (query) tokens = nb * block_size */
  int d_nope; /* qk_nope_head_dim */
  int d_rope; /* qk_rope_head_dim (head-shared key slice) */
  int d_v;    /* v_head_dim */
  float scale; /* <= 0 selects (d_nope + d_rope)^-0.5 */
} dflash_dims_t;

/* Tile grid of the schedule: DFLASH_TILE_M query rows x DFLASH_TILE_N keys,
 * anchored at query row 0 and key 0 of each batch row. */
#define DFLASH_TILE_M 128
#define DFLASH_TILE_N 128
enum { DFLASH_TILE_SKIP = 0, DFLASH_TILE_PARTIAL = 1, DFLASH_TILE_FULL = 2 };

/* Kernel limits.  bf16 with (d_nope, d_rope, d_v) = (128, 64, 128) runs on the
 * tensor-core (tcgen05) kernels; every other supported shape, and all fp32,
 * runs on the exact CUDA-core kernel. */
#define DFLASH_MAX_DQK 512 /* d_nope + d_rope */
#define DFLASH_MAX_DV 256

/*
 * Dense additive-mask entry point (KimiK3DFlashAttention.forward: the
 * additive mask [batch, 1, blocks*block_size, sequence + blocks*block_size]
 * is used unchanged).  A key is visible to a row iff its mask entry is not
 * -inf; the entry is added to the scaled score.  The mask is first scanned
 * on the device into per-tile classes (all 0 / all -inf / mixed) so that
 * all--inf tiles are skipped and all-0 tiles need no mask reads.
 *   workspace: >= dflash_attn_workspace_size(DFLASH_MODE_DENSE, ...) bytes,
 *              256-byte aligned, device memory; contents need no initialisation.
 */
DFLASH_API dflash_status_t dflash_attn_dense(const dflash_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                  const void* k_nope, const void* k_rope, const void* v,
                                  const void* mask, void* out, float* lse, void* workspace,
                                  size_t ws_bytes, dflash_stream_t stream);

/*
 * Anchored entry point.  anchors [B, nb] int32 on the device; Q = nb *
 * block_size.  Query row i of batch row b belongs to block j = i / block_size
 * and sees exactly the context keys p < anchors[b, j] and the block_size noise
 * keys S + j*block_size + t of its own block (the DFlash block contract of the
 * draft_kimi_k3 page: one block = [anchor, MASK, ...] predicted in one
 * non-causal forward).  Anchors must lie in [0, S]; sortedness and
 * distinctness are not required.  An anchor outside [0, S] is clamped and
 * recorded as DFLASH_ERR_INVALID in the device error word.
 */
DFLASH_API dflash_status_t dflash_attn_anchored(const dflash_dims_t* dims, dflash_dtype_t dtype,
                                     const void* q, const void* k_nope, const void* k_rope,
                                     const void* v, const int32_t* anchors, int nb,
                                     int block_size, void* out, float* lse, void* workspace,
                                     size_t ws_bytes, dflash_stream_t stream);

/*
 * Ragged (serving) entry point: R requests packed along the token axis by row
 * offsets (max.pipelines.architectures.dflash_kimi_k25 page, DFlashKimiK25:
 * input_row_offsets; ctx_at_draft_cache_length = True; supports_zero_draft_rows
 * = False).  Request r owns query rows [q_offsets[r], q_offsets[r+1]) and key
 * rows [kv_offsets[r], kv_offsets[r+1]); its keys are its context followed by
 * its q_len noise tokens, so S_r = kv_len - q_len.  q_len must be a positive
 * multiple of block_size and q_offsets[r] a multiple of block_size; anchors
 * are indexed by global block q_offsets[r]/block_size + local block, and obey
 * the anchored rule inside the request.
 *   q [total_q, H, d_nope+d_rope], k_nope [total_kv, H, d_nope],
 *   k_rope [total_kv, d_rope], v [total_kv, H, d_v], out [total_q, H, d_v],
 *   lse [H, total_q] fp32 (optional), offsets int32 [R+1] on the device.
 *   total_q, total_kv: extents of the packed tensors (q_offsets[R],
 *   kv_offsets[R]); max_q_len: an upper bound on every request's q_len.
 * Offsets that break these rules, and a request whose q_len exceeds
 * max_q_len, are recorded as DFLASH_ERR_INVALID in the device error word and
 * the offending request is skipped (its out and lse rows are not written).
 * Decode-shaped batches (small q_len, long context) are split along the
 * context and merged with a log-sum-exp combine kernel.
 */
DFLASH_API dflash_status_t dflash_attn_ragged(int R, int H, int d_nope, int d_rope, int d_v, float scale,
                                   dflash_dtype_t dtype, const void* q, const void* k_nope,
                                   const void* k_rope, const void* v, const int32_t* q_offsets,
                                   const int32_t* kv_offsets, const int32_t* anchors,
                                   int block_size, int total_q, int total_kv, int max_q_len,
                                   void* out, float* lse, void* workspace, size_t ws_bytes,
                                   dflash_stream_t stream);

/*
 * Ragged entry point over compressed KV latents (Kimi K3 MLA).  Each token
 * carries its KV latent c (kv_rank values, after the latent norm) and the
 * head-shared rope key; kv_b_proj expands the latent to one k_nope + v slice
 * per head (nemo_automodel.components.speculative.dflash.draft_kimi_k3 page,
 * KimiK3DFlashAttention: kv_b_proj produces num_attention_heads slices of
 * qk_nope_head_dim + v_head_dim; ...dspark.draft_kimi_k3 page,
 * KimiK3DSparkAttention: kv_lora_rank, kv_b_proj; nemo_automodel.components.
 * models.kimi_k3.model page: the compressed latent is kv_lora_rank +
 * qk_rope_head_dim values per token).  With w_kv_b viewed as [H, d_nope + d_v,
 * kv_rank] (per head: the d_nope key rows, then the d_v value rows):
 *   k_nope[t,h,e] = sum_c w_kv_b[h,e,c] c_kv[t,c],
 *   v[t,h,e]      = sum_c w_kv_b[h,d_nope+e,c] c_kv[t,c],
 * and the result is dflash_attn_ragged over those keys and values (same
 * offsets, anchors, block rule, scale, out and lse).
 *   q [total_q, H, d_nope+d_rope], c_kv [total_kv, kv_rank],
 *   k_rope [total_kv, d_rope], w_kv_b [H, d_nope+d_v, kv_rank] (the
 *   projection weight, row-major), out [total_q, H, d_v], lse [H, total_q].
 * bf16 with (d_nope, d_rope, d_v, kv_rank) = (128, 64, 128, 512), H a multiple
 * of 4 and max_q_len <= 16 (the serving decode shape) runs absorbed on the
 * tensor cores: W_UK is folded into q, the attention runs over the latents
 * (every head reads each token's latent once), and W_UV is applied after the
 * softmax; q_abs and o_lat are rounded to bf16 on the way.  Every other shape
 * (and fp32) expands the keys and values into the workspace and runs the
 * ragged kernels on them.  A request skipped for invalid offsets or q_len >
 * max_q_len is recorded as DFLASH_ERR_INVALID; its rows are written as 0
 * (lse -inf) on the absorbed path and left unwritten on the expanded path.
 *   workspace: >= dflash_attn_latent_workspace_size(...) bytes, 256-byte
 *   aligned; needs no initialisation.
 */
#define DFLASH_MAX_KV_RANK 1024
DFLASH_API size_t dflash_attn_latent_workspace_size(int R, int H, int d_nope, int d_rope, int d_v, int kv_rank,
                                                    dflash_dtype_t dtype, int total_q, int total_kv, int max_q_len);
DFLASH_API dflash_status_t dflash_attn_latent_ragged(int R, int H, int d_nope, int d_rope, int d_v, int kv_rank,
                                                     float scale, dflash_dtype_t dtype, const void* q,
                                                     const void* c_kv, const void* k_rope, const void* w_kv_b,
                                                     const int32_t* q_offsets, const int32_t* kv_offsets,
                                                     const int32_t* anchors, int block_size, int total_q,
                                                     int total_kv, int max_q_len, void* out, float* lse,
                                                     void* workspace, size_t ws_bytes, dflash_stream_t stream);

/*
 * Dense entry point that allocates nothing and takes no workspace.  (No
 * counterpart on the pages: this is a convenience of this library.)
 *
 * For callers that cannot provide device scratch memory -- runtimes that plan
 * all device memory once at start-up and forbid allocations while serving,
 * or plugin interfaces whose fixed signature has no workspace argument.  The
 * dense path's only scratch, one class byte per 128x128 mask tile, lives in a
 * fixed device array inside the library (DFLASH_NOALLOC_MAX_TILES + 256 bytes,
 * held on every GPU that loads the library until the process exits).
 * Arguments and results are those of dflash_attn_dense.
 *   - Returns DFLASH_ERR_WORKSPACE when B * ceil(Q/128) * ceil((S+Q)/128)
 *     exceeds DFLASH_NOALLOC_MAX_TILES; nothing is launched then.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it; make that first call before any
 *     stream capture.
 *   - Every call shares the one array, which keeps the previous call's
 *     contents (each call rewrites every byte it reads).  Calls that overlap
 *     on the GPU (different streams, or different host threads on one device)
 *     race on it and must be serialised by the caller.
 *   - Calls no cudaMalloc, cudaFree or allocating library routine.
 */
#define DFLASH_NOALLOC_MAX_TILES (1 << 20)
DFLASH_API dflash_status_t dflash_attn_dense_noalloc(const dflash_dims_t* dims, dflash_dtype_t dtype,
                                                     const void* q, const void* k_nope, const void* k_rope,
                                                     const void* v, const void* mask, void* out, float* lse,
                                                     dflash_stream_t stream);

enum {
  DFLASH_MODE_DENSE = 0,
  DFLASH_MODE_ANCHORED = 1,
  DFLASH_MODE_RAGGED = 2,
  DFLASH_MODE_DENSE_BACKWARD = 3,
  DFLASH_MODE_ANCHORED_BACKWARD = 4
};

/*
 * Backward pass of the anchored and dense entry points: gradients of the
 * scalar L = sum over (b, i, h, d) of dout * out.  The DFlash draft is a
 * trained module (nemo_automodel.components.speculative.dflash.draft_kimi_k3
 * page, module docstring), so the attention's gradients are needed.  Per head
 * and query row i over its visible keys k, with P the softmax weights
 * recomputed from the forward's lse:
 *   dP(i,k) = dout(i) . v(k),  D(i) = dout(i) . out(i),  dS = P (dP - D)
 *   dq(i)      = scale * sum_k dS(i,k) [k_nope(k) | k_rope(k)]
 *   dk_nope(k) = scale * sum_i dS(i,k) q_nope(i)
 *   dk_rope(k) = scale * sum_h sum_i dS(i,k) q_rope(i)   (one rope key per token
 *                serves every head, so its gradient is the sum over heads)
 *   dv(k)      = sum_i P(i,k) dout(i)
 * The mask (dense) is a constant input and gets no gradient.
 *   q, k_nope, k_rope, v, anchors/mask: the forward's inputs (same layouts).
 *   out [B,Q,H,d_v] and lse [B,H,Q] fp32: the forward's outputs for these
 *     inputs (lse is required here).
 *   dout [B,Q,H,d_v]: gradient of L with respect to out.
 *   dq [B,Q,H,d_nope+d_rope], dk_nope [B,S+Q,H,d_nope], dk_rope [B,S+Q,d_rope],
 *   dv [B,S+Q,H,d_v]: written in dtype; every element is written (keys no row
 *     sees get 0).  With Q = 0 only the key gradients are written (all 0) and
 *     the query-side pointers may be null.
 *   workspace: >= dflash_attn_workspace_size(DFLASH_MODE_*_BACKWARD, ...)
 *     bytes, 256-byte aligned, device memory; needs no initialisation.
 * Limits: d_nope + d_rope <= DFLASH_BWD_MAX_DQK and d_v <= DFLASH_BWD_MAX_DV
 * (else DFLASH_ERR_UNSUPPORTED).  Device pointers, 16-byte aligned; the call
 * is asynchronous on `stream` and allocates no device memory.  On the
 * tensor-core path (bf16, head dims 128/64/128) the dq kernel runs on a second
 * stream that the library creates once per host thread and device; it is
 * forked from `stream` (an event) and joined back into it before the call
 * returns, so work queued on `stream` afterwards sees every gradient.  Errors
 * as for the forward entry points.
 */
#define DFLASH_BWD_MAX_DQK 256
#define DFLASH_BWD_MAX_DV 128
DFLASH_API dflash_status_t dflash_attn_anchored_backward(
    const dflash_dims_t* dims, dflash_dtype_t dtype, const void* q, const void* k_nope, const void* k_rope,
    const void* v, const int32_t* anchors, int nb, int block_size, const void* out, const float* lse,
    const void* dout, void* dq, void* dk_nope, void* dk_rope, void* dv, void* workspace, size_t ws_bytes,
    dflash_stream_t stream);
DFLASH_API dflash_status_t dflash_attn_dense_backward(const dflash_dims_t* dims, dflash_dtype_t dtype,
                                                      const void* q, const void* k_nope, const void* k_rope,
                                                      const void* v, const void* mask, const void* out,
                                                      const float* lse, const void* dout, void* dq,
                                                      void* dk_nope, void* dk_rope, void* dv, void* workspace,
                                                      size_t ws_bytes, dflash_stream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The serving step of a grouped-query draft (max.pipelines.architectures.
 * dflash_kimi_k25 page: DFlashKimiK25, whose draft has grouped key/value heads,
 * rotary positions and optional query/key norms; materialize writes projected
 * context into the draft's cache, forward_block attends one drafted block per
 * request over it, ragged by input_row_offsets):
 *   dflash_qk_norm_rope   norm and rotation of query and key heads (+ backward),
 *   dflash_cache_append   the same on the way into a paged cache,
 *   dflash_attn_paged     attention of the new tokens over the pages,
 *   dflash_verify         acceptance of drafted tokens;
 * and where trees of tokens are drafted, or requests share their beginnings:
 *   dflash_attn_tree      attention of a tree's nodes over the pages,
 *   dflash_sample         tokens, or distributions, from logits,
 *   dflash_tree_accept    the walk down the tree along the sampled tokens,
 *   dflash_cache_compact  the accepted nodes moved together,
 *   dflash_pages_resize, dflash_pages_fork, dflash_cache_copy
 *                         pages taken, given back, shared and copied.
 * Element types, ownership, streams and errors as above.  The device that holds
 * the tensors has to be the current one.  Calls that may run at the same time
 * (on two streams, or in graphs that are replayed side by side) need a workspace
 * each.  Every call may be captured into a graph.  What a call of the second list writes
 * must not overlap what it reads, nor one result another, except where it says so; among the
 * whole numbers of the walk, of compaction and of the pages' calls that is refused
 * (DFLASH_ERR_INVALID).
 */

/*
 * Norm and rotation of query and key heads.  Per token t and head vector x of
 * D components:
 *   y = x * (mean_d x_d^2 + eps)^-1/2 * w          (w given; y = x when it is null)
 *   out = y with its first rot_dim components rotated in rot_dim/2 planes by
 *         the angles of position positions[t]; the others are passed on.
 * Plane i joins components (i, i + rot_dim/2), or (2i, 2i+1) when interleaved:
 *   a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i.
 * Everything is computed in fp32 and rounded once, to the element type.
 *   q [T, H_q, D] and k [T, H_kv, D]: tokens q_stride / k_stride elements apart
 *     (0: H * D), the heads of a token contiguous, so that slices of one
 *     projection's output [T, (H_q + 2 H_kv) D] are taken as they are.
 *   q_norm, k_norm [D], each nullable: the norm weights, element type = dtype.
 *   cos_sin [max_pos, rot_dim] fp32: rot_dim/2 cosines, then rot_dim/2 sines of
 *     each position; null when rot_dim = 0 (then positions is not read either).
 *   positions [T] int32.  A position outside [0, max_pos) is recorded as
 *     DFLASH_ERR_INVALID in the device error word and its token is skipped (its
 *     output rows are left as they were; it adds nothing to the norm gradients).
 *   q_out [T, H_q, D], k_out [T, H_kv, D]: contiguous; may be q and k themselves
 *     where those are contiguous.  H_q or H_kv may be 0 (its pointers unused).
 * D: a multiple of 8 up to DFLASH_PAGED_MAX_D; rot_dim even, at most D.
 */
#define DFLASH_PAGED_MAX_D 256
typedef struct {
  int T;           /* tokens */
  int H_q, H_kv;   /* query and key heads */
  int D;           /* head dimension */
  int rot_dim;     /* rotated components of a head */
  int max_pos;     /* rows of cos_sin */
  int interleaved; /* 0: planes (i, i + rot_dim/2); 1: planes (2i, 2i + 1) */
  float eps;       /* norm epsilon, >= 0 (the gradients take one below 2^-126 for 2^-126) */
  int64_t q_stride, k_stride; /* elements from token to token of q and k; 0: contiguous */
} dflash_rope_dims_t;

DFLASH_API dflash_status_t dflash_qk_norm_rope(const dflash_rope_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                               const void* k, const void* q_norm, const void* k_norm,
                                               const float* cos_sin, const int32_t* positions, void* q_out,
                                               void* k_out, dflash_stream_t stream);

/*
 * Gradients of sum(dq_out * q_out) + sum(dk_out * k_out).  With g the rotation's
 * transpose applied to the output gradient, x^ = x r, r = (mean x^2 + eps)^-1/2:
 *   dw = sum over tokens and heads of g x^,
 *   dx = r (g w - x^ mean_d(g w x^))       (dx = g without a norm).
 *   q, k: the forward's inputs (strides as there; unused, and nullable, where
 *     the norm weight is null).  dq_out, dk_out, dq, dk: contiguous; dq and dk
 *     may be dq_out and dk_out themselves.
 *   dq_norm, dk_norm [D] fp32: written (0 for no tokens); required where the
 *     weight is given, unused elsewhere.  Sums run in a fixed order: equal
 *     inputs give equal bits on one device type.
 *   workspace: >= dflash_qk_norm_rope_workspace_size(dims) bytes, 256-byte
 *     aligned; needs no initialisation.
 */
DFLASH_API size_t dflash_qk_norm_rope_workspace_size(const dflash_rope_dims_t* dims);
DFLASH_API dflash_status_t dflash_qk_norm_rope_backward(
    const dflash_rope_dims_t* dims, dflash_dtype_t dtype, const void* q, const void* k, const void* q_norm,
    const void* k_norm, const float* cos_sin, const int32_t* positions, const void* dq_out, const void* dk_out,
    void* dq, void* dk, float* dq_norm, float* dk_norm, void* workspace, size_t ws_bytes, dflash_stream_t stream);

/*
 * A paged key/value cache.  Page g holds page_size consecutive positions of one
 * request, each with H_kv heads of D values: k_cache and v_cache are
 * [num_pages, page_size, H_kv, D], pages k_page_stride / v_page_stride elements
 * apart (0: contiguous), so that both may be halves of one
 * [num_pages, 2, page_size, H_kv, D] tensor.  Position p of request r lies in
 * row p % page_size of page page_table[r, p / page_size].
 *
 * A step's batch: R requests, request r with the new tokens
 * [q_offsets[r], q_offsets[r+1]) of the packed token axis (possibly none), which
 * are the last ones of its kv_lens[r] positions.  Table entries behind
 * ceil(kv_lens[r] / page_size) and what lies behind position kv_lens[r] in the
 * last page are never used.  Packed rows behind q_offsets[R] are left as they
 * were.  All int32, on the device.
 */
typedef struct {
  int R;                /* requests, at most 2^30 */
  int H_q, H_kv;        /* query and key/value heads; H_kv divides H_q */
  int D;                /* head dimension */
  int total_q;          /* rows of the packed token axis (>= q_offsets[R]) */
  int max_q_len;        /* bound on every request's new tokens */
  int num_pages;        /* pages of the cache */
  int page_size;        /* positions of a page */
  int max_pages;        /* columns of page_table [R, max_pages] */
  int64_t k_page_stride, v_page_stride; /* elements from page to page; 0: contiguous */
} dflash_paged_dims_t;

/*
 * Appends the new tokens' keys and values to their pages, keys (and, where q is
 * given, queries) normed and rotated as by dflash_qk_norm_rope at the position
 * they take in their request, kv_lens[r] - n + i.  kv_lens already counts the
 * new tokens.  Values are copied.  (DFlashKimiK25.materialize: without q.)
 *   rope: norm and rotation (T, H_q, H_kv and D are not read; q_stride and
 *     k_stride are, v_stride is this call's).  rot_dim = 0 and null weights
 *     append the keys as they are.
 *   q, k, v: packed [total_q, heads, D] with token strides; q and q_out are
 *     null where no queries are wanted; q_out [total_q, H_q, D] contiguous.
 * A token whose position is negative, lies beyond the rotation table or beyond
 * the page table, or whose page id is outside [0, num_pages), and every token
 * of a request whose offsets are not ascending within [0, total_q], is recorded
 * as DFLASH_ERR_INVALID and skipped (its cache and q_out rows stay as they
 * were); where offsets descend, tokens of requests next to that may be skipped
 * too.  Two tokens must not be given one cache row: requests may share pages
 * that only hold earlier positions.  max_q_len is not read.
 */
DFLASH_API dflash_status_t dflash_cache_append(const dflash_paged_dims_t* dims, const dflash_rope_dims_t* rope,
                                               dflash_dtype_t dtype, const void* q, const void* k, const void* v,
                                               int64_t v_stride, const void* q_norm, const void* k_norm,
                                               const float* cos_sin, const int32_t* page_table,
                                               const int32_t* kv_lens, const int32_t* q_offsets, void* q_out,
                                               void* k_cache, void* v_cache, dflash_stream_t stream);

/*
 * Attention of the new tokens over their requests' pages.  Token i of a request
 * with n new tokens and length L = kv_lens[r] sees positions p < L (causal = 0:
 * the drafted block, which sees its context and all of itself) or
 * p < L - n + i + 1 (causal = 1: prefill chunks, verification, single tokens).
 * Query head h reads key/value head h / (H_q / H_kv).
 *   out(i,h) = sum_p softmax_p(q(i,h) . k(p) scale) v(p),  scale <= 0: D^-0.5
 *   q, out [total_q, H_q, D] contiguous; lse [H_q, total_q] fp32, optional.
 * A row that sees nothing gets out = 0 and lse = -inf; one with a score that is
 * NaN or +inf gets NaN in both, and no other row is touched by it.  Keys and values of the
 * positions p < L have to be finite; a page id outside [0, num_pages) is recorded
 * as DFLASH_ERR_INVALID and read as zeros.  A request whose offsets or length
 * are out of range (n < 0 or > max_q_len, L < 0 or > max_pages * page_size) is
 * recorded as DFLASH_ERR_INVALID and skipped (rows left as they were).
 * D: a multiple of 8 up to DFLASH_PAGED_MAX_D.  bf16 with D <= 128,
 * H_q / H_kv <= 128 and page_size a multiple of 8 runs on the tensor cores;
 * everything else, and all fp32, on the CUDA-core kernel.  Work is dealt in
 * equal runs of key tiles to the SMs whatever the lengths, and the pieces of
 * divided rows are merged by a second kernel, in a fixed order.  max_q_len also
 * chooses the form of the tensor-core kernel: with a bound of more tokens than 128
 * rows hold, single tokens take about a quarter longer, so that a batch of single
 * tokens wants a bound of its own.
 *   workspace: >= dflash_attn_paged_workspace_size(dims, dtype) bytes, 256-byte
 *     aligned; its size does not depend on the lengths; needs no initialisation.
 */
DFLASH_API size_t dflash_attn_paged_workspace_size(const dflash_paged_dims_t* dims, dflash_dtype_t dtype);
DFLASH_API dflash_status_t dflash_attn_paged(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                             const void* k_cache, const void* v_cache, const int32_t* page_table,
                                             const int32_t* kv_lens, const int32_t* q_offsets, int causal, float scale,
                                             void* out, float* lse, void* workspace, size_t ws_bytes,
                                             dflash_stream_t stream);

/*
 * Attention of drafted trees over the pages.  A request's new tokens are the nodes
 * of a tree, in an order in which every node comes behind its parent; they lie in
 * the last n of its L = kv_lens[r] positions, node i at position L - n + i
 * (what is rotated, if it is, is the depth: dflash_qk_norm_rope with positions
 * L - n + depth, dflash_cache_append then without a rotation).  Node i sees the
 * context p < L - n, itself, its parent, that one's parent and so on, and no other
 * node.  (Keys and values of all L positions have to be finite all the same: a node that is
 * not seen has the weight 0, and 0 times a value that is infinite or NaN is NaN.)
 *   parents [total_q] int32: index of the parent among the request's nodes, -1
 *     for a root (there may be several).  A value that is not smaller than the
 *     node's own index, or negative, ends the chain like -1.
 * A node's chain is followed on the device, once for every 128 (or fewer) positions
 * of the tree: deep trees of thousands of nodes are slow.  Everything else, the
 * workspace and its size too, is as for dflash_attn_paged, whose causal form this
 * is where every node's parent is the node before it.
 */
DFLASH_API dflash_status_t dflash_attn_tree(const dflash_paged_dims_t* dims, dflash_dtype_t dtype, const void* q,
                                            const void* k_cache, const void* v_cache, const int32_t* page_table,
                                            const int32_t* kv_lens, const int32_t* q_offsets, const int32_t* parents,
                                            float scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                                            dflash_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, with given
 * random numbers.  Request r drafted n = draft_offsets[r+1] - draft_offsets[r]
 * tokens x_0 .. x_{n-1} (possibly none).  With p_j the target's probabilities at
 * drafted position j (p_n: behind the last one) and q_j the draft's:
 *   a = first j with not (u_j q_j(x_j) < p_j(x_j)), or n where there is none;
 *   w = max(p_a - q_a, 0) where a < n and that is not all zero, else p_a;
 *   z = smallest i with w_0 + ... + w_i > s_r (w_0 + ... + w_{V-1}).
 * out_tokens[r] = x_0 .. x_{a-1}, z, then -1; num_accepted[r] = a.  A token
 * drawn from q_j is so turned into one that is distributed as p_j.
 *   target_probs [rows, V] fp32, request r's rows from draft_offsets[r] + r on
 *     (n + 1 of them); draft_probs [total_draft, V] fp32, or null for a draft
 *     that took its most likely token (q_j is then 1 at x_j and 0 elsewhere).
 *     Rows target_stride / draft_stride elements apart (0: V).
 *   draft_tokens [total_draft], draft_offsets [R+1] int32; accept_u
 *     [total_draft] and sample_u [R] fp32 in [0, 1).
 *   out_tokens [R, max_draft + 1], num_accepted [R] int32: every element written.
 * Comparisons are made in 64 bits, and weights are added up as whole steps of
 * 2^-45, so that the result does not depend on the order of the sum (a w below
 * 2^-46 counts as zero).  Probabilities lie in [0, 1]; an entry where one is NaN
 * has no weight, and rows that are no distribution give some token of the
 * vocabulary.  A drafted token outside [0, V)
 * is recorded as DFLASH_ERR_INVALID and rejected; a request whose w is all zero
 * is recorded and gets z = 0; one whose offsets are out of range is recorded and
 * gets num_accepted = 0 and tokens -1.
 */
typedef struct {
  int R;           /* requests */
  int V;           /* vocabulary */
  int total_draft; /* rows of the packed draft axis (>= draft_offsets[R]) */
  int max_draft;   /* bound on every request's drafted tokens, at most 2^30 */
  int64_t target_stride, draft_stride; /* elements from row to row; 0: V */
} dflash_verify_dims_t;
DFLASH_API dflash_status_t dflash_verify(const dflash_verify_dims_t* dims, const float* target_probs,
                                         const float* draft_probs, const int32_t* draft_tokens,
                                         const int32_t* draft_offsets, const float* accept_u, const float* sample_u,
                                         int32_t* out_tokens, int32_t* num_accepted, dflash_stream_t stream);

/*
 * Tokens drawn from logits with given random numbers, and the distributions they are
 * drawn from.  Row r with logits l, T = temperature[r], m = max l, w_i = exp((l_i - m) / T):
 *   in the order of falling logits, equal ones by rising i,
 *   K = the first top_k[r] tokens (all where that is <= 0 or >= V),
 *   P = the shortest beginning of K whose weights reach top_p[r] times the weight of K
 *       (one token at least; all of K where top_p[r] >= 1),
 *   S = the tokens of P with w_i >= min_p[r] (<= 0: all; above 1 it counts as 1);
 *   tokens[r] = smallest i in S such that the weights of S up to i exceed u[r] times
 *               the weight of S (by rising i);
 *   probs[r, i] = w_i / weight of S in S, 0 elsewhere.
 * T = 0 takes the first of the largest logits (probs 1 there).  With probs as target_probs
 * or draft_probs of dflash_verify blocks are verified against the filtered distribution.
 *   logits [N, V] of dtype, rows logits_stride elements apart (0: V); u [N] fp32 in
 *   [0, 1); temperature, top_p, min_p [N] fp32 and top_k [N] int32, each nullable (1, 1, 0, 0);
 *   tokens [N] int32; probs [N, V] fp32, nullable, rows probs_stride elements apart (0: V);
 *   probs may be the fp32 logits themselves.
 * A logit below -2^126 (-inf, a type's lowest value: a masked token) and NaN are no
 * choice; one above 2^126 counts as 2^126.
 * A row without a choice, and one whose temperature is negative, infinite or NaN, is
 * recorded as DFLASH_ERR_INVALID and gets token 0 and probs 0.  NaN in top_p or min_p
 * leaves the filter out; a temperature below 2^-100 counts as 2^-100.
 * Weights are held in steps of 2^-44 of the largest and added up as whole numbers: the
 * result does not depend on the order of the sums.  A w below 2^-45 counts as zero in them;
 * its probability is still written, u = 0 draws the first token of S whatever it weighs, and a
 * beginning that meets top_p exactly falls short of it where such tokens follow.  V up to
 * DFLASH_SAMPLE_MAX_V.
 */
#define DFLASH_SAMPLE_MAX_V 393216
typedef struct {
  int N;  /* rows */
  int V;  /* vocabulary */
  int64_t logits_stride, probs_stride; /* elements from row to row; 0: V */
} dflash_sample_dims_t;
DFLASH_API dflash_status_t dflash_sample(const dflash_sample_dims_t* dims, dflash_dtype_t dtype, const void* logits,
                                         const float* u, const float* temperature, const int32_t* top_k,
                                         const float* top_p, const float* min_p, int32_t* tokens, float* probs,
                                         dflash_stream_t stream);

/*
 * The walk down a drafted tree.  Request r's nodes [q_offsets[r], q_offsets[r+1]) (see
 * dflash_attn_tree; node 0, the last token that was accepted before, is accepted) carry
 * tokens, and sampled[t] is the token drawn from the target's logits behind node t.  From
 * node 0 on: of the current node's children the first one with tokens[child] =
 * sampled[current] is accepted and becomes the current one; where there is none the walk
 * ends, as it does with max_path nodes.
 *   path [R, max_path]: the accepted nodes' indexes in the request, 0 first, then -1;
 *   out_tokens [R, max_path]: sampled[] along the path, then -1: the accepted children's
 *     tokens and behind them the new one;
 *   num_accepted [R]: nodes of the path (0 for a request without nodes).
 * A child has to come behind its parent; other entries of parents name no parent.  A
 * request whose offsets are out of range or which has more than DFLASH_TREE_MAX_NODES
 * nodes is recorded as DFLASH_ERR_INVALID and gets num_accepted = 0.
 */
#define DFLASH_TREE_MAX_NODES 4096
typedef struct {
  int R;         /* requests */
  int total;     /* rows of the packed node axis (>= q_offsets[R]) */
  int max_path;  /* columns of path and out_tokens */
} dflash_accept_dims_t;
DFLASH_API dflash_status_t dflash_tree_accept(const dflash_accept_dims_t* dims, const int32_t* sampled,
                                              const int32_t* tokens, const int32_t* parents,
                                              const int32_t* q_offsets, int32_t* path, int32_t* out_tokens,
                                              int32_t* num_accepted, dflash_stream_t stream);

/*
 * Moving keys and values within a paged cache, in all layers at once: k_cache and
 * v_cache [L, num_pages, page_size, H_kv, D], layers k_layer_stride / v_layer_stride elements
 * apart (0: contiguous), all of one page table.
 */
typedef struct {
  int L;  /* layers */
  int64_t k_layer_stride, v_layer_stride; /* elements from layer to layer; 0: contiguous */
} dflash_layers_t;

/*
 * The accepted nodes of a step moved together: with a = num_accepted[r] and L - n the
 * position of the request's first new token, the keys and values of position
 * L - n + path[r, j] go to position L - n + j, j < a, and new_lens[r] = L - n + a.
 * (new_lens does not overlap kv_lens: other caches are still to be moved by the old lengths.)
 *   path [R, max_path]: rising indexes below n, as dflash_tree_accept writes them.
 * A request whose offsets, length, count or path are out of range is recorded as
 * DFLASH_ERR_INVALID and left as it is (new_lens = kv_lens); a row whose page id is out
 * of range is recorded and not moved.  The positions moved must not lie in pages that
 * other requests share.  H_q and max_q_len are not read.
 */
DFLASH_API dflash_status_t dflash_cache_compact(const dflash_paged_dims_t* dims, const dflash_layers_t* layers,
                                                dflash_dtype_t dtype, const int32_t* page_table,
                                                const int32_t* kv_lens, const int32_t* q_offsets, const int32_t* path,
                                                int max_path, const int32_t* num_accepted, void* k_cache,
                                                void* v_cache, int32_t* new_lens, dflash_stream_t stream);

/*
 * Pages copied: the first rows[i] positions (null: all) of page src[i] to page dst[i],
 * i < n, as dflash_pages_fork asks for.  A pair with -1 in it is left out; one with another
 * id outside [0, num_pages), or rows outside [0, page_size], is recorded as
 * DFLASH_ERR_INVALID and left out.  A page is the dst of one pair at most, and then the
 * src of none.  Of dims H_kv, D, num_pages, page_size and the page strides are read.
 */
DFLASH_API dflash_status_t dflash_cache_copy(const dflash_paged_dims_t* dims, const dflash_layers_t* layers,
                                             dflash_dtype_t dtype, int n, const int32_t* src, const int32_t* dst,
                                             const int32_t* rows, void* k_cache, void* v_cache,
                                             dflash_stream_t stream);

/*
 * The pages of a cache handed out on the device.  refs [num_pages] int32 counts for every
 * page the rows of page_table [R, max_pages] that hold it; a page with 0 is free.  (All 0
 * and all lengths 0 at the beginning.)  Free pages are taken lowest first.
 *   missing [1] int32: written; how many pages could not be had.  The table entries that
 *     would have held them are -1, which giving them back passes over.
 *   workspace: >= dflash_pages_workspace_size(dims) bytes, 256-byte aligned; needs no
 *     initialisation.
 * Calls on one pool must not run at the same time.  R and the number of forks up to
 * DFLASH_POOL_MAX_ROWS, R * max_pages below 2^31.
 */
#define DFLASH_POOL_MAX_ROWS 65536
typedef struct {
  int R;          /* rows of the page table */
  int max_pages;  /* its columns */
  int page_size;  /* positions of a page */
  int num_pages;  /* pages of the cache */
} dflash_pool_dims_t;
DFLASH_API size_t dflash_pages_workspace_size(const dflash_pool_dims_t* dims);

/*
 * Requests made shorter or longer: row r holds ceil(old_lens[r] / page_size) pages and is
 * to hold ceil(new_lens[r] / page_size).  All rows' pages that are too many are given back
 * first (their entries become -1), then rows that need more take them, by rising r.  Length 0
 * frees a request.  A request with a length outside [0, max_pages * page_size] is recorded
 * as DFLASH_ERR_INVALID and left as it is; an entry that is given back and is no page, or a
 * page that was free, is recorded.
 */
DFLASH_API dflash_status_t dflash_pages_resize(const dflash_pool_dims_t* dims, int32_t* page_table,
                                               const int32_t* old_lens, const int32_t* new_lens, int32_t* refs,
                                               int32_t* missing, void* workspace, size_t ws_bytes,
                                               dflash_stream_t stream);

/*
 * Requests forked: row dst[i], which has to be empty (lens 0), gets lens[src[i]] positions of
 * row src[i], i < n.  Whole pages are shared (their counts rise), for the rest in the
 * last page a page is taken, in the order of i; copy_src[i], copy_dst[i] and copy_rows[i]
 * say what dflash_cache_copy has to copy for it (-1, -1, 0 where the last page is whole).
 * lens [R] is updated.  A row may be the source of many forks.  A fork whose row or source
 * is out of range, whose row is not empty, is another fork's too or is some fork's source,
 * is recorded as DFLASH_ERR_INVALID and left out (-1, -1, 0); an entry of the source that
 * is no page is recorded, and the fork's is the same.  Positions in shared pages
 * must not be written; a row is not shortened into them and then appended to.
 */
DFLASH_API dflash_status_t dflash_pages_fork(const dflash_pool_dims_t* dims, int32_t* page_table, int32_t* lens, int n,
                                             const int32_t* src, const int32_t* dst, int32_t* refs, int32_t* copy_src,
                                             int32_t* copy_dst, int32_t* copy_rows, int32_t* missing, void* workspace,
                                             size_t ws_bytes, dflash_stream_t stream);

/*
 * Workspace bytes a call needs.  For DENSE/ANCHORED (and their _BACKWARD
 * modes) pass dims (dims->B, S, Q,
 * H, head dims) and ignore the ragged arguments; for RAGGED pass dims = NULL
 * and R, H, head dims via the ragged arguments.  Returns 0 on invalid input.
 */
DFLASH_API size_t dflash_attn_workspace_size(int mode, const dflash_dims_t* dims, dflash_dtype_t dtype,
                                  int R, int H, int d_nope, int d_rope, int d_v, int total_q,
                                  int total_kv, int max_q_len);

/*
 * Host builder of the anchored tile schedule (exported for tests).  anchors
 * [B, nb] int32 in HOST memory.  classes (host, uint8) receives
 * [B, ceil(Q/DFLASH_TILE_M), ceil((S+Q)/DFLASH_TILE_N)] tile classes
 * (DFLASH_TILE_*), computed from each tile's minimum and maximum anchor with
 * the same formula the kernels use.
 */
DFLASH_API dflash_status_t dflash_build_schedule_host(int B, int S, int Q, const int32_t* anchors, int nb,
                                           int block_size, uint8_t* classes);

/*
 * Device scan of a dense mask into tile classes (exported for tests): mask
 * [B,1,Q,S+Q] of dtype on the device, classes [B, ceil(Q/TILE_M),
 * ceil((S+Q)/TILE_N)] uint8 on the device.  An all-0 tile is FULL, an
 * all--inf tile SKIP, anything else PARTIAL.
 */
DFLASH_API dflash_status_t dflash_scan_mask(int B, int S, int Q, dflash_dtype_t dtype, const void* mask,
                                 uint8_t* classes, dflash_stream_t stream);

/*
 * Number of kernels this library has launched in the calling process since it
 * was loaded (all devices, all streams).  Diagnostic counter for benchmarks.
 */
DFLASH_API uint64_t dflash_kernel_launches(void);

/*
 * Builds the additive DFlash block mask of the anchored rule on the device:
 * mask [B, 1, Q, S+Q] of dtype gets 0 where row i (block j = i/block_size) may
 * attend -- context keys p < anchors[b, j] and the block_size noise keys of
 * block j -- and -inf everywhere else.  This is the dense mask the trainer
 * hands the draft (nemo_automodel.components.speculative.dflash.draft_kimi_k3
 * page, module docstring: the block structure is supplied entirely by the
 * attention mask; KimiK3DFlashAttention.forward: its shape).  anchors [B, nb]
 * int32 on the device; anchors outside [0, S] are clamped and recorded as
 * DFLASH_ERR_INVALID in the device error word.  Asynchronous on `stream`.
 */
DFLASH_API dflash_status_t dflash_build_mask(int B, int S, int Q, const int32_t* anchors, int nb, int block_size,
                                             dflash_dtype_t dtype, void* mask, dflash_stream_t stream);

/*
 * Test export: fault injection for the bounded-wait path.  Every mbarrier wait
 * of the tensor-core kernels (forward, split-context decode, latent decode and
 * backward) gives up after a budget -- 2 s unless set here -- records
 * DFLASH_ERR_TIMEOUT in the device error word, and the CTA winds down: its
 * issued TMA loads land, its issued MMAs complete, its TMEM is freed, and it
 * returns; the context stays usable.  This call sets, process-wide and for
 * every later call until it is called again:
 *   wait_budget_ns  budget of one wait (0 restores the 2 s default);
 *   stall_cta       the CTA (of each of those kernels) whose TMA producer
 *                   leaves its first work item's key tiles (the backward's
 *                   dk/dv kernel: query tiles) unloaded, so that the waits on
 *                   them run out (-1: none).  Other CTAs compute normally; the
 *                   stalled CTA's results are left unwritten or incomplete.
 * Not for production use; not synchronised with calls in flight.
 */
DFLASH_API void dflash_test_inject_stall(unsigned long long wait_budget_ns, int stall_cta);

/*
 * Test export: the backward kernels work out, once per CTA, which tiles of the
 * axis they loop over (dq: key tiles; dk/dv: query tiles) they need, and keep
 * these flags in a shared-memory table of 16384 entries; tiles past the table
 * are worked out when they come up.  This call caps the table at n entries
 * (n <= 0 restores the full table), process-wide for every later call, so that
 * tests reach the path past the table at small sizes.  Results do not depend
 * on n.  Not for production use; not synchronised with calls in flight.
 */
DFLASH_API void dflash_test_limit_tile_flags(int n);

/* Human-readable name of a status code (static storage). */
DFLASH_API const char* dflash_status_string(dflash_status_t status);

/*
 * Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns DFLASH_OK when no kernel recorded an error since the last
 * read, DFLASH_ERR_CUDA when the synchronisation itself failed.
 */
DFLASH_API dflash_status_t dflash_last_device_error(dflash_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_ATTN_H_ */
