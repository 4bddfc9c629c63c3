/*
 * bl_attn.h -- C ABI of libbl_attn.so: BackLite-style attention on GB300.
 *
 * Three calls make up the hot path, in this order:
 *
 *   bl_attn_fwd         exact attention forward that also records, for every
 *                       (query row, key tile), the log-sum-exp of that row's
 *                       scores over the tile ("BackLite" README, How It Works,
 *                       Phase 1; "Introducing BackLite", Using Sparsity).
 *   bl_mask_from_stats  turns those statistics into a block-sparse mask and
 *                       compacted tile lists (README, How It Works, Phase 2).
 *   bl_attn_bwd         attention backward that reads and computes nothing
 *                       for masked tiles ("Introducing BackLite",
 *                       Backpropagation for attention, and Using Sparsity).
 *
 * Tensors
 *   q, o, g_o, g_q : [B, n, H,  d] bf16 (batch, seq, head, dim), contiguous
 *                    unless bl_shape gives strides
 *   k, v, g_k, g_v : [B, n, Hk, d] bf16, likewise; query head h reads kv
 *                    head h / (H / Hk) (grouped-query attention, README,
 *                    Forward signature: key/value carry heads_k heads).
 *   lse            : [B, H, n] fp32, natural log: LSE_r = log sum_c exp(s q_r.k_c)
 *   tile_stats     : [B, H, T_c, T_r*block_q] fp32, key-tile major:
 *                    tile_stats[b,h,j,r] = log sum_{c in key tile j} exp(s q_r.k_c);
 *                    -inf where the tile's terms underflow and for rows r >= n.
 *   T_r = ceil(n / block_q), T_c = ceil(n / block_k).
 *
 * Every pointer is device memory owned by the caller; the library allocates
 * nothing and frees nothing.  Calls are asynchronous on the given stream
 * (a cudaStream_t passed as void*; NULL is the legacy default stream).
 * Arguments are validated on the host before any launch: a failing check
 * launches nothing and returns an error code.  Device pointers must be
 * 16-byte aligned.
 */
#ifndef BL_ATTN_H
#define BL_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BL_OK = 0,
  BL_ERR_INVALID_ARG = 1,    /* bad shape, pointer, alignment or parameter   */
  BL_ERR_UNSUPPORTED = 2,    /* valid but not built (e.g. head_dim 96)       */
  BL_ERR_CUDA = 3,           /* a CUDA runtime call or launch failed         */
  BL_ERR_WORKSPACE = 4,      /* workspace missing or too small               */
  BL_ERR_CORRUPT_LISTS = 5,  /* a tile list held an out-of-range entry       */
  BL_ERR_TIMEOUT = 6         /* a bounded device-side wait ran out           */
} bl_status;

/* Problem shape.  d in {64, 128}; block_q, block_k in {64, 128}; H % Hk == 0;
 * n >= 1.  One shape describes the forward, the mask and the backward: the
 * statistics, the mask and the backward all use the same block_q x block_k
 * tiles.
 *   causal  0: every query attends to every key; 1: query r attends to keys
 *           c <= r.
 *   window  0: no limit; W > 0 (needs causal = 1): query r attends to keys
 *           r - W < c <= r, the sliding windows the BackLite blog trains
 *           Nanochat with ("Introducing BackLite", Training Nanochat).
 * causal/window need 128 x 128 tiles.  A tile with no attending (query, key)
 * pair has tile statistic -inf and is never kept by the mask. */
typedef struct {
  int B, n, H, Hk, d;
  int block_q, block_k;
  int causal, window;
  /* Element strides of the four BSHD dims [batch, seq, head, dim], for
   * tensors that are views of larger ones (a kv-head slice of a batch, a
   * fused QKV projection): q_strides for q and g_q, k_strides for k and g_k,
   * v_strides for v and g_v, o_strides for o and g_o.  All four entries 0
   * (what a zero-initialised struct holds) means contiguous BSHD.  Otherwise
   * the dim stride is 1, the others positive multiples of 8 (16 bytes), and
   * the head stride at least d.  The packed (varlen) calls take contiguous
   * tensors. */
  int64_t q_strides[4], k_strides[4], v_strides[4], o_strides[4];
} bl_shape;

/* Block-sparse tile lists of one backward, all device memory.
 *   mask   [B,H,T_r,T_c] uint8   1 = compute tile (i, j), 0 = skip
 *   kv_idx [B,H,T_r,T_c] int32   per query tile: active key tiles, ascending,
 *                                then -1 up to T_c
 *   kv_cnt [B,H,T_r]     int32   number of active key tiles per query tile
 *   q_idx  [B,H,T_c,T_r] int32   per key tile: active query tiles, ascending,
 *                                then -1 up to T_r
 *   q_cnt  [B,H,T_c]     int32   number of active query tiles per key tile
 *   nan_count            int32*  optional (may be NULL): the mask pass adds
 *                                the number of NaN tile weights it met (such
 *                                tiles are kept).  The caller zeroes it.
 * The mask is per query head: the heads of one GQA group each have their own
 * lists ("BackLite" README, Key properties: sparsity per sample, per head). */
typedef struct {
  uint8_t* mask;
  int32_t* kv_idx;
  int32_t* kv_cnt;
  int32_t* q_idx;
  int32_t* q_cnt;
  int32_t* nan_count;
} bl_lists;

/* Number of fp32 elements of tile_stats: B*H*T_c*T_r*block_q. */
size_t bl_tile_stats_elems(const bl_shape* shape);

/* Element counts of the five list arrays of bl_lists, written to out[0..4]
 * in field order: mask and kv_idx B*H*T_r*T_c each, kv_cnt B*H*T_r, q_idx
 * B*H*T_c*T_r, q_cnt B*H*T_c.  Returns the total bytes of the five arrays
 * (uint8 mask, int32 others), or 0 for an invalid shape (out untouched). */
size_t bl_lists_elems(const bl_shape* shape, size_t out[5]);

/* Bytes of device workspace bl_attn_bwd needs (16-byte aligned base):
 * D = rowsum(G_O * O) [B,H,n] fp32, the fp32 dQ accumulator [B,n,H,d], with
 * 64-wide tiles the tile lists regrouped into 128 x 128 tiles, a device
 * status word and the backward kernel's work-item counter.  The call
 * initialises all of it, so the workspace needs no clearing between calls;
 * two calls in flight at the same time must not share one. */
size_t bl_bwd_workspace_bytes(const bl_shape* shape);

/* Exact attention forward ("Introducing BackLite", Backpropagation for
 * attention: S = s Q K^T, P = softmax_row(S), O = P V; the forward is not
 * approximated, Using Sparsity).
 *   scale       softmax scale s (finite, > 0); 1/sqrt(d) is the usual value.
 *   o, lse      outputs (layouts above).
 *   tile_stats  output, or NULL to skip recording the statistics (the
 *               negl_prob = 0 path: README, Key properties, zero forward
 *               overhead when nothing will be skipped).
 * Errors: BL_ERR_INVALID_ARG (shape, pointers, alignment, scale),
 *         BL_ERR_UNSUPPORTED (d or tile size), BL_ERR_CUDA (launch). */
bl_status bl_attn_fwd(const bl_shape* shape, const void* q, const void* k,
                      const void* v, float scale, void* o, float* lse,
                      float* tile_stats, void* stream);

/* Tile selection (README, How It Works, Phase 2; Key properties).  For
 * every (b, h, query tile i) and key tile j:
 *   d_ij = max over rows r < n of tile i of fp32(tile_stats[b,h,j,r] - lse[b,h,r]),
 *          clamped to <= 0, so w_ij = exp(d_ij) bounds the weight any row of
 *          the tile puts on key tile j;
 *   E_ij = ceil(detexp(d_ij) * 2^40), a 40-bit fixed-point weight (detexp is
 *          an exp evaluated by a fixed sequence of round-to-nearest fp32
 *          operations, so every implementation gets the same integers);
 *   the key tiles are ordered by (d ascending, j ascending) and the longest
 *   prefix whose integer running sum stays below ceil(negl_prob * 2^40) is
 *   skipped.  negl_prob = 0 skips nothing.
 * Writes every field of *lists (layouts above).
 * Errors: BL_ERR_INVALID_ARG (negl_prob outside [0, 1), null pointers),
 *         BL_ERR_UNSUPPORTED (T_c > 2048), BL_ERR_CUDA. */
bl_status bl_mask_from_stats(const bl_shape* shape, const float* tile_stats,
                             const float* lse, double negl_prob,
                             const bl_lists* lists, void* stream);

/* ---------------------------------------------------------------------------
 * Tile weights reduced in the forward.
 *
 * The statistics hold n * T_c floats per head (17 GB at n = 131072 with 32
 * heads), and the mask pass reads all of them.  The forward can instead
 * reduce them itself, right after a query tile's last key tile, into the
 * per-(query tile, key tile) log-weights the selection rule starts from
 * ("BackLite" README, How It Works, Phase 2: p_tile = exp(LSE_tile - LSE_row);
 * "Introducing BackLite", Training Nanochat, reports the stored statistics at
 * about 1% of peak memory):
 *   tile_logw : [B, H, T_r, T_c] fp32,
 *               tile_logw[b,h,i,j] = d_ij = max over rows r < n of query tile
 *               i of fp32(tile_stats[b,h,j,r] - lse[b,h,r]) (NaN if any term
 *               is NaN), clamped to <= 0 with -0 stored as +0; key tiles that
 *               no row of the tile attends (causal / window) enter with
 *               tile_stats = -inf.  This is exactly the d_ij of
 *               bl_mask_from_stats, bit for bit.
 * Tiles of 64 or 128 on either side, T_c <= 2048.
 * ------------------------------------------------------------------------- */

/* Bytes of scratch bl_attn_fwd_tile_weights needs when tile_stats is NULL:
 * one slot of 260 * T_c floats for every forward CTA that can be resident on
 * the CURRENT device at once (about 152 * 260 * T_c * 4 bytes on a GB300:
 * 40 MB at T_c = 256, 162 MB at T_c = 1024), plus one lock word per slot.
 * 0 for an invalid or unsupported shape. */
size_t bl_fwd_workspace_bytes(const bl_shape* shape);

/* bl_attn_fwd that also writes tile_logw (above).
 *   tile_stats  the statistics output as in bl_attn_fwd, or NULL: then the
 *               statistics rows live only in `workspace` (at least
 *               bl_fwd_workspace_bytes, 16-byte aligned), one slot per
 *               resident CTA, and are not returned.  Two calls in flight at
 *               the same time must not share a workspace.  workspace may be
 *               NULL when tile_stats is given.
 * O, LSE and tile_stats are the same as bl_attn_fwd's, and tile_logw does not
 * depend on whether tile_stats is given.
 * Errors: as bl_attn_fwd; BL_ERR_UNSUPPORTED (T_c > 2048);
 *         BL_ERR_WORKSPACE (tile_stats NULL and the workspace missing or
 *         too small). */
bl_status bl_attn_fwd_tile_weights(const bl_shape* shape, const void* q, const void* k,
                                   const void* v, float scale, void* o, float* lse,
                                   float* tile_stats, float* tile_logw, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* bl_mask_from_stats from the tile weights: the same lists, bit for bit, as
 * bl_mask_from_stats on the statistics and LSE the weights were reduced from,
 * reading T_r * T_c floats per head instead of n * T_c.
 * Errors: as bl_mask_from_stats. */
bl_status bl_mask_from_tile_weights(const bl_shape* shape, const float* tile_logw,
                                    double negl_prob, const bl_lists* lists, void* stream);

/* Masked attention backward ("Introducing BackLite", Backpropagation for
 * attention and Using Sparsity), with M the element mask expanded from
 * lists->mask and P recomputed from the full-row lse:
 *   D = rowsum(G_O * O), P^ = P * M, G_V = P^T G_O, G_P = G_O V^T,
 *   G_S = P^ * (G_P - D), G_Q = s G_S K, G_K = s G_S^T Q
 * (kv-head gradients sum over the query heads of their group).  Tiles not
 * in the lists are neither loaded nor computed.  lists == NULL runs the
 * dense backward (every tile).  Only q_idx/q_cnt of the lists are read.
 *   workspace  device buffer of at least bl_bwd_workspace_bytes(shape).
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_WORKSPACE,
 *         BL_ERR_CUDA.  A list entry outside [0, T_r) (or a count outside
 *         [0, T_r]) is skipped on the device and recorded in the status word;
 *         bl_bwd_check_status reports it as BL_ERR_CORRUPT_LISTS. */
bl_status bl_attn_bwd(const bl_shape* shape, const void* q, const void* k,
                      const void* v, const void* o, const void* g_o,
                      const float* lse, float scale, const bl_lists* lists,
                      void* g_q, void* g_k, void* g_v, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Synchronises the stream and reads the status word a previous bl_attn_bwd
 * left in this workspace: BL_OK, BL_ERR_CORRUPT_LISTS, or BL_ERR_TIMEOUT (a
 * bounded device-side wait gave up; the outputs of that call are invalid). */
bl_status bl_bwd_check_status(const bl_shape* shape, const void* workspace,
                              void* stream);

/* LSE-combine ("BackLite" README, Key properties: the LSE output serves to
 * combine partial attention results).  Given `parts` results of the same
 * queries over disjoint key sets,
 *   o_parts   [parts, B, n, H, d] bf16   (each part laid out like o)
 *   lse_parts [parts, B, H, n]    fp32   (each part laid out like lse)
 * writes LSE = log sum_p exp(LSE_p) and O = sum_p exp(LSE_p - LSE) O_p into
 * o [B, n, H, d] bf16 and lse [B, H, n] fp32.  A part whose LSE is -inf (it
 * saw no key) carries no weight; a row with no finite part gets O = 0 and
 * LSE = -inf.  parts in [1, 32], d in {64, 128}.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_CUDA. */
bl_status bl_lse_combine(int parts, int B, int n, int H, int d, const void* o_parts,
                         const float* lse_parts, void* o, float* lse, void* stream);

/* Error statistics of a gradient against a reference, for choosing negl_prob
 * ("Introducing BackLite", Using Sparsity: the sparse backward is judged by
 * the cosine similarity and relative L2 error of its gradients against the
 * dense backward, and the post proposes tuning negl_prob to a target on
 * them).  a and b: n bf16 values each (device, 16-byte aligned), b the
 * reference.  out: 4 doubles of device memory (8-byte aligned), overwritten
 * with
 *   out[0] = sum (a - b)^2,  out[1] = sum b^2,  out[2] = sum a*b,  out[3] = sum a^2
 * so rel-L2 = sqrt(out[0] / out[1]) and cos = out[2] / sqrt(out[1] * out[3]).
 * Asynchronous on the stream.  Errors: BL_ERR_INVALID_ARG, BL_ERR_CUDA. */
bl_status bl_grad_error(const void* a, const void* b, size_t n, double* out, void* stream);

/* Size of the fixed device scratch array behind bl_attn_bwd_noalloc: 32 MiB
 * on every GPU that loads the library, held until the process exits. */
#define BL_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/* bl_attn_bwd without a workspace argument, for callers that cannot allocate
 * device memory themselves (for instance a host runtime that owns every byte
 * of device memory through its own pool, or a latency-critical caller that
 * cannot afford cudaMalloc's implicit synchronisation).  The BackLite pages
 * have no counterpart: this is a deployment convenience of this library.
 *
 * Same arguments, results and errors as bl_attn_bwd, except that the
 * scratch (D, the fp32 dQ accumulator, the status word) lives in a fixed
 * file-scope device array of BL_NOALLOC_SCRATCH_BYTES.  The call allocates
 * nothing.  A shape whose bl_bwd_workspace_bytes exceeds that size is
 * rejected with BL_ERR_WORKSPACE before any launch.  The first call on each
 * device looks the array's device address up (cudaGetSymbolAddress) with that
 * device current; make that first call before any stream capture.  All calls
 * share the one array and it keeps the last call's contents (each call
 * clears what must start at zero), so calls that overlap on the GPU -- on
 * different streams, or from different threads -- race and must be
 * serialised by the caller.  List entries out of range are skipped exactly
 * as in bl_attn_bwd and recorded in a status word inside the array, which
 * bl_bwd_noalloc_check_status reads back. */
bl_status bl_attn_bwd_noalloc(const bl_shape* shape, const void* q, const void* k,
                              const void* v, const void* o, const void* g_o,
                              const float* lse, float scale, const bl_lists* lists,
                              void* g_q, void* g_k, void* g_v, void* stream);

/* bl_bwd_check_status for bl_attn_bwd_noalloc: synchronises the stream and
 * reads the status word the last bl_attn_bwd_noalloc call with this shape
 * left in the fixed scratch array of the current device: BL_OK,
 * BL_ERR_CORRUPT_LISTS, or BL_ERR_TIMEOUT (a bounded device-side wait gave
 * up; that call's outputs are invalid).  Allocates nothing.  A later call
 * with another shape moves the word, so read it before the next call. */
bl_status bl_bwd_noalloc_check_status(const bl_shape* shape, void* stream);

/* ---------------------------------------------------------------------------
 * Around the attention: rotary positions, the root-mean-square norm with the
 * residual's addition, and activations held in 8 bits until the backward.
 * (The BackLite pages have no counterpart: these are the steps a training
 * block runs directly before the attention, and what it keeps meanwhile.)
 *
 * Rows.  The norm and the 8-bit calls see a tensor as [rows, cols] with a
 * contiguous last dim; a row stride (in elements, >= cols) is taken where an
 * argument gives one, every other tensor is contiguous.  rows = 0 is allowed
 * and reads and writes no row.  Pointers need the alignment of their element
 * only; 16-byte aligned rows of a multiple of 8 elements run on vector loads.
 * Outputs must not overlap inputs unless a call says so.
 * ------------------------------------------------------------------------- */
typedef enum { BL_BF16 = 0, BL_FP16 = 1, BL_FP32 = 2 } bl_dtype;
typedef enum { BL_INT8 = 1, BL_E4M3 = 2 } bl_format8;

/* A [rows, cols] tensor in 8 bits: one fp32 scale for every `group`
 * consecutive elements of a row (32, 64 or 128; the last group of a row may
 * be cut), or one a row (group = 0).
 *   scale = amax * fl32(1 / qmax), at least 2^-126 and at most the largest number
 *           whose product with qmax is finite; qmax = 127 (int8) or 448 (e4m3)
 *   code  = round to nearest even of fl32(x * fl32(1 / scale))
 *   value = code * scale
 * A group that holds a NaN or an infinity gets the scale NaN and loads as NaN.
 *   codes  [rows, cols]  int8 or e4m3, contiguous
 *   scales [rows, ceil(cols / group)] fp32 ([rows] with group = 0) */
typedef struct {
  void* codes;
  float* scales;
  int format;               /* bl_format8 */
  int group;
} bl_act8;

/* x [rows, cols] (dtype, row stride x_stride) into codes and scales.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_CUDA. */
bl_status bl_act_save(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                      const bl_act8* out, void* stream);

/* The values of codes and scales, rounded to dtype, into x [rows, cols]
 * (contiguous).  Errors: BL_ERR_INVALID_ARG, BL_ERR_CUDA. */
bl_status bl_act_load(int64_t rows, int64_t cols, int dtype, const bl_act8* in, void* x,
                      void* stream);

/* Largest number of columns of the norm. */
#define BL_NORM_MAX_COLS 16384

/* h = x + residual (h = x without one), rstd = 1 / sqrt(mean(h^2) + eps),
 * y = h * rstd * weight, row by row.
 *   x, residual   [rows, cols] of dtype, row strides x_stride, residual_stride;
 *                 residual may be NULL.
 *   weight        [cols] of weight_dtype (dtype or BL_FP32), or NULL: ones.
 *   y             [rows, cols] of dtype, or NULL when y8 is given.
 *   h             [rows, cols] of dtype, h rounded: the residual stream behind
 *                 the addition.  May be NULL; NULL without a residual.
 *   rstd          [rows] fp32, for the backward; may be NULL.
 *   y8            y in 8 bits (from y before its rounding to dtype), beside y
 *                 or in its place; may be NULL.
 * y and y8 come from the unrounded h.  eps >= 0, cols <= BL_NORM_MAX_COLS.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED (cols), BL_ERR_CUDA. */
bl_status bl_rms_norm_fwd(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                          const void* residual, int64_t residual_stride, const void* weight,
                          int weight_dtype, float eps, void* y, void* h, float* rstd,
                          const bl_act8* y8, void* stream);

/* Bytes of device workspace bl_rms_norm_bwd needs when it forms g_w (16-byte
 * aligned base; the call initialises it). */
size_t bl_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);

/* Gradients of bl_rms_norm_fwd.  With u = h rstd and c = mean(weight g_y u):
 *   g_x = rstd (weight g_y - u c) + g_h     (of x and of the residual alike)
 *   g_w = sum over the rows of g_y u        (in a fixed order: reproducible)
 *   g_y, g_h, g_x [rows, cols] of dtype; g_h, the gradient that reaches h along
 *                 the residual stream, may be NULL.
 *   h, h8         h as the forward wrote it (x without a residual), or its
 *                 8-bit checkpoint, which is read as it is: exactly one of both.
 *   rstd          [rows] fp32 from the forward.
 *   g_w           [cols] of weight_dtype, or NULL; then no workspace is needed.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_WORKSPACE, BL_ERR_CUDA. */
bl_status bl_rms_norm_bwd(int64_t rows, int64_t cols, int dtype, const void* g_y, const void* h,
                          const bl_act8* h8, const float* rstd, const void* weight,
                          int weight_dtype, const void* g_h, void* g_x, void* g_w,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Rotary positions with up to four axes (one: the ordinary rotation; three:
 * time, height and width of a video grid), on q and k in one launch.
 * The first 2 * pairs dimensions of every head turn in pairs, the others pass
 * through.  The pairs are dealt to the axes in consecutive sections
 * (sections[0..axes) >= 1, their sum is `pairs`); pair p of axis a turns by
 * positions[token][a] * f_p:
 *   (u, v) -> (u cos - v sin, u sin + v cos),
 *   (u, v) = (x[2p], x[2p+1]) with interleaved = 1, (x[p], x[p+pairs]) with 0.
 * inverse = 1 turns back: applied to the gradients of the outputs it gives
 * those of the inputs.
 *   q, q_out  [B, n, H, d] of dtype, k, k_out [B, n, Hk, d]; Hk = 0: no k.
 *             Element strides {batch, token, head}, the dim stride is 1.
 *             q_out may be q itself (with the same strides), likewise k_out.
 *             q_out's strides, sorted, each span the dims behind (as those of any
 *             slice or permutation of a dense tensor do), likewise k_out's;
 *             q_out and k_out must not share elements: refused where their
 *             batch and token strides are alike, else up to the caller.
 *   positions [B, n, axes] int32, contiguous: positions_batch_stride is n * axes,
 *             or 0 for [n, axes] that all batches share.
 *   freqs     [pairs] uint64 on the device: round(f_p / (2 pi) * 2^64) modulo
 *             2^64, f_p in radians a position.
 * 1 <= pairs <= d / 2, (H + Hk) * d < 2^31.  Errors: BL_ERR_INVALID_ARG, BL_ERR_CUDA. */
typedef struct {
  int B, n, H, Hk, d, pairs, axes;
  int sections[4];
  int interleaved, inverse, dtype;
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_strides[3], k_strides[3], q_out_strides[3], k_out_strides[3];
  const int32_t* positions;
  int64_t positions_batch_stride;
  const uint64_t* freqs;
} bl_rope_args;
bl_status bl_rope(const bl_rope_args* args, void* stream);

/* bl_attn_bwd from an 8-bit checkpoint: q, k and v come as codes with one
 * scale a (token, head) (group 0 over rows of d: q8->codes [B,n,H,d],
 * q8->scales [B,n,H]) and stand for their values rounded to bf16; o comes
 * either in bf16 (o) or as codes (o8), exactly one of both.  All codes have
 * the same format.  Contiguous tensors only (zero strides in the shape).
 * Up to 64 tokens P and dS enter their products within 2^-16 of their values,
 * beyond as bf16, as in bl_attn_bwd.
 * The workspace begins with bl_attn_bwd's, so bl_bwd_check_status reads it. */
size_t bl_attn_bwd_act8_workspace_bytes(const bl_shape* shape);
bl_status bl_attn_bwd_act8(const bl_shape* shape, const bl_act8* q8, const bl_act8* k8,
                           const bl_act8* v8, const void* o, const bl_act8* o8, const void* g_o,
                           const float* lse, float scale, const bl_lists* lists, void* g_q,
                           void* g_k, void* g_v, void* workspace, size_t workspace_bytes,
                           void* stream);

/* ---------------------------------------------------------------------------
 * The linear layers around the attention: products of e4m3 codes with a scale
 * for each block of 128, the layer norm, and dropout whose mask is never stored.
 * (These too have no counterpart in the BackLite pages.)  Rows, strides and
 * alignment as above.
 * ------------------------------------------------------------------------- */

/* x [rows, cols] (dtype, row stride x_stride) in e4m3, in one reading, with the
 * format of bl_act8 and one scale for every
 *   128 elements of a row      row_codes,   row_scales [rows, ceil(cols / 128)]
 *                              (what bl_act_save gives with group 128)
 *   128 elements of a column   col_codes,   col_scales [ceil(rows / 128), cols]
 *   128 x 128 elements         block_codes, block_scales [ceil(rows / 128), ceil(cols / 128)]
 * (groups at the ends may be cut).  Codes are [rows, cols] with the row strides
 * given; NULL codes are not wanted.  At least one of the three, and not both
 * columns and blocks.  Bytes behind the columns stay as they were.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED (2^31 tiles of 128 x 128 and more),
 * BL_ERR_CUDA. */
typedef struct {
  int64_t rows, cols, x_stride, row_stride, col_stride, block_stride;
  const void* x;
  void* row_codes;
  float* row_scales;
  void* col_codes;
  float* col_scales;
  void* block_codes;
  float* block_scales;
  int dtype;
} bl_tile8_args;
bl_status bl_tile8_save(const bl_tile8_args* args, void* stream);

/* The values of codes [rows, cols] (row stride `stride`) with scales for 128
 * elements of a column (blocks = 0) or for 128 x 128 (blocks = 1), rounded to
 * dtype, into x [rows, cols] (contiguous). */
bl_status bl_tile8_load(int64_t rows, int64_t cols, int dtype, const void* codes, int64_t stride,
                        const float* scales, int blocks, void* x, void* stream);

/* The products of a linear layer y = x w^T, x [tokens, in], w [out, in], of values
 * held as e4m3 codes:
 *   form            a                           b                       out
 *   BL_MATMUL8_Y    x   scales of rows          w  scales of blocks     y   [tokens, out]
 *   BL_MATMUL8_G_X  g_y scales of rows          w  scales of blocks     g_x [tokens, in]  = g_y w
 *   BL_MATMUL8_G_W  g_y scales of columns       x  scales of columns    g_w [out, in]     = g_y^T x
 * Scales are laid out as bl_tile8_save's, contiguous; codes have row strides.
 * Products of codes are summed in fp32 over blocks of 128 of the summed dim, and
 * the blocks' sums, times the product of their two scales, in fp32 in the blocks'
 * order (in a few parts of it, each in order, where few tiles share a sum); the
 * result is rounded once, to out_dtype.  The product of two scales is an fp32
 * number: below 2^-126 it loses bits, beyond 2^128 it is infinite, and the block's
 * part too, or NaN where its codes' products sum to 0.  A block whose scale is NaN
 * makes what it reaches NaN.  tokens = 0 gives g_w = 0.
 * Where a code tensor's rows are not 16-byte aligned, the call copies it to the
 * workspace first (bl_matmul8_workspace_bytes, which reads everything but `out`
 * and the workspace; 16-byte aligned).  When a device-side wait gives up
 * (bl_set_wait_limit), the tiles that it left are NaN.
 * Errors: BL_ERR_INVALID_ARG, BL_ERR_UNSUPPORTED, BL_ERR_WORKSPACE, BL_ERR_CUDA. */
typedef enum { BL_MATMUL8_Y = 0, BL_MATMUL8_G_X = 1, BL_MATMUL8_G_W = 2 } bl_matmul8_form;
typedef struct {
  int64_t tokens, out_features, in_features;
  const void* a_codes;
  const float* a_scales;
  int64_t a_stride;
  const void* b_codes;
  const float* b_scales;
  int64_t b_stride;
  void* out;                 /* contiguous */
  void* workspace;
  size_t workspace_bytes;
  int form, out_dtype;
} bl_matmul8_args;
size_t bl_matmul8_workspace_bytes(const bl_matmul8_args* args);
bl_status bl_matmul8(const bl_matmul8_args* args, void* stream);

/* Layer norm: h = x + residual (h = x without one), m = mean(h),
 * rstd = 1 / sqrt(mean((h - m)^2) + eps), y = (h - m) rstd weight + bias, row by
 * row.  Arguments as bl_rms_norm_fwd's; weight and bias [cols] have the same type,
 * either may be NULL (ones, zeros); mean and rstd [rows] fp32 for the backward may
 * be NULL.  The squares are summed of distances from a mean of some of the row's
 * elements and put right, so a row far from zero loses nothing by it. */
typedef struct {
  int64_t rows, cols, x_stride, residual_stride;
  const void* x;
  const void* residual;
  const void* weight;
  const void* bias;
  void* y;
  void* h;
  float* mean;
  float* rstd;
  const bl_act8* y8;
  float eps;
  int dtype, weight_dtype;
} bl_layer_norm_args;
bl_status bl_layer_norm_fwd(const bl_layer_norm_args* args, void* stream);

/* Its gradients.  With u = (h - m) rstd and c = mean(weight g_y u):
 *   g_x = rstd (weight g_y - mean(weight g_y) - u c) + g_h
 *   g_w = sum over the rows of g_y u,  g_b = sum over the rows of g_y
 * (in a fixed order: reproducible).  Arguments as bl_rms_norm_bwd's; g_w and g_b
 * have weight_dtype, either may be NULL, and without both no workspace is needed. */
size_t bl_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t cols);
typedef struct {
  int64_t rows, cols;
  const void* g_y;
  const void* h;
  const bl_act8* h8;
  const float* mean;
  const float* rstd;
  const void* weight;
  const void* g_h;
  void* g_x;
  void* g_w;
  void* g_b;
  void* workspace;
  size_t workspace_bytes;
  int dtype, weight_dtype;
} bl_layer_norm_bwd_args;
bl_status bl_layer_norm_bwd(const bl_layer_norm_bwd_args* args, void* stream);

/* Dropout: y = x / (1 - p) where an element is kept, else 0, plus the residual
 * (may be NULL).  Element i = row * cols + col, whatever the strides, is kept iff
 * word i mod 4 of Philox4x32-10 of the counter (i / 4, offset), two 64-bit numbers,
 * lower words first, and the key `seed` is at least round(p * 2^32); with p = 1 none is.
 *   state  {seed, offset}, two int64 on the device, read when the kernel runs
 *   y      [rows, cols] of dtype, contiguous; may be x or residual where that is too
 * What is dropped gives 0 whatever x is, infinities and NaN too.  The gradient is
 * the same call on g_y, without a residual.  rows * cols up to 2^42. */
bl_status bl_dropout(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                     const void* residual, int64_t residual_stride, double p,
                     const int64_t* state, void* y, void* stream);

/* used = state, and then state's offset one on: the generator's next call, in stream
 * order, so that a captured graph draws anew with every replay.  Calls that share a
 * state must not overlap. */
bl_status bl_dropout_next(int64_t* state, int64_t* used, void* stream);

/* ---------------------------------------------------------------------------
 * Packed variable-length batches.
 *
 * nseq sequences of lengths n_s = cu_seqlens[s+1] - cu_seqlens[s] are packed
 * back to back along the token axis; a query attends only to keys of its own
 * sequence.  The BackLite pages train on fixed-length batches and say
 * nothing about packing; this is the plain reading of packing: the result
 * for every sequence is exactly the result of the fixed-length call with
 * B = 1, n = n_s on that sequence alone, and every per-sequence array is
 * that call's array, stored one sequence after another.
 *
 * Tensors (total = cu_seqlens[nseq])
 *   q, o, g_o, g_q : [total, H,  d] bf16, contiguous
 *   k, v, g_k, g_v : [total, Hk, d] bf16, contiguous
 *   lse            : per sequence a [H, n_s] fp32 block, at element offset
 *                    H * cu_seqlens[s]
 *   tile_stats     : per sequence a [H, T_c(s), T_r(s)*block_q] fp32 block,
 *                    blocks back to back in sequence order
 *   lists          : each field per sequence a block laid out as the
 *                    fixed-length field with B = 1, blocks back to back;
 *                    nan_count is one counter for the whole batch
 * with T_r(s) = ceil(n_s / block_q), T_c(s) = ceil(n_s / block_k).
 * bl_varlen_layout gives every size.  A sequence of length 0 owns nothing
 * and launches nothing.
 *
 * Execution: the calls walk the sequences on the host and run the
 * fixed-length kernels once per run of consecutive sequences of equal
 * length (such a run is exactly a [count, n_s, ...] batch).  The runs are
 * spread over up to `streams` side streams of the library (largest run
 * first, each to the least-loaded stream), forked from and joined back to
 * the caller's stream with events, so that short sequences fill the GPU
 * together; the call returns with all its work ordered before anything the
 * caller enqueues next on its stream.  Nothing waits on the host, so the
 * calls can be captured in a CUDA graph.  The side streams belong to the
 * library, one set per device shared by every caller: packed calls on
 * different caller streams are serialised through them, and a packed call
 * made while another thread captures a packed call on the same device would
 * be recorded into that capture, so callers serialise packed calls that may
 * overlap a capture on one device.  lse only needs 4-byte alignment here;
 * the other device pointers need 16 bytes, as in the fixed-length calls.
 * ------------------------------------------------------------------------- */

/* cu_seqlens: HOST array of nseq + 1 int32, cu_seqlens[0] = 0,
 * non-decreasing, cu_seqlens[nseq] >= 1.  streams: most runs in flight at
 * once, 1..8, or 0 for the default of 8; 1 runs them one after another on
 * the caller's stream.  The other fields mean what they mean in bl_shape and
 * obey the same limits. */
typedef struct {
  int nseq;
  const int32_t* cu_seqlens;
  int H, Hk, d;
  int block_q, block_k;
  int causal, window;
  int streams;
} bl_varlen;

/* Element counts (bytes for bwd_workspace_bytes) of a packed batch. */
typedef struct {
  size_t total;                /* packed tokens                                  */
  size_t lse;                  /* fp32: H * total                                */
  size_t tile_stats;           /* fp32: sum_s H * T_c(s) * T_r(s) * block_q      */
  size_t mask;                 /* uint8 mask and int32 kv_idx: sum_s H*T_r*T_c   */
  size_t kv_cnt;               /* int32: sum_s H * T_r(s)                        */
  size_t q_idx;                /* int32: sum_s H * T_c(s) * T_r(s)               */
  size_t q_cnt;                /* int32: sum_s H * T_c(s)                        */
  size_t bwd_workspace_bytes;  /* workspace of bl_attn_bwd_varlen                */
  int groups;                  /* launches of each kernel per call               */
} bl_varlen_sizes;

/* Validates *varlen and fills *sizes.  Errors: BL_ERR_INVALID_ARG (bad
 * cu_seqlens or shape fields), BL_ERR_UNSUPPORTED (d or tile size). */
bl_status bl_varlen_layout(const bl_varlen* varlen, bl_varlen_sizes* sizes);

/* bl_attn_fwd over a packed batch (layouts above; tile_stats may be NULL). */
bl_status bl_attn_fwd_varlen(const bl_varlen* varlen, const void* q, const void* k,
                             const void* v, float scale, void* o, float* lse,
                             float* tile_stats, void* stream);

/* bl_mask_from_stats over a packed batch: the selection of every sequence
 * uses only that sequence's statistics.  BL_ERR_UNSUPPORTED when a sequence
 * has more than 2048 key tiles. */
bl_status bl_mask_from_stats_varlen(const bl_varlen* varlen, const float* tile_stats,
                                    const float* lse, double negl_prob,
                                    const bl_lists* lists, void* stream);

/* Tile weights over a packed batch: bl_attn_fwd_tile_weights on every
 * sequence.  tile_logw holds sizes.mask floats, each sequence's
 * [H, T_r, T_c] block where its mask block is (at the same element offset).
 * At most 2048 key tiles per sequence.  Without
 * tile_stats the statistics rows live in `workspace` (at least
 * bl_fwd_workspace_bytes_varlen, 16-byte aligned), whose slots every launch
 * group of the call shares.  Two calls in flight at the same time must not
 * share a workspace.
 * Errors: as bl_attn_fwd_varlen; BL_ERR_UNSUPPORTED (more than 2048 key
 *         tiles); BL_ERR_WORKSPACE. */
size_t bl_fwd_workspace_bytes_varlen(const bl_varlen* varlen);
bl_status bl_attn_fwd_tile_weights_varlen(const bl_varlen* varlen, const void* q, const void* k,
                                          const void* v, float scale, void* o, float* lse,
                                          float* tile_stats, float* tile_logw, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* bl_mask_from_stats_varlen from the tile weights: the same lists, bit for
 * bit, as from the statistics the weights were reduced from. */
bl_status bl_mask_from_tile_weights_varlen(const bl_varlen* varlen, const float* tile_logw,
                                           double negl_prob, const bl_lists* lists,
                                           void* stream);

/* bl_attn_bwd over a packed batch.  workspace: at least
 * sizes.bwd_workspace_bytes; every run has its own D and dQ areas and status
 * word in it. */
bl_status bl_attn_bwd_varlen(const bl_varlen* varlen, const void* q, const void* k,
                             const void* v, const void* o, const void* g_o,
                             const float* lse, float scale, const bl_lists* lists,
                             void* g_q, void* g_k, void* g_v, void* workspace,
                             size_t workspace_bytes, void* stream);

/* bl_bwd_check_status for bl_attn_bwd_varlen: synchronises the stream and
 * reports the worst status word of the call's runs (BL_ERR_TIMEOUT before
 * BL_ERR_CORRUPT_LISTS before BL_OK). */
bl_status bl_varlen_bwd_check_status(const bl_varlen* varlen, const void* workspace,
                                     void* stream);

/* Every device-side wait of the tcgen05 kernels (an mbarrier phase, a peer
 * warp's hand-off) is bounded: when one runs out the kernel records it (the
 * backward's status word: BL_ERR_TIMEOUT; the forward: NaN in the LSE rows it
 * could not finish), skips the rest of its work, waits with a fixed 2 s
 * limit for the copies and MMAs it already issued, frees its tensor memory
 * and ends, so the context stays usable.  This sets the limit for kernels
 * launched from now on, process-wide: seconds in [0, 2) (0 gives up on any
 * wait that is not already satisfied), anything else restores the default of
 * 2 s.  Returns the previous limit in seconds.  A diagnostic knob for testing
 * the failure path; calls racing with launches in other threads see either
 * value. */
double bl_set_wait_limit(double seconds);

/* Static description of a status code. */
const char* bl_status_string(bl_status status);

#ifdef __cplusplus
}
#endif

#endif /* BL_ATTN_H */
