// Host-side launchers of the bl_attn kernels (internal to libbl_attn.so).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bl {

struct Shape;

// Limit (ns of global time) the kernels launched now give every bounded
// device-side wait (bl_set_wait_limit; 2 s by default).
uint64_t wait_limit_ns();

// Forward + optional tile statistics (stats == nullptr skips them).
cudaError_t launch_fwd(const Shape& sh, const void* q, const void* k, const void* v, void* o,
                       float* lse, float* stats, float scale, cudaStream_t st);

// Tile selection: per-query-tile mask row, kv list and count, then the
// transposed per-key-tile q list and count.  From the statistics and the
// LSE, or (stats == nullptr) from the tile weights logw [B,H,T_r,T_c].
cudaError_t launch_mask(const Shape& sh, const float* stats, const float* lse,
                        const float* logw, unsigned long long threshold, uint8_t* mask,
                        int32_t* kv_idx, int32_t* kv_cnt, int32_t* q_idx, int32_t* q_cnt,
                        int32_t* nan_count, cudaStream_t st);

// Backward.  q_idx/q_cnt == nullptr runs every tile.  ws_D [B,H,n] fp32,
// ws_dq [B,n,H,d] fp32, ws_sub bwd_sub_lists_bytes(sh) (64-wide tiles),
// ws_status two int32.
cudaError_t launch_bwd(const Shape& sh, const void* q, const void* k, const void* v,
                       const void* o, const void* g_o, const float* lse, float scale,
                       const int32_t* q_idx, const int32_t* q_cnt, void* g_q, void* g_k,
                       void* g_v, float* ws_D, float* ws_dq, int32_t* ws_sub,
                       int32_t* ws_status, cudaStream_t st);

// tcgen05 dK/dV/dQ pass (head dim 64 or 128).  Shapes with 64-wide tiles run
// as 128 x 128 tiles whose lists (built in sub_ws) carry 64 x 64 quarter masks.
// part (contiguous tensors, 128 x 128 tiles): fp32 [2][B,n,H,d] scratch, work
// items of single query heads whose dK and dV are summed over the groups after.
bool bwd_tc_supported(const Shape& sh);
size_t bwd_sub_lists_bytes(const Shape& sh);
cudaError_t launch_bwd_tc(const Shape& sh, const void* q, const void* k, const void* v,
                          const void* g_o, const float* lse, const float* Dv,
                          const int32_t* q_idx, const int32_t* q_cnt, void* g_k, void* g_v,
                          float* dq_acc, int32_t* sub_ws, int32_t* status, float scale,
                          cudaStream_t st, float* part = nullptr);

// tcgen05 forward with tile statistics for 128 x 128 tiles (head dim 64 or
// 128).  logw != nullptr also writes the tile weights [B,H,T_r,T_c]; with
// stats == nullptr their rows go through `scratch` (fwd_scratch_bytes).
bool fwd_tc_supported(const Shape& sh);
bool fwd_tile_weights_supported(const Shape& sh);
size_t fwd_scratch_bytes(const Shape& sh);
size_t fwd_scratch_bytes(int d, int T_c);
// Clears the slot locks of a forward scratch (the first bytes of it).
cudaError_t fwd_scratch_clear(int d, void* scratch, cudaStream_t st);
// slot_tc: key tiles a scratch slot holds (0: sh.T_c); zero_locks: clear the
// slot locks on st first (launches that share a scratch clear it once, before
// any of them).
cudaError_t launch_fwd_tc(const Shape& sh, const void* q, const void* k, const void* v, void* o,
                          float* lse, float* stats, float* logw, void* scratch, float scale,
                          cudaStream_t st, int slot_tc = 0, bool zero_locks = true);

// LSE-combine of `parts` partial results (layouts in include/bl_attn.h).
// Error sums of bf16 a against bf16 b (n elements) into out[4] (fp64).
cudaError_t launch_grad_error(const void* a, const void* b, int64_t n, double* out,
                              cudaStream_t st);
cudaError_t launch_combine(int parts, int B, int n, int H, int d, const void* o_parts,
                           const float* lse_parts, void* o, float* lse, cudaStream_t st);

// Rows of a root-mean-square norm (norm.cuh).  Strides in elements; y, h, g_y,
// g_x, g_h and codes are contiguous [rows, cols].
struct NormFwd {
  int64_t rows, cols, x_stride, r_stride, groups;
  const void *x, *r, *w;          // r: residual or null; w: weight or null (ones)
  void *y, *h;                    // y or codes may be null; h only with r
  float* rstd;
  uint8_t* codes;                 // 8-bit output, with scales [rows, groups]
  float* scales;
  float eps;
  int group, fmt, shift;          // shift: from a column to its group, set by the launch
  bool w_f32;                     // the weight is fp32, whatever x is
};
struct NormBwd {
  int64_t rows, cols, groups;
  const void *g_y, *h, *w, *g_h;  // h null: codes and scales
  const uint8_t* codes;
  const float *scales, *rstd;
  void* g_x;
  float* partial;                 // [norm_bwd_parts, cols], or null without g_w
  int group, fmt, shift;
  bool w_f32;
};
cudaError_t launch_norm_fwd(int dtype, const NormFwd& a, cudaStream_t st);
// Partial rows of g_w that the backward writes.
int norm_bwd_parts(int64_t rows, int64_t cols);
cudaError_t launch_norm_bwd(int dtype, const NormBwd& a, void* g_w, cudaStream_t st);

// 8-bit activations (act8.cu).
struct ActSave {
  int64_t rows, cols, x_stride, groups;
  const void* x;
  uint8_t* codes;
  float* scales;
  int group, fmt;
};
struct ActLoad {
  int64_t rows, cols, groups;
  const uint8_t* codes;
  const float* scales;
  void* x;
  int group, fmt;
};
cudaError_t launch_act_save(int dtype, const ActSave& a, cudaStream_t st);
// With one scale a row, where the row kernels of norm_fwd.cu take the rows
// (cudaErrorNotSupported, and nothing launched, where they do not).
cudaError_t launch_row_save(int dtype, const ActSave& a, cudaStream_t st);
cudaError_t launch_act_load(int dtype, const ActLoad& a, cudaStream_t st);
// Codes of up to three tensors [rows, d] with one scale a row, to bf16.
struct Expand {
  const uint8_t* codes[3];
  const float* scales[3];
  void* out[3];
  int64_t rows[3], blocks[3];
};
cudaError_t launch_expand(int d, int fmt, const Expand& a, cudaStream_t st);

// The backward whose q, k and v have been expanded into bf16 and whose o is
// either bf16 (o_codes null) or codes with one scale a (token, head).
cudaError_t launch_bwd_act8(const Shape& sh, const void* q, const void* k, const void* v,
                            const void* o, const uint8_t* o_codes, const float* o_scales,
                            int o_fmt, const void* g_o, const float* lse, float scale,
                            const int32_t* q_idx, const int32_t* q_cnt, void* g_q, void* g_k,
                            void* g_v, float* ws_D, float* ws_dq, int32_t* ws_sub,
                            int32_t* ws_status, cudaStream_t st, float* part = nullptr);

// The same for up to kFewTokens tokens (bwd_few.cu), from the codes; o either in
// bf16 or (o null) as codes; q_idx/q_cnt [B,H] of one tile, or null;
// status two int32.
constexpr int kFewTokens = 64;
struct BwdFew {
  int B, n, H, Hk, causal, window;
  float scale;
  const uint8_t *q, *k, *v, *o_codes;
  const float *q_scales, *k_scales, *v_scales, *o_scales;
  const __nv_bfloat16 *o, *g_o;
  const float* lse;
  const int32_t *q_idx, *q_cnt;
  __nv_bfloat16 *g_q, *g_k, *g_v;
  int32_t* status;
};
cudaError_t launch_bwd_few(int d, int fmt, const BwdFew& a, cudaStream_t st);

// Rotary positions (rope.cu).  Strides {batch, token, head} in elements.
struct Rope {
  int B, n, H, Hk, d, pairs, axes;
  int ends[3];                    // first pair of axes 1, 2, 3 (pairs where there is none)
  bool half, inverse, copy;       // copy: the dims behind 2 * pairs too
  const void *q, *k;
  void *q_out, *k_out;
  int64_t qs[3], ks[3], qos[3], kos[3];
  const int32_t* pos;             // [B or 1, n, axes]
  int64_t pos_batch;              // 0: shared by the batches
  const uint64_t* freqs;          // [pairs], turns in 64-bit fixed point
  int lanes, tile;                // set by the launch, like:
  bool flat, pos_flat;            // tokens (positions) of all batches equally spaced
};
cudaError_t launch_rope(int dtype, const Rope& a, cudaStream_t st);

// 4-D TMA map of a BSHD bf16 tensor [B][n][heads][d] with element strides
// st = {batch, seq, head} (d contiguous): box of 64 elements of d x 1 head x
// `rows` tokens x 1 batch, 128-byte swizzle, out-of-range reads 0.
bool make_bshd_map(CUtensorMap* m, const void* base, int B, int n, int heads, int d, int rows,
                   const int64_t* st);

// The same for an fp32 BSHD tensor, box of 32 elements of d (128 bytes) x 1
// head x `rows` tokens, 128-byte swizzle: the target of dQ reduce-adds.
bool make_bshd_map_f32(CUtensorMap* m, const void* base, int B, int n, int heads, int d,
                       int rows);

}  // namespace bl
