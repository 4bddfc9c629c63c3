// C ABI of the linear layers around the attention: argument checks and launches of
// products in 8 bits, the layer norm and dropout.  They are documented in
// include/bl_attn.h.
#include <math.h>
#include <stdint.h>

#include "../../include/bl_attn.h"
#include "abi.h"
#include "kernels.h"
#include "rows.cuh"

namespace {

bl_status cuda_status(cudaError_t e) { return e == cudaSuccess ? BL_OK : BL_ERR_CUDA; }
size_t size_of(int dtype) { return dtype == BL_FP32 ? 4 : 2; }
bool dtype_ok(int t) { return t == BL_BF16 || t == BL_FP16 || t == BL_FP32; }
bool elem_ok(const void* p, int dtype) { return bl::aligned_to(p, size_of(dtype)); }
bool rows_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= (int64_t)1 << 40 && cols >= 1 && cols <= (int64_t)1 << 30;
}
bool act8_ok(const bl_act8* a, int64_t rows) {
  if (a->format != BL_INT8 && a->format != BL_E4M3) return false;
  if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return false;
  return rows == 0 || (a->codes && a->scales && bl::aligned_to(a->scales, 4));
}
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// A code tensor of a product: the summed dim is its columns, or (along_rows) its rows.
struct Operand {
  int64_t rows, cols, stride;
  const void* codes;
  const float* scales;
  bool packed() const { return stride % 16 == 0 && bl::aligned16(codes); }
  // bytes of a copy with aligned rows, where the tensor's are not
  size_t copy_bytes() const {
    return packed() ? 0 : up256((size_t)rows * (size_t)((cols + 15) / 16 * 16));
  }
};

bool operands(const bl_matmul8_args* p, Operand* a, Operand* b) {
  const int64_t most = (int64_t)1 << 30;
  if (!p || p->form < BL_MATMUL8_Y || p->form > BL_MATMUL8_G_W) return false;
  if (p->tokens < 0 || p->tokens > most || p->out_features < 1 || p->out_features > most ||
      p->in_features < 1 || p->in_features > most)
    return false;
  const bool g_w = p->form == BL_MATMUL8_G_W;
  *a = Operand{p->tokens, p->form == BL_MATMUL8_Y ? p->in_features : p->out_features, p->a_stride,
               p->a_codes, p->a_scales};
  *b = Operand{g_w ? p->tokens : p->out_features, p->in_features, p->b_stride, p->b_codes,
               p->b_scales};
  for (const Operand* o : {a, b}) {
    if (o->stride < o->cols || o->stride > (int64_t)1 << 38) return false;
    if (o->rows && (!o->codes || !o->scales || !bl::aligned_to(o->scales, 4))) return false;
  }
  return true;
}

}  // namespace

extern "C" {

bl_status bl_tile8_save(const bl_tile8_args* p, void* stream) {
  if (!p || !rows_ok(p->rows, p->cols) || !dtype_ok(p->dtype)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(p->x, p->dtype) || p->x_stride < p->cols) return BL_ERR_INVALID_ARG;
  if (p->block_codes && p->col_codes) return BL_ERR_INVALID_ARG;
  const void* codes[3] = {p->row_codes, p->col_codes, p->block_codes};
  const float* scales[3] = {p->row_scales, p->col_scales, p->block_scales};
  const int64_t strides[3] = {p->row_stride, p->col_stride, p->block_stride};
  bool any = false;
  for (int i = 0; i < 3; ++i) {
    if (!codes[i]) continue;
    any = true;
    if (strides[i] < p->cols || !scales[i] || !bl::aligned_to(scales[i], 4))
      return BL_ERR_INVALID_ARG;
  }
  if (p->rows == 0) return BL_OK;
  if (!any || !p->x) return BL_ERR_INVALID_ARG;
  if (((p->rows + 127) / 128) * ((p->cols + 127) / 128) > INT32_MAX) return BL_ERR_UNSUPPORTED;
  bl::TileSave a{};
  a.rows = p->rows; a.cols = p->cols; a.x = p->x; a.x_stride = p->x_stride;
  a.row_codes = static_cast<uint8_t*>(p->row_codes); a.row_scales = p->row_scales;
  a.col_codes = static_cast<uint8_t*>(p->col_codes); a.col_scales = p->col_scales;
  a.block_codes = static_cast<uint8_t*>(p->block_codes); a.block_scales = p->block_scales;
  a.row_stride = a.row_codes ? p->row_stride : 0;
  a.col_stride = a.col_codes ? p->col_stride : 0;
  a.block_stride = a.block_codes ? p->block_stride : 0;
  return cuda_status(bl::launch_tile_save(p->dtype, a, (cudaStream_t)stream));
}

bl_status bl_tile8_load(int64_t rows, int64_t cols, int dtype, const void* codes, int64_t stride,
                        const float* scales, int blocks, void* x, void* stream) {
  if (!rows_ok(rows, cols) || !dtype_ok(dtype) || stride < cols || (blocks & ~1))
    return BL_ERR_INVALID_ARG;
  if (rows && (!codes || !scales || !x)) return BL_ERR_INVALID_ARG;
  if (!bl::aligned_to(scales, 4) || !elem_ok(x, dtype)) return BL_ERR_INVALID_ARG;
  bl::TileLoad a{rows, cols, stride, blocks ? (cols + 127) / 128 : cols,
                 static_cast<const uint8_t*>(codes), scales, x, blocks ? 7 : 0};
  return cuda_status(bl::launch_tile_load(dtype, a, (cudaStream_t)stream));
}

size_t bl_matmul8_workspace_bytes(const bl_matmul8_args* args) {
  Operand a, b;
  if (!operands(args, &a, &b)) return 0;
  return a.copy_bytes() + b.copy_bytes();
}

bl_status bl_matmul8(const bl_matmul8_args* p, void* stream) {
  Operand a, b;
  if (!operands(p, &a, &b) || !dtype_ok(p->out_dtype)) return BL_ERR_INVALID_ARG;
  const bool g_w = p->form == BL_MATMUL8_G_W;
  const int64_t m = g_w ? p->out_features : p->tokens;
  const int64_t n = p->form == BL_MATMUL8_Y ? p->out_features : p->in_features;
  const int64_t k = g_w ? p->tokens : a.cols;
  if (m == 0) return BL_OK;
  if (!p->out || !elem_ok(p->out, p->out_dtype)) return BL_ERR_INVALID_ARG;
  if (m * n > (int64_t)1 << 44) return BL_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (k == 0)
    return cuda_status(cudaMemsetAsync(p->out, 0, (size_t)(m * n) * size_of(p->out_dtype), st));
  const size_t need = a.copy_bytes() + b.copy_bytes();
  if (need && (!p->workspace || !bl::aligned16(p->workspace) || p->workspace_bytes < need))
    return BL_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  bl::Repitch copies[2] = {};
  for (int i = 0; i < 2; ++i) {
    Operand& o = i ? b : a;
    if (o.packed()) continue;
    const int64_t pitch = (o.cols + 15) / 16 * 16;
    const size_t bytes = o.copy_bytes();
    copies[i] = bl::Repitch{static_cast<const uint8_t*>(o.codes), ws, o.stride, pitch, o.rows,
                            o.cols};
    o.codes = ws;
    o.stride = pitch;
    ws += bytes;
  }
  if (need) {
    const cudaError_t e = bl::launch_repitch(copies[0], copies[1], st);
    if (e != cudaSuccess) return BL_ERR_CUDA;
  }
  bl::Gemm8 g{};
  g.m = (int)m; g.n = (int)n; g.k = (int)k;
  g.a = static_cast<const uint8_t*>(a.codes); g.b = static_cast<const uint8_t*>(b.codes);
  g.a_pitch = a.stride; g.b_pitch = b.stride;
  g.a_mn = g_w; g.b_mn = p->form != BL_MATMUL8_Y;
  g.sa = a.scales; g.sb = b.scales;
  if (g_w) {                                          // [blocks of tokens, features]
    g.sa_i = 1; g.sa_b = m;
    g.sb_i = 1; g.sb_b = n;
  } else {
    const int64_t blocks = (p->in_features + 127) / 128;   // of a row of the weight's scales
    g.sa_i = (k + 127) / 128; g.sa_b = 1;
    g.sb_shift = 7;
    g.sb_i = p->form == BL_MATMUL8_Y ? blocks : 1;
    g.sb_b = p->form == BL_MATMUL8_Y ? 1 : blocks;
  }
  g.out = p->out; g.out_i = n; g.out_j = 1;
  return cuda_status(bl::launch_gemm8(p->out_dtype, g, st));
}

bl_status bl_layer_norm_fwd(const bl_layer_norm_args* p, void* stream) {
  if (!p || !rows_ok(p->rows, p->cols) || !dtype_ok(p->dtype)) return BL_ERR_INVALID_ARG;
  const int64_t rows = p->rows, cols = p->cols;
  if ((p->weight || p->bias) && p->weight_dtype != p->dtype && p->weight_dtype != BL_FP32)
    return BL_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || !isfinite(p->eps)) return BL_ERR_INVALID_ARG;
  if (rows && (!p->x || (!p->y && !p->y8))) return BL_ERR_INVALID_ARG;
  if (p->x_stride < cols || (p->residual && p->residual_stride < cols)) return BL_ERR_INVALID_ARG;
  if (p->h && !p->residual) return BL_ERR_INVALID_ARG;
  if (p->y8 && !act8_ok(p->y8, rows)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(p->x, p->dtype) || !elem_ok(p->residual, p->dtype) || !elem_ok(p->y, p->dtype) ||
      !elem_ok(p->h, p->dtype) || !bl::aligned_to(p->mean, 4) || !bl::aligned_to(p->rstd, 4))
    return BL_ERR_INVALID_ARG;
  if ((p->weight && !elem_ok(p->weight, p->weight_dtype)) ||
      (p->bias && !elem_ok(p->bias, p->weight_dtype)))
    return BL_ERR_INVALID_ARG;
  if (cols > BL_NORM_MAX_COLS) return BL_ERR_UNSUPPORTED;
  bl::LayerNormFwd a{};
  a.rows = rows; a.cols = cols;
  a.x_stride = p->x_stride; a.r_stride = p->residual ? p->residual_stride : 0;
  a.x = p->x; a.r = p->residual; a.w = p->weight; a.b = p->bias;
  a.y = p->y; a.h = p->h; a.mean = p->mean; a.rstd = p->rstd; a.eps = p->eps;
  a.w_f32 = p->weight_dtype == BL_FP32;
  if (p->y8) {
    a.codes = static_cast<uint8_t*>(p->y8->codes); a.scales = p->y8->scales;
    a.group = p->y8->group; a.fmt = p->y8->format;
    a.groups = bl::groups_of(cols, p->y8->group);
  }
  return cuda_status(bl::launch_layer_norm_fwd(p->dtype, a, (cudaStream_t)stream));
}

size_t bl_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!rows_ok(rows, cols) || cols > BL_NORM_MAX_COLS) return 0;
  return 2 * (size_t)bl::layer_norm_bwd_parts(rows, cols) * (size_t)cols * sizeof(float);
}

bl_status bl_layer_norm_bwd(const bl_layer_norm_bwd_args* p, void* stream) {
  if (!p || !rows_ok(p->rows, p->cols) || !dtype_ok(p->dtype)) return BL_ERR_INVALID_ARG;
  const int64_t rows = p->rows, cols = p->cols;
  if ((p->weight || p->g_w || p->g_b) && p->weight_dtype != p->dtype && p->weight_dtype != BL_FP32)
    return BL_ERR_INVALID_ARG;
  if (p->h8 && (p->h || !act8_ok(p->h8, rows))) return BL_ERR_INVALID_ARG;
  if (rows && (!p->g_y || (!p->h && !p->h8) || !p->mean || !p->rstd || !p->g_x))
    return BL_ERR_INVALID_ARG;
  if (!elem_ok(p->g_y, p->dtype) || !elem_ok(p->h, p->dtype) || !elem_ok(p->g_h, p->dtype) ||
      !elem_ok(p->g_x, p->dtype) || !bl::aligned_to(p->mean, 4) || !bl::aligned_to(p->rstd, 4))
    return BL_ERR_INVALID_ARG;
  if ((p->weight && !elem_ok(p->weight, p->weight_dtype)) ||
      (p->g_w && !elem_ok(p->g_w, p->weight_dtype)) ||
      (p->g_b && !elem_ok(p->g_b, p->weight_dtype)))
    return BL_ERR_INVALID_ARG;
  if (cols > BL_NORM_MAX_COLS) return BL_ERR_UNSUPPORTED;
  const bool sums = p->g_w || p->g_b;
  if (sums && rows &&
      (!p->workspace || !bl::aligned16(p->workspace) ||
       p->workspace_bytes < bl_layer_norm_bwd_workspace_bytes(rows, cols)))
    return BL_ERR_WORKSPACE;
  bl::NormBwd a{};
  a.rows = rows; a.cols = cols;
  a.g_y = p->g_y; a.h = p->h; a.w = p->weight; a.g_h = p->g_h; a.mean = p->mean; a.rstd = p->rstd;
  a.g_x = p->g_x;
  a.partial = sums ? static_cast<float*>(p->workspace) : nullptr;
  a.w_f32 = p->weight_dtype == BL_FP32;
  if (p->h8) {
    a.codes = static_cast<const uint8_t*>(p->h8->codes); a.scales = p->h8->scales;
    a.group = p->h8->group; a.fmt = p->h8->format;
    a.groups = bl::groups_of(cols, p->h8->group);
  }
  return cuda_status(bl::launch_layer_norm_bwd(p->dtype, a, p->g_w, p->g_b, (cudaStream_t)stream));
}

bl_status bl_dropout(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                     const void* residual, int64_t residual_stride, double p, const int64_t* state,
                     void* y, void* stream) {
  if (rows < 0 || cols < 1 || !dtype_ok(dtype)) return BL_ERR_INVALID_ARG;
  if (!(p >= 0. && p <= 1.)) return BL_ERR_INVALID_ARG;
  if (rows > ((int64_t)1 << 42) / cols) return BL_ERR_UNSUPPORTED;
  if (x_stride < cols || (residual && residual_stride < cols)) return BL_ERR_INVALID_ARG;
  if (rows && (!x || !y || !state)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(x, dtype) || !elem_ok(residual, dtype) || !elem_ok(y, dtype) ||
      !bl::aligned_to(state, 8))
    return BL_ERR_INVALID_ARG;
  bl::Dropout a{};
  a.rows = rows; a.cols = cols; a.x_stride = x_stride; a.r_stride = residual ? residual_stride : 0;
  a.x = x; a.r = residual; a.y = y; a.state = state;
  const double words = nearbyint(p * 4294967296.);
  a.all = words >= 4294967296.;                         // no word is as large
  a.threshold = a.all ? 0xffffffffu : (uint32_t)words;
  a.scale = p < 1. ? (float)(1. / (1. - p)) : 0.f;
  return cuda_status(bl::launch_dropout(dtype, a, (cudaStream_t)stream));
}

bl_status bl_dropout_next(int64_t* state, int64_t* used, void* stream) {
  if (!state || !used || state == used || !bl::aligned_to(state, 8) || !bl::aligned_to(used, 8))
    return BL_ERR_INVALID_ARG;
  return cuda_status(bl::launch_dropout_next(state, used, (cudaStream_t)stream));
}

}  // extern "C"
