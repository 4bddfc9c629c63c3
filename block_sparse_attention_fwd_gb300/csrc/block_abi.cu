// C ABI of the operators around the attention: argument checks and launches.
// They are documented in include/bl_attn.h.
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
bool rows_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= (int64_t)1 << 40 && cols >= 1 && cols <= (int64_t)1 << 30;
}
bool elem_ok(const void* p, int dtype) { return bl::aligned_to(p, size_of(dtype)); }
// With no rows, pointers may be NULL (an empty tensor has none).
bool act8_ok(const bl_act8* a, int64_t rows) {
  if (a->format != BL_INT8 && a->format != BL_E4M3) return false;
  if (a->group != 0 && a->group != 32 && a->group != 64 && a->group != 128) return false;
  return rows == 0 || (a->codes && a->scales && bl::aligned_to(a->scales, 4));
}
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Bytes of the scratch that lets the attention backward's work items be single
// query heads, or 0 where it does not pay: without groups there is nothing to
// split, few tokens have their own kernel, and with an item for every SM the
// extra passes over fp32 tiles cost more than the idle SMs do.
size_t part_bytes(const bl::Shape& sh) {
  if (sh.n <= bl::kFewTokens) return 0;
  if (sh.H == sh.Hk || sh.block_q != 128 || sh.block_k != 128) return 0;
  if ((int64_t)sh.T_c * sh.Hk * sh.B >= 152) return 0;
  return 2 * (size_t)sh.B * sh.n * sh.H * sh.d * sizeof(float);
}

// Dims from the largest stride to the smallest.
void order_by_stride(const int64_t* stride, int* order) {
  for (int i = 0; i < 3; ++i) order[i] = i;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (stride[order[j]] < stride[order[j + 1]]) {
        const int s = order[j];
        order[j] = order[j + 1];
        order[j + 1] = s;
      }
}
// Whether each stride of a tensor of heads of d spans the dims behind it, so that
// no two heads meet.  Every view that slices, steps over or permutes the dims of
// a dense tensor is such.
bool spans(const int64_t* stride, const int64_t* size, int64_t d) {
  int order[3];
  order_by_stride(stride, order);
  int64_t extent = d;
  for (int i = 2; i >= 0; --i) {
    const int64_t s = stride[order[i]], m = size[order[i]];
    if (m == 1) continue;
    if (s < extent || s > ((int64_t)1 << 60) / m) return false;
    extent += (m - 1) * s;
  }
  return true;
}

// Whether some head of k lies on elements of one of q's, where both have the
// same strides: `gap` elements between their first ones, t[i] in [lo[i], hi[i]]
// the distance of a head of k and one of q along dim i, dims from the largest
// stride to the smallest.  Exact where each stride spans the dims behind it (spans).
bool heads_meet(int64_t gap, const int64_t* stride, const int64_t* lo, const int64_t* hi, int dims,
                int64_t d) {
  if (dims == 0) return gap > -d && gap < d;
  const int64_t near = stride[0] ? -(gap / stride[0]) : 0;
  for (int64_t s = near - 1; s <= near + 1; ++s) {
    const int64_t t = s < lo[0] ? lo[0] : s > hi[0] ? hi[0] : s;
    if (heads_meet(gap + t * stride[0], stride + 1, lo + 1, hi + 1, dims - 1, d)) return true;
  }
  return false;
}

// Whether k_out shares elements with q_out (each spans its dims), as far as their
// batches and tokens have the same strides.
bool outputs_meet(const bl_rope_args* r, const int64_t* q, const int64_t* k) {
  // the stride of a dim of one element says nothing
  const int64_t batch = r->B > 1 ? q[0] : 0, token = r->n > 1 ? q[1] : 0;
  if ((r->B > 1 && k[0] != batch) || (r->n > 1 && k[1] != token)) return false;
  const int64_t q_head = r->H > 1 ? q[2] : 0, k_head = r->Hk > 1 ? k[2] : 0;
  const int64_t gap =
      (int64_t)((intptr_t)r->k_out - (intptr_t)r->q_out) / (int64_t)size_of(r->dtype);
  // heads a step of their own apart: q's one by one
  const bool one_step = r->H == 1 || r->Hk == 1 || q_head == k_head;
  const int64_t at[3] = {batch, token, one_step && r->Hk == 1 ? q_head : k_head};
  int order[3];
  order_by_stride(at, order);
  int64_t stride[3], lo[3], hi[3];
  for (int i = 0; i < 3; ++i) {
    const int64_t span = order[i] == 0 ? r->B - 1 : r->n - 1;
    stride[i] = at[order[i]];
    lo[i] = order[i] == 2 ? (one_step ? 1 - (int64_t)r->H : 0) : -span;
    hi[i] = order[i] == 2 ? r->Hk - 1 : span;
  }
  for (int64_t h = 0; h < (one_step ? 1 : r->H); ++h)
    if (heads_meet(gap - h * q_head, stride, lo, hi, 3, r->d)) return true;
  return false;
}

}  // namespace

extern "C" {

bl_status bl_act_save(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                      const bl_act8* out, void* stream) {
  if (!rows_ok(rows, cols) || !dtype_ok(dtype) || !out || !act8_ok(out, rows))
    return BL_ERR_INVALID_ARG;
  if ((rows && !x) || !elem_ok(x, dtype) || x_stride < cols) return BL_ERR_INVALID_ARG;
  bl::ActSave a{rows, cols, x_stride, bl::groups_of(cols, out->group), x,
                static_cast<uint8_t*>(out->codes), out->scales, out->group, out->format};
  return cuda_status(bl::launch_act_save(dtype, a, (cudaStream_t)stream));
}

bl_status bl_act_load(int64_t rows, int64_t cols, int dtype, const bl_act8* in, void* x,
                      void* stream) {
  if (!rows_ok(rows, cols) || !dtype_ok(dtype) || !in || !act8_ok(in, rows))
    return BL_ERR_INVALID_ARG;
  if ((rows && !x) || !elem_ok(x, dtype)) return BL_ERR_INVALID_ARG;
  bl::ActLoad a{rows, cols, bl::groups_of(cols, in->group),
                static_cast<const uint8_t*>(in->codes), in->scales, x, in->group, in->format};
  return cuda_status(bl::launch_act_load(dtype, a, (cudaStream_t)stream));
}

bl_status bl_rms_norm_fwd(int64_t rows, int64_t cols, int dtype, const void* x, int64_t x_stride,
                          const void* residual, int64_t residual_stride, const void* weight,
                          int weight_dtype, float eps, void* y, void* h, float* rstd,
                          const bl_act8* y8, void* stream) {
  if (!rows_ok(rows, cols) || !dtype_ok(dtype)) return BL_ERR_INVALID_ARG;
  if (weight && weight_dtype != dtype && weight_dtype != BL_FP32) return BL_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !isfinite(eps)) return BL_ERR_INVALID_ARG;
  if (rows && (!x || (!y && !y8))) return BL_ERR_INVALID_ARG;
  if (x_stride < cols || (residual && residual_stride < cols)) return BL_ERR_INVALID_ARG;
  if (h && !residual) return BL_ERR_INVALID_ARG;
  if (y8 && !act8_ok(y8, rows)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(x, dtype) || !elem_ok(residual, dtype) || !elem_ok(y, dtype) ||
      !elem_ok(h, dtype) || !elem_ok(weight, weight_dtype) || !bl::aligned_to(rstd, 4))
    return BL_ERR_INVALID_ARG;
  if (cols > BL_NORM_MAX_COLS) return BL_ERR_UNSUPPORTED;
  bl::NormFwd a{};
  a.rows = rows; a.cols = cols;
  a.x_stride = x_stride; a.r_stride = residual ? residual_stride : 0;
  a.x = x; a.r = residual; a.w = weight;
  a.y = y; a.h = h; a.rstd = rstd; a.eps = eps;
  a.w_f32 = weight_dtype == BL_FP32;
  if (y8) {
    a.codes = static_cast<uint8_t*>(y8->codes); a.scales = y8->scales;
    a.group = y8->group; a.fmt = y8->format;
    a.groups = bl::groups_of(cols, y8->group);
  }
  return cuda_status(bl::launch_norm_fwd(dtype, a, (cudaStream_t)stream));
}

size_t bl_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t cols) {
  if (!rows_ok(rows, cols) || cols > BL_NORM_MAX_COLS) return 0;
  return (size_t)bl::norm_bwd_parts(rows, cols) * (size_t)cols * sizeof(float);
}

bl_status bl_rms_norm_bwd(int64_t rows, int64_t cols, int dtype, const void* g_y, const void* h,
                          const bl_act8* h8, const float* rstd, const void* weight,
                          int weight_dtype, const void* g_h, void* g_x, void* g_w,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!rows_ok(rows, cols) || !dtype_ok(dtype)) return BL_ERR_INVALID_ARG;
  if ((weight || g_w) && weight_dtype != dtype && weight_dtype != BL_FP32)
    return BL_ERR_INVALID_ARG;
  if (h8 && (h || !act8_ok(h8, rows))) return BL_ERR_INVALID_ARG;
  if (rows && (!g_y || (!h && !h8) || !rstd || !g_x)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(g_y, dtype) || !elem_ok(h, dtype) || !elem_ok(g_h, dtype) ||
      !elem_ok(g_x, dtype) || !elem_ok(weight, weight_dtype) || !elem_ok(g_w, weight_dtype) ||
      !bl::aligned_to(rstd, 4))
    return BL_ERR_INVALID_ARG;
  if (cols > BL_NORM_MAX_COLS) return BL_ERR_UNSUPPORTED;
  if (g_w && rows &&
      (!workspace || !bl::aligned16(workspace) ||
       workspace_bytes < bl_rms_norm_bwd_workspace_bytes(rows, cols)))
    return BL_ERR_WORKSPACE;
  bl::NormBwd a{};
  a.rows = rows; a.cols = cols;
  a.g_y = g_y; a.h = h; a.w = weight; a.g_h = g_h; a.rstd = rstd; a.g_x = g_x;
  a.partial = g_w ? static_cast<float*>(workspace) : nullptr;
  a.w_f32 = weight_dtype == BL_FP32;
  if (h8) {
    a.codes = static_cast<const uint8_t*>(h8->codes); a.scales = h8->scales;
    a.group = h8->group; a.fmt = h8->format;
    a.groups = bl::groups_of(cols, h8->group);
  }
  return cuda_status(bl::launch_norm_bwd(dtype, a, g_w, (cudaStream_t)stream));
}

bl_status bl_rope(const bl_rope_args* r, void* stream) {
  if (!r || r->B < 0 || r->n < 0 || r->H < 1 || r->Hk < 0 || r->d < 2) return BL_ERR_INVALID_ARG;
  if (r->H > 65535 || r->Hk > 65535 || r->d > 65536) return BL_ERR_INVALID_ARG;
  if (((int64_t)r->H + r->Hk) * r->d > INT32_MAX) return BL_ERR_INVALID_ARG;
  if (r->pairs < 1 || r->pairs > r->d / 2 || r->axes < 1 || r->axes > 4) return BL_ERR_INVALID_ARG;
  if (!dtype_ok(r->dtype)) return BL_ERR_INVALID_ARG;
  if ((r->interleaved & ~1) || (r->inverse & ~1)) return BL_ERR_INVALID_ARG;
  bl::Rope a{};
  int64_t sum = 0;
  for (int i = 0; i < r->axes; ++i) {
    if (r->sections[i] < 1) return BL_ERR_INVALID_ARG;
    if (i > 0) a.ends[i - 1] = (int)sum;
    sum += r->sections[i];
    if (sum > r->pairs) return BL_ERR_INVALID_ARG;
  }
  if (sum != r->pairs) return BL_ERR_INVALID_ARG;
  for (int i = r->axes - 1; i < 3; ++i) a.ends[i] = r->pairs;
  if (r->B == 0 || r->n == 0) return BL_OK;
  if (!r->q || !r->q_out || !r->positions || !r->freqs) return BL_ERR_INVALID_ARG;
  if (r->Hk && (!r->k || !r->k_out)) return BL_ERR_INVALID_ARG;
  if (!elem_ok(r->q, r->dtype) || !elem_ok(r->q_out, r->dtype) || !elem_ok(r->k, r->dtype) ||
      !elem_ok(r->k_out, r->dtype) || !bl::aligned_to(r->positions, 4) ||
      !bl::aligned_to(r->freqs, 8))
    return BL_ERR_INVALID_ARG;
  const int64_t* in[4] = {r->q_strides, r->k_strides, r->q_out_strides, r->k_out_strides};
  int64_t* to[4] = {a.qs, a.ks, a.qos, a.kos};
  for (int t = 0; t < 4; ++t)
    for (int i = 0; i < 3; ++i) {
      if (in[t][i] < 0) return BL_ERR_INVALID_ARG;
      to[t][i] = t % 2 && !r->Hk ? 0 : in[t][i];     // no k: its strides say nothing
    }
  // the heads of an output may not lie on one another
  const bool q_same = r->q == r->q_out, k_same = r->Hk && r->k == r->k_out;
  for (int i = 0; i < 3; ++i) {
    if (q_same && a.qs[i] != a.qos[i]) return BL_ERR_INVALID_ARG;
    if (k_same && a.ks[i] != a.kos[i]) return BL_ERR_INVALID_ARG;
  }
  const int64_t q_size[3] = {r->B, r->n, r->H}, k_size[3] = {r->B, r->n, r->Hk};
  if (!spans(a.qos, q_size, r->d) || (r->Hk && !spans(a.kos, k_size, r->d)))
    return BL_ERR_INVALID_ARG;
  // nor those of k on those of q, where both are views of one tensor
  if (r->Hk && (r->q_out == r->k_out || outputs_meet(r, a.qos, a.kos))) return BL_ERR_INVALID_ARG;
  if (r->positions_batch_stride != 0 &&
      r->positions_batch_stride != (int64_t)r->n * r->axes)
    return BL_ERR_INVALID_ARG;
  a.B = r->B; a.n = r->n; a.H = r->H; a.Hk = r->Hk; a.d = r->d;
  a.pairs = r->pairs; a.axes = r->axes;
  a.half = !r->interleaved; a.inverse = r->inverse != 0;
  a.copy = !(q_same && (!r->Hk || k_same));
  a.q = r->q; a.k = r->Hk ? r->k : nullptr;
  a.q_out = r->q_out; a.k_out = r->Hk ? r->k_out : nullptr;
  a.pos = r->positions; a.pos_batch = r->positions_batch_stride; a.freqs = r->freqs;
  return cuda_status(bl::launch_rope(r->dtype, a, (cudaStream_t)stream));
}

size_t bl_attn_bwd_act8_workspace_bytes(const bl_shape* shape) {
  bl::Shape sh;
  if (bl::check_shape(shape, &sh) != BL_OK || sh.strided) return 0;
  const size_t tokens = (size_t)sh.B * sh.n * sh.d * 2;
  return up256(bl_bwd_workspace_bytes(shape)) + up256(tokens * sh.H) +
         2 * up256(tokens * sh.Hk) + part_bytes(sh);
}

bl_status bl_attn_bwd_act8(const bl_shape* shape, const bl_act8* q8, const bl_act8* k8,
                           const bl_act8* v8, const void* o, const bl_act8* o8, const void* g_o,
                           const float* lse, float scale, const bl_lists* lists, void* g_q,
                           void* g_k, void* g_v, void* workspace, size_t workspace_bytes,
                           void* stream) {
  bl::Shape sh;
  const bl_status s = bl::check_shape(shape, &sh);
  if (s != BL_OK) return s;
  if (sh.strided) return BL_ERR_UNSUPPORTED;
  if (!q8 || !k8 || !v8 || (o != nullptr) == (o8 != nullptr)) return BL_ERR_INVALID_ARG;
  const bl_act8* in[4] = {q8, k8, v8, o8};
  for (const bl_act8* a : in) {
    if (!a) continue;
    if (!act8_ok(a, 1) || a->group != 0 || a->format != q8->format) return BL_ERR_INVALID_ARG;
    if (!bl::aligned16(a->codes)) return BL_ERR_INVALID_ARG;
  }
  const void* ptrs[] = {g_o, lse, g_q, g_k, g_v};
  for (const void* p : ptrs)
    if (!p || !bl::aligned16(p)) return BL_ERR_INVALID_ARG;
  if (!bl::aligned16(o)) return BL_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return BL_ERR_INVALID_ARG;
  if (lists && (!lists->q_idx || !lists->q_cnt)) return BL_ERR_INVALID_ARG;
  if (!workspace || !bl::aligned16(workspace)) return BL_ERR_WORKSPACE;
  if (workspace_bytes < bl_attn_bwd_act8_workspace_bytes(shape)) return BL_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t tokens = (size_t)sh.B * sh.n * sh.d * 2;
  uint8_t* q = ws + up256(bl_bwd_workspace_bytes(shape));
  uint8_t* k = q + up256(tokens * sh.H);
  uint8_t* v = k + up256(tokens * sh.Hk);
  int32_t* ws_status = reinterpret_cast<int32_t*>(ws + bl::ws_status_off(sh));
  if (sh.n <= bl::kFewTokens) {
    bl::BwdFew f{};
    f.B = sh.B; f.n = sh.n; f.H = sh.H; f.Hk = sh.Hk;
    f.causal = sh.causal; f.window = sh.window;
    f.scale = scale;
    f.q = static_cast<const uint8_t*>(q8->codes); f.q_scales = q8->scales;
    f.k = static_cast<const uint8_t*>(k8->codes); f.k_scales = k8->scales;
    f.v = static_cast<const uint8_t*>(v8->codes); f.v_scales = v8->scales;
    f.o = static_cast<const __nv_bfloat16*>(o);
    f.g_o = static_cast<const __nv_bfloat16*>(g_o);
    if (o8) {
      f.o_codes = static_cast<const uint8_t*>(o8->codes);
      f.o_scales = o8->scales;
    }
    f.lse = lse;
    if (lists) {
      f.q_idx = lists->q_idx;
      f.q_cnt = lists->q_cnt;
    }
    f.g_q = static_cast<__nv_bfloat16*>(g_q);
    f.g_k = static_cast<__nv_bfloat16*>(g_k);
    f.g_v = static_cast<__nv_bfloat16*>(g_v);
    f.status = ws_status;
    const cudaError_t e = bl::launch_bwd_few(sh.d, q8->format, f, (cudaStream_t)stream);
    if (e != cudaErrorNotSupported) return cuda_status(e);
  }
  float* part = part_bytes(sh) ? reinterpret_cast<float*>(v + up256(tokens * sh.Hk)) : nullptr;
  bl::Expand e{};
  uint8_t* out[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    e.codes[i] = static_cast<const uint8_t*>(in[i]->codes);
    e.scales[i] = in[i]->scales;
    e.out[i] = out[i];
    e.rows[i] = (int64_t)sh.B * sh.n * (i == 0 ? sh.H : sh.Hk);
  }
  const cudaError_t err = bl::launch_expand(sh.d, q8->format, e, (cudaStream_t)stream);
  if (err != cudaSuccess) return BL_ERR_CUDA;
  float* ws_D = reinterpret_cast<float*>(ws);
  float* ws_dq = reinterpret_cast<float*>(ws + bl::ws_D_bytes(sh));
  int32_t* ws_sub = reinterpret_cast<int32_t*>(ws + bl::ws_D_bytes(sh) + bl::ws_dq_bytes(sh));
  return cuda_status(bl::launch_bwd_act8(
      sh, q, k, v, o, o8 ? static_cast<const uint8_t*>(o8->codes) : nullptr,
      o8 ? o8->scales : nullptr, q8->format, g_o, lse, scale, lists ? lists->q_idx : nullptr,
      lists ? lists->q_cnt : nullptr, g_q, g_k, g_v, ws_D, ws_dq, ws_sub, ws_status,
      (cudaStream_t)stream, part));
}

}  // extern "C"
