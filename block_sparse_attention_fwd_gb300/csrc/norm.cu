// Root-mean-square norm of rows, with the residual's addition in front, an
// output in 8 bits and the backward pass:
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = (h rstd) w
//
// and, for the gradients g_y of y and g_h of h (the residual stream's own),
//   u = h rstd,  c = mean(w g_y u),
//   g_x = g_r = rstd (w g_y - u c) + g_h,   g_w = sum over rows of g_y u.
//
// Sums run in fp32; y comes from the unrounded h, so it is rounded once.
// The passes are bound by HBM: each input read once, each output written once.
#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

// A row is held by LPR lanes of a warp (LPR = 8, 16, 32: up to 64, 128, 256
// columns) or by the whole block (LPR = 0), each thread NV chunks of it.
template <typename T, int LPR, int NV, bool VEC, bool Q8>
__global__ void __launch_bounds__(512) norm_fwd_kernel(NormFwd a) {
  __shared__ uint32_t buf[2][32];
  constexpr int TPR = LPR;
  const int rows_here = LPR ? blockDim.x / (LPR ? LPR : 1) : 1;
  const int t = LPR ? threadIdx.x % (LPR ? LPR : 1) : threadIdx.x;
  const int step = LPR ? TPR : blockDim.x;      // chunks between a thread's own
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  int slot = 0;
  // the loop is uniform over the block (lanes past the last row work on zeros)
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + (LPR ? threadIdx.x / (LPR ? LPR : 1) : 0);
    const bool in = row < a.rows;
    float h[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      const int valid = in ? cols - col : 0;
      const Chunk<T> x =
          load8<T, VEC>(static_cast<const T*>(a.x) + row * a.x_stride + col, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = to_f32(x.e[i]);
    }
    if (a.r) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (t + k * step) * 8;
        const int valid = in ? cols - col : 0;
        const Chunk<T> r =
            load8<T, VEC>(static_cast<const T*>(a.r) + row * a.r_stride + col, valid);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += to_f32(r.e[i]);
        if (a.h) store8<T, VEC>(static_cast<T*>(a.h) + row * cols + col, h[k], valid);
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[k][i], h[k][i], ss);
    if constexpr (LPR != 0) {
      ss = lanes_sum(ss, LPR);
    } else {
      ss = block_sum(ss, buf, slot);
      slot ^= 1;
    }
    const float rstd = 1.f / sqrtf(fmaf(ss, inv_cols, a.eps));
    if (t == 0 && in && a.rstd) a.rstd[row] = rstd;
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      const int valid = in ? cols - col : 0;
      float w[8];
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[i];
      if (a.y) store8<T, VEC>(static_cast<T*>(a.y) + row * cols + col, h[k], valid);
      if constexpr (Q8) {
        uint32_t m = amax_bits8(h[k]);
        if (a.group) {
          m = lanes_max(m, min(a.group / 8, LPR ? LPR : 32));
          const float scale = scale_of(m, a.fmt);
          const Codes c = encode8(a.fmt, h[k], scale);
          store_codes<VEC>(a.codes + row * cols + col, c, valid);
          if (valid > 0 && col % a.group == 0)
            a.scales[row * a.groups + col / a.group] = scale;
        } else {
          top = max(top, m);
        }
      }
    }
    if constexpr (Q8) {
      if (!a.group) {
        if constexpr (LPR != 0) {
          top = lanes_max(top, LPR);
        } else {
          top = block_max(top, buf, slot);
          slot ^= 1;
        }
        const float scale = scale_of(top, a.fmt);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int col = (t + k * step) * 8;
          const int valid = in ? cols - col : 0;
          store_codes<VEC>(a.codes + row * cols + col, encode8(a.fmt, h[k], scale), valid);
        }
        if (t == 0 && in) a.scales[row] = scale;
      }
    }
  }
}

// One pass over the rows: g_x, and per block the partial sums of g_w over the
// block's rows, which stay in registers until the end ([grid, cols] fp32 in
// the workspace).  FMT 0 reads h in the type T, otherwise its 8-bit codes.
template <typename T, int LPR, int NV, bool VEC, int FMT>
__global__ void __launch_bounds__(512) norm_bwd_kernel(NormBwd a) {
  __shared__ uint32_t buf[2][32];
  __shared__ float part[LPR ? 512 * 8 : 1];
  const int rows_here = LPR ? blockDim.x / (LPR ? LPR : 1) : 1;
  const int t = LPR ? threadIdx.x % (LPR ? LPR : 1) : threadIdx.x;
  const int step = LPR ? LPR : blockDim.x;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  float acc[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
  int slot = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + (LPR ? threadIdx.x / (LPR ? LPR : 1) : 0);
    const bool in = row < a.rows;
    const float rstd = in ? a.rstd[row] : 0.f;
    Chunk<T> gy[NV];
    float u[NV][8];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      const int valid = in ? cols - col : 0;
      gy[k] = load8<T, VEC>(static_cast<const T*>(a.g_y) + row * cols + col, valid);
      if constexpr (FMT == 0) {
        const Chunk<T> h = load8<T, VEC>(static_cast<const T*>(a.h) + row * cols + col, valid);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] = to_f32(h.e[i]) * rstd;
      } else {
        const Codes c = load_codes<VEC>(a.codes + row * cols + col, valid);
        const float s = valid > 0 ? a.scales[row * a.groups + (a.group ? col / a.group : 0)] : 0.f;
        decode8<FMT>(c, u[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[k][i] = u[k][i] * s * rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      float w[8];
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = to_f32(gy[k].e[i]);
        acc[k][i] = fmaf(g, u[k][i], acc[k][i]);
        dot = fmaf(g * w[i], u[k][i], dot);
      }
    }
    if constexpr (LPR != 0) {
      dot = lanes_sum(dot, LPR);
    } else {
      dot = block_sum(dot, buf, slot);
      slot ^= 1;
    }
    const float c = dot * inv_cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      const int valid = in ? cols - col : 0;
      float w[8], g[8];
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = rstd * (to_f32(gy[k].e[i]) * w[i] - u[k][i] * c);
      if (a.g_h) {
        const Chunk<T> e = load8<T, VEC>(static_cast<const T*>(a.g_h) + row * cols + col, valid);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += to_f32(e.e[i]);
      }
      store8<T, VEC>(static_cast<T*>(a.g_x) + row * cols + col, g, valid);
    }
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * cols;
  if constexpr (LPR != 0) {
    // the block's row slots are added in their order
#pragma unroll
    for (int i = 0; i < 8; ++i) part[threadIdx.x * 8 + i] = acc[0][i];
    __syncthreads();
    for (int col = threadIdx.x; col < cols; col += blockDim.x) {
      float s = 0.f;
      for (int r = 0; r < rows_here; ++r) s += part[r * (LPR * 8) + col];
      out[col] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (t + k * step) * 8;
      store8<float, VEC>(out + col, acc[k], cols - col);
    }
  }
}

// g_w[col] = sum of the blocks' partial sums, 32 columns a block, 32 slices of
// the partial rows side by side and then added in their order: no atomics, so
// the result does not vary.
template <typename T>
__global__ void __launch_bounds__(1024) norm_gw_kernel(const float* __restrict__ partial, int parts,
                                                       int cols, void* g_w, bool f32) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  float v = 0.f;
  if (col < cols)
    for (int p = y; p < parts; p += 32) v += partial[(int64_t)p * cols + col];
  s[y][x] = v;
  __syncthreads();
  if (y == 0 && col < cols) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][x];
    if (f32)
      static_cast<float*>(g_w)[col] = sum;
    else
      static_cast<T*>(g_w)[col] = from_f32<T>(sum);
  }
}

// Threads, blocks and chunks a thread of a launch over rows of `cols` columns.
struct Plan {
  int lpr, nv, threads;
  int64_t blocks;
};
Plan plan(int64_t rows, int64_t cols, int max_blocks) {
  const int chunks = (int)((cols + 7) / 8);
  Plan p;
  if (chunks <= 32) {
    p.lpr = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    p.nv = 1;
    p.threads = 256;
    p.blocks = (rows + 256 / p.lpr - 1) / (256 / p.lpr);
  } else {
    p.lpr = 0;
    p.nv = chunks <= 256 ? 1 : chunks <= 1024 ? 2 : 4;
    p.threads = ((chunks + p.nv - 1) / p.nv + 31) / 32 * 32;
    p.blocks = rows;
  }
  if (p.blocks > max_blocks) p.blocks = max_blocks;
  return p;
}

constexpr int kFwdBlocks = 152 * 8, kBwdBlocks = 152 * 4;

template <typename T, bool VEC, bool Q8>
void fwd(const NormFwd& a, const Plan& p, cudaStream_t st) {
  const unsigned g = (unsigned)p.blocks;
  if (p.lpr == 8)
    norm_fwd_kernel<T, 8, 1, VEC, Q8><<<g, p.threads, 0, st>>>(a);
  else if (p.lpr == 16)
    norm_fwd_kernel<T, 16, 1, VEC, Q8><<<g, p.threads, 0, st>>>(a);
  else if (p.lpr == 32)
    norm_fwd_kernel<T, 32, 1, VEC, Q8><<<g, p.threads, 0, st>>>(a);
  else if (p.nv == 1)
    norm_fwd_kernel<T, 0, 1, VEC, Q8><<<g, p.threads, 0, st>>>(a);
  else if (p.nv == 2)
    norm_fwd_kernel<T, 0, 2, VEC, Q8><<<g, p.threads, 0, st>>>(a);
  else
    norm_fwd_kernel<T, 0, 4, VEC, Q8><<<g, p.threads, 0, st>>>(a);
}

template <typename T, bool VEC, int FMT>
void bwd(const NormBwd& a, const Plan& p, cudaStream_t st) {
  const unsigned g = (unsigned)p.blocks;
  if (p.lpr == 8)
    norm_bwd_kernel<T, 8, 1, VEC, FMT><<<g, p.threads, 0, st>>>(a);
  else if (p.lpr == 16)
    norm_bwd_kernel<T, 16, 1, VEC, FMT><<<g, p.threads, 0, st>>>(a);
  else if (p.lpr == 32)
    norm_bwd_kernel<T, 32, 1, VEC, FMT><<<g, p.threads, 0, st>>>(a);
  else if (p.nv == 1)
    norm_bwd_kernel<T, 0, 1, VEC, FMT><<<g, p.threads, 0, st>>>(a);
  else if (p.nv == 2)
    norm_bwd_kernel<T, 0, 2, VEC, FMT><<<g, p.threads, 0, st>>>(a);
  else
    norm_bwd_kernel<T, 0, 4, VEC, FMT><<<g, p.threads, 0, st>>>(a);
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t cols) { return (int)plan(rows, cols, kBwdBlocks).blocks; }

cudaError_t launch_norm_fwd(int dtype, const NormFwd& a, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const Plan p = plan(a.rows, a.cols, kFwdBlocks);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 && a.r_stride % 8 == 0 &&
                     aligned_to(a.x, 16) && aligned_to(a.r, 16) && aligned_to(a.h, 16) &&
                     aligned_to(a.y, 16) && aligned_to(a.w, 16) && aligned_to(a.codes, 8);
    if (a.codes)
      vec ? fwd<T, true, true>(a, p, st) : fwd<T, false, true>(a, p, st);
    else
      vec ? fwd<T, true, false>(a, p, st) : fwd<T, false, false>(a, p, st);
    return cudaGetLastError();
  });
}

cudaError_t launch_norm_bwd(int dtype, const NormBwd& a, void* g_w, cudaStream_t st) {
  const Plan p = plan(a.rows, a.cols, kBwdBlocks);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && aligned_to(a.g_y, 16) && aligned_to(a.h, 16) &&
                     aligned_to(a.g_h, 16) && aligned_to(a.g_x, 16) && aligned_to(a.w, 16) &&
                     aligned_to(a.codes, 8) && aligned_to(a.partial, 16);
    if (a.rows > 0) {
      if (!a.codes)
        vec ? bwd<T, true, 0>(a, p, st) : bwd<T, false, 0>(a, p, st);
      else if (a.fmt == kFmtInt8)
        vec ? bwd<T, true, kFmtInt8>(a, p, st) : bwd<T, false, kFmtInt8>(a, p, st);
      else
        vec ? bwd<T, true, kFmtE4m3>(a, p, st) : bwd<T, false, kFmtE4m3>(a, p, st);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (g_w) {
      norm_gw_kernel<T><<<(unsigned)((a.cols + 31) / 32), 1024, 0, st>>>(
          a.partial, a.rows ? (int)p.blocks : 0, (int)a.cols, g_w, a.w_f32);
      return cudaGetLastError();
    }
    return cudaSuccess;
  });
}

}  // namespace bl
