// Backward of the root-mean-square norm (norm.cuh).
#include "norm_bwd.cuh"

namespace bl {

namespace {

// The backward of rows that the ring does not take, straight from global memory: fp32
// that starts anywhere and is held by a warp or comes in 8 bits (IN8) or is too wide,
// and 16-bit rows that start anywhere of more than 16376 columns.
template <typename T, int LPR, int NV, bool VEC, bool IN8>
__global__ void __launch_bounds__(LPR ? 256 : 512) norm_bwd_kernel(NormBwd a) {
  __shared__ float buf[2][32];
  __shared__ float part[LPR ? 256 * 8 * NV : 1];
  constexpr bool SPREAD = !VEC && !IN8;
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  float acc[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
  int slot = 0;
  auto unit_of = [&](int64_t row, int k, int here, float rstd, float (&u)[8]) {
    if constexpr (!IN8) {
      const Chunk<T> h =
          load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.h) + row * cols, R, k, here);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = to_f32(h.e[i]) * rstd;
    } else {
      const int col = (R.t + k * R.step) * 8, valid = here - col;
      const Codes c = load_codes<VEC>(a.codes + row * cols + col, valid);
      const float s = valid > 0 ? a.scales[row * a.groups + (col >> a.shift)] : 0.f;
      decode8(a.fmt, c, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = u[i] * s * rstd;
    }
  };
  for (int64_t row0 = (int64_t)blockIdx.x * R.here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * R.here) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    const int here = in ? cols : 0;
    const float rstd = in ? a.rstd[row] : 0.f;
    Chunk<T> gy[NV];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      gy[k] = load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.g_y) + row * cols, R, k, here);
      float w[8], u[8];
      unit_of(row, k, here, rstd, u);
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = to_f32(gy[k].e[i]);
        acc[k][i] = fmaf(g, u[i], acc[k][i]);
        dot = fmaf(g * w[i], u[i], dot);
      }
    }
    const float c = row_sum<LPR>(dot, buf, slot) * inv_cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8], u[8], g[8];
      unit_of(row, k, here, rstd, u);                  // from the caches
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = rstd * (to_f32(gy[k].e[i]) * w[i] - u[i] * c);
      if (a.g_h) {
        const Chunk<T> e =
            load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.g_h) + row * cols, R, k, here);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += to_f32(e.e[i]);
      }
      store_unit<T, VEC, SPREAD>(static_cast<T*>(a.g_x) + row * cols, R, k, here, g);
    }
  }
  if (a.partial) write_partial<LPR, NV, VEC, SPREAD>(a, R, acc, part);
}

// g_w[col] = sum of the blocks' partial sums, 32 columns a block, 32 slices of
// the partial rows side by side and then added in their order: no atomics, so
// the result does not vary.  4 us at 4096 columns, most of it the launch.
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

template <typename T, int FMT>
cudaError_t bwd(int dtype, const NormBwd& a, bool vec, int* blocks, cudaStream_t st) {
  cudaError_t e =
      vec ? bwd_ring<T, FMT, false>(a, blocks, st) : bwd_odd(dtype, a, blocks, st);
  if (e != cudaErrorNotSupported) return e;
  const Plan p = plan(a.cols, 512, 96);
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr ((L == 0 && N == 4) || (sizeof(T) == 4 && (FMT != 0 || L != 0))) {
      constexpr bool WIDE = sizeof(T) == 4 && L == 0 && N == 4;     // too wide for the ring
      *blocks = (int)grid(a.rows, p.here, resident(p.threads, bwd_regs(L, N), 0));
      if (vec && WIDE)
        norm_bwd_kernel<T, L, N, WIDE, FMT != 0><<<*blocks, p.threads, 0, st>>>(a);
      else
        norm_bwd_kernel<T, L, N, false, FMT != 0><<<*blocks, p.threads, 0, st>>>(a);
      e = cudaGetLastError();
    }
  });
  return e;
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t cols) {
  // of either way to lay out the rows
  int most = 0;
  for (bool odd : {false, true}) {
    const Plan p = plan(cols, 512, 96, odd);
    const int blocks = (int)grid(rows, p.here, resident(p.threads, bwd_regs(p.lpr, p.nv), 0));
    if (blocks > most) most = blocks;
  }
  return most;
}

cudaError_t launch_norm_bwd(int dtype, const NormBwd& in, void* g_w, cudaStream_t st) {
  NormBwd a = in;
  a.shift = group_shift(a.group);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const size_t al = chunk_align(dtype);
    const bool vec = a.cols % 8 == 0 && aligned_to(a.g_y, al) && aligned_to(a.h, al) &&
                     aligned_to(a.g_h, al) && aligned_to(a.g_x, al) &&
                     aligned_to(a.w, a.w_f32 ? 32 : 16) && aligned_to(a.codes, 8) &&
                     aligned_to(a.partial, 32);
    int blocks = 0;
    if (a.rows > 0) {
      const cudaError_t e = !a.codes              ? bwd<T, 0>(dtype, a, vec, &blocks, st)
                            : a.fmt == kFmtInt8   ? bwd<T, kFmtInt8>(dtype, a, vec, &blocks, st)
                                                  : bwd<T, kFmtE4m3>(dtype, a, vec, &blocks, st);
      if (e != cudaSuccess) return e;
    }
    if (g_w) {
      norm_gw_kernel<T><<<(unsigned)((a.cols + 31) / 32), 1024, 0, st>>>(
          a.partial, blocks, (int)a.cols, g_w, a.w_f32);
      return cudaGetLastError();
    }
    return cudaSuccess;
  });
}

}  // namespace bl
