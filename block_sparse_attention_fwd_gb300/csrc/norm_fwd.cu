// Forward of the root-mean-square norm (norm.cuh) and row-wise saving in 8 bits.
#include "norm_fwd.cuh"

namespace bl {

namespace {

// Rows that the ring does not take, straight from global memory: fp32 that starts
// anywhere or is too wide, and 16-bit rows that start anywhere of more than 16376
// columns.  OUT8: with the 8-bit output, whose
// groups are neighbours, so those rows keep to chunks.
template <typename T, int LPR, int NV, bool VEC, bool OUT8>
__global__ void __launch_bounds__(LPR ? 256 : 1024) norm_fwd_kernel(NormFwd a) {
  __shared__ float buf[2][32];
  constexpr bool SPREAD = !VEC && !OUT8;
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  int slot = 0;
  // the loop is uniform over the block (lanes past the last row work on zeros)
  for (int64_t row0 = (int64_t)blockIdx.x * R.here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * R.here) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    const int here = in ? cols : 0;
    float h[NV][8];
    float s0 = 0.f, s1 = 0.f;                          // as the ring kernel sums them
    Chunk<T> x[NV], r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x[k] = load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.x) + row * a.x_stride, R, k, here);
      if (a.r)
        r[k] = load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.r) + row * a.r_stride, R, k, here);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = to_f32(x[k].e[i]);
      if (a.r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += to_f32(r[k].e[i]);
        if (a.h) store_unit<T, VEC, SPREAD>(static_cast<T*>(a.h) + row * cols, R, k, here, h[k]);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        s0 = fmaf(h[k][i], h[k][i], s0);
        s1 = fmaf(h[k][i + 1], h[k][i + 1], s1);
      }
    }
    const float ss = row_sum<LPR>(s0 + s1, buf, slot);
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (R.t == 0 && in && a.rstd) a.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8];
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[i];
      if (a.y) store_unit<T, VEC, SPREAD>(static_cast<T*>(a.y) + row * cols, R, k, here, h[k]);
      if constexpr (OUT8) {
        const int col = (R.t + k * R.step) * 8;
        const int valid = in ? cols - col : 0;
        float m = amax8(h[k]);
        if (a.group) {
          m = lanes_amax(m, min(a.group / 8, LPR ? LPR : 32));
          const float scale = scale_of(m, a.fmt);
          store_codes<VEC>(a.codes + row * cols + col, encode8(a.fmt, h[k], scale), valid);
          if (valid > 0 && (col & (a.group - 1)) == 0)
            a.scales[row * a.groups + (col >> a.shift)] = scale;
        } else {
          top = amax2(top, m);
        }
      }
    }
    if constexpr (OUT8) {
      if (!a.group) {
        if constexpr (LPR != 0) {
          top = lanes_amax(top, LPR);
        } else {
          top = block_amax(top, buf, slot);
          slot ^= 1;
        }
        const float scale = scale_of(top, a.fmt);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int col = (R.t + k * R.step) * 8;
          const int valid = in ? cols - col : 0;
          store_codes<VEC>(a.codes + row * cols + col, encode8(a.fmt, h[k], scale), valid);
        }
        if (R.t == 0 && in) a.scales[row] = scale;
      }
    }
  }
}

template <typename T, int FMT8>
cudaError_t fwd(int dtype, const NormFwd& a, bool vec, cudaStream_t st) {
  cudaError_t e = vec ? fwd_ring<T, FMT8, true, false>(a, st) : fwd_odd(dtype, true, a, st);
  if (e != cudaErrorNotSupported) return e;
  const Plan p = plan(a.cols, 1024, 64);
  const unsigned g = grid(a.rows, p.here, kSMs * 32);
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr (N <= 2 && (sizeof(T) == 4 || (L == 0 && N == 2))) {
      constexpr bool WIDE = sizeof(T) == 4 && L == 0 && N == 2;     // too wide for the ring
      if (vec && WIDE)
        norm_fwd_kernel<T, L, N, WIDE, FMT8 != 0><<<g, p.threads, 0, st>>>(a);
      else
        norm_fwd_kernel<T, L, N, false, FMT8 != 0><<<g, p.threads, 0, st>>>(a);
      e = cudaGetLastError();
    }
  });
  return e;
}

}  // namespace

cudaError_t launch_norm_fwd(int dtype, const NormFwd& in, cudaStream_t st) {
  NormFwd a = in;
  if (a.rows == 0) return cudaSuccess;
  a.shift = group_shift(a.group);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const size_t al = chunk_align(dtype);
    const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 && a.r_stride % 8 == 0 &&
                     aligned_to(a.x, al) && aligned_to(a.r, al) && aligned_to(a.h, al) &&
                     aligned_to(a.y, al) && aligned_to(a.w, a.w_f32 ? 32 : 16) &&
                     aligned_to(a.codes, 8);
    const int fmt = a.codes ? a.fmt : 0;
    return fmt == 0          ? fwd<T, 0>(dtype, a, vec, st)
           : fmt == kFmtInt8 ? fwd<T, kFmtInt8>(dtype, a, vec, st)
                             : fwd<T, kFmtE4m3>(dtype, a, vec, st);
  });
}

cudaError_t launch_row_save(int dtype, const ActSave& s, cudaStream_t st) {
  if (s.cols > 16384) return cudaErrorNotSupported;
  NormFwd a{};
  a.rows = s.rows; a.cols = s.cols; a.x_stride = s.x_stride; a.groups = s.groups;
  a.x = s.x; a.codes = s.codes; a.scales = s.scales;
  a.group = s.group; a.fmt = s.fmt; a.shift = group_shift(s.group);
  const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 &&
                   aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 8);
  if (!vec) return fwd_odd(dtype, false, a, st);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return s.fmt == kFmtInt8 ? fwd_ring<T, kFmtInt8, false, false>(a, st)
                             : fwd_ring<T, kFmtE4m3, false, false>(a, st);
  });
}

}  // namespace bl
