// Forward of the root-mean-square norm (norm.cuh) and row-wise saving in 8 bits.
#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// Any rows, straight from global memory.  OUT8: with the 8-bit output.
template <typename T, int LPR, int NV, bool VEC, bool OUT8>
__global__ void __launch_bounds__(LPR ? 256 : 1024) norm_fwd_kernel(NormFwd a) {
  __shared__ float buf[2][32];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  int slot = 0;
  // the loop is uniform over the block (lanes past the last row work on zeros)
  for (int64_t row0 = (int64_t)blockIdx.x * R.here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * R.here) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    float h[NV][8];
    float s0 = 0.f, s1 = 0.f;                          // as the ring kernel sums them
    Chunk<T> x[NV], r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      const int valid = in ? cols - col : 0;
      x[k] = load8<T, VEC>(static_cast<const T*>(a.x) + row * a.x_stride + col, valid);
      if (a.r) r[k] = load8<T, VEC>(static_cast<const T*>(a.r) + row * a.r_stride + col, valid);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      const int valid = in ? cols - col : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = to_f32(x[k].e[i]);
      if (a.r) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += to_f32(r[k].e[i]);
        if (a.h) store8<T, VEC>(static_cast<T*>(a.h) + row * cols + col, h[k], valid);
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
      const int col = (R.t + k * R.step) * 8;
      const int valid = in ? cols - col : 0;
      float w[8];
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[i];
      if (a.y) store8<T, VEC>(static_cast<T*>(a.y) + row * cols + col, h[k], valid);
      if constexpr (OUT8) {
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

// The same for rows whose chunks are whole and aligned: a block takes rows
// gridDim.x apart, and x and r of the next S - 1 of them are on their way to
// shared memory meanwhile, each thread's chunks into places of its own.  Loading
// straight into registers instead leaves the memory idle while a row is reduced.
// Bound by HBM: 32760 x 5120 bf16 in 100 us, with the residual in 196 us
// (6.8 TB/s), with the residual to e4m3 in 175 us (6.7 TB/s; issue slots are 74%
// busy there).  FMT8: 0 without the 8-bit output, else its format.  NORM = false
// only saves x in 8 bits with one scale a row: the same walk without the norm.
template <typename T, int LPR, int NV, int FMT8, int S, bool NORM>
__global__ void __launch_bounds__(LPR ? 256 : 1024) norm_fwd_ring_kernel(NormFwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  __shared__ float buf[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const int nt = blockDim.x;
  const int64_t stride = (int64_t)gridDim.x * R.here;
  // the thread's place in stage s, chunk k: x, and r another nt * CB behind
  auto place = [&](int s, int k) -> uint8_t* {
    return ring + (s * NV + k) * nt * (NORM ? 2 : 1) * CB + threadIdx.x * 16;
  };
  auto fetch = [&](int s, int64_t row) {
    if (row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* r = static_cast<const T*>(a.r) + row * a.r_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (R.t + k * R.step) * 8;
        if (col < cols) {
          uint8_t* p = place(s, k);
#pragma unroll
          for (int v = 0; v < CB / 16; ++v) {
            copy_async<16>(p + v * nt * 16, x + col + v * (16 / sizeof(T)));
            if (NORM && a.r) copy_async<16>(p + nt * CB + v * nt * 16, r + col + v * (16 / sizeof(T)));
          }
        }
      }
    }
    copy_commit();
  };
  auto chunk = [&](const uint8_t* p) {
    Chunk<T> c;
#pragma unroll
    for (int v = 0; v < CB / 16; ++v)
      reinterpret_cast<uint4*>(&c)[v] = *reinterpret_cast<const uint4*>(p + v * nt * 16);
    return c;
  };
  const int64_t first = (int64_t)blockIdx.x * R.here;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(s, first + s * stride + R.mine);
  uint64_t w[NV][4];                                 // pairs of fp32, like h
  if constexpr (NORM) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      float f[8];
      load_weight8<T, true>(a.w, a.w_f32, col, cols - col, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
    }
  }
  int slot = 0, now = 0, fill = S - 1;
  for (int64_t row0 = first; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + R.mine;
    const bool in = LPR == 0 || row < a.rows;
    fetch(fill, row + (S - 1) * stride);
    copy_wait<S - 1>();
    uint64_t h[NV][4], ss = 0;
    const int64_t at = row * cols + R.t * 8;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool has = in && (R.t + k * R.step) * 8 < cols;
      if (has) {
        const uint8_t* p = place(now, k);
        unpack2(chunk(p), h[k]);
        if (NORM && a.r) {
          uint64_t r[4];
          unpack2(chunk(p + nt * CB), r);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[k][i] = fadd2(h[k][i], r[i]);
          if (a.h) store8(static_cast<T*>(a.h) + at + k * R.step * 8, h[k]);
        }
        if constexpr (NORM) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = ffma2(h[k][i], h[k][i], ss);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[k][i] = 0;
      }
    }
    if constexpr (NORM) {
      float s0, s1;
      f2_unpack(ss, s0, s1);
      const float sum = row_sum<LPR>(s0 + s1, buf, slot);
      const float rstd = rsqrtf(fmaf(sum, inv_cols, a.eps));
      if (R.t == 0 && in && a.rstd) a.rstd[row] = rstd;
      const uint64_t rr = f2_pack(rstd, rstd);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const bool has = in && (R.t + k * R.step) * 8 < cols;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[k][i] = fmul2(fmul2(h[k][i], rr), w[k][i]);
        if (a.y && has) store8(static_cast<T*>(a.y) + at + k * R.step * 8, h[k]);
      }
    }
    if constexpr (FMT8 != 0) {
      float top = 0.f;
      const bool grouped = NORM && a.group;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (R.t + k * R.step) * 8;
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(h[k][i], f[2 * i], f[2 * i + 1]);
        const float m = amax8(f);
        if (grouped) {
          const float scale = scale_of(lanes_amax(m, min(a.group / 8, LPR ? LPR : 32)), FMT8);
          if (in && col < cols) {
            store_codes<true>(a.codes + at + k * R.step * 8, encode8<FMT8>(f, scale), 8);
            if ((col & (a.group - 1)) == 0) a.scales[row * a.groups + (col >> a.shift)] = scale;
          }
        } else {
          top = amax2(top, m);
        }
      }
      if (!grouped) {
        if constexpr (LPR != 0) {
          top = lanes_amax(top, LPR);
        } else {
          top = block_amax(top, buf, slot);
          slot ^= 1;
        }
        const float scale = scale_of(top, FMT8);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (!in || (R.t + k * R.step) * 8 >= cols) continue;
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(h[k][i], f[2 * i], f[2 * i + 1]);
          store_codes<true>(a.codes + at + k * R.step * 8, encode8<FMT8>(f, scale), 8);
        }
        if (R.t == 0 && in) a.scales[row] = scale;
      }
    }
    fill = fill == S - 1 ? 0 : fill + 1;
    now = now == S - 1 ? 0 : now + 1;
  }
}

// Blocks of the ring kernel.  One block for each that is resident runs them all
// in step: the reads of all blocks and then their writes come in bursts.  Eight
// times as many, as far as a block keeps about six rows, take turns out of step and
// work on neighbouring rows: 5120 columns 84 -> 99% of the copy rate without and
// 90 -> 101% with a residual, 128 columns 83 -> 96%; blocks of fewer rows lose it
// again to filling their rings (4096 rows of 4096: 87 -> 70% at eight times).
int fwd_blocks(int64_t rows, const Plan& p, int regs, size_t smem) {
  const int once = resident(p.threads, regs, smem);
  int64_t times = rows / ((int64_t)once * p.here * 6);
  if (times > 8) times = 8;
  if (times < 1) times = 1;
  return (int)(once * times);
}

template <typename T, int FMT8, bool NORM>
cudaError_t fwd(const NormFwd& a, bool vec, cudaStream_t st) {
  const Plan p = plan(a.cols, 1024, 64);
  cudaError_t e = cudaSuccess;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr (N <= 2) {
      const size_t stage = (size_t)N * p.threads * (NORM ? 2 : 1) * sizeof(Chunk<T>);
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_fwd_ring_kernel<T, L, N, FMT8, S, NORM>;
        const size_t smem = S * stage;
        e = allow_smem<k>();
        if (e == cudaSuccess)
          k<<<grid(a.rows, p.here, fwd_blocks(a.rows, p, NORM ? 64 : 48, smem)), p.threads, smem, st>>>(a);
      };
      if (vec && (L != 0 || N == 1 || 3 * stage <= kMaxSmem / 2))
        ring(Int<NORM ? 3 : 2>());
      else if (vec && 2 * stage <= kMaxSmem)
        ring(Int<(L == 0 && N == 2) || !NORM ? 2 : 3>());
      else if constexpr (!NORM)
        e = cudaErrorNotSupported;
      else if (vec && sizeof(T) == 4 && L == 0 && N == 2)   // too wide for the ring
        norm_fwd_kernel<T, L, N, sizeof(T) == 4 && L == 0 && N == 2, FMT8 != 0>
            <<<grid(a.rows, p.here, kSMs * 32), p.threads, 0, st>>>(a);
      else
        norm_fwd_kernel<T, L, N, false, FMT8 != 0>
            <<<grid(a.rows, p.here, kSMs * 32), p.threads, 0, st>>>(a);
    }
  });
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_norm_fwd(int dtype, const NormFwd& in, cudaStream_t st) {
  NormFwd a = in;
  if (a.rows == 0) return cudaSuccess;
  a.shift = group_shift(a.group);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 && a.r_stride % 8 == 0 &&
                     aligned_to(a.x, 16) && aligned_to(a.r, 16) && aligned_to(a.h, 16) &&
                     aligned_to(a.y, 16) && aligned_to(a.w, 16) && aligned_to(a.codes, 8);
    const int fmt = a.codes ? a.fmt : 0;
    return fmt == 0          ? fwd<T, 0, true>(a, vec, st)
           : fmt == kFmtInt8 ? fwd<T, kFmtInt8, true>(a, vec, st)
                             : fwd<T, kFmtE4m3, true>(a, vec, st);
  });
}

cudaError_t launch_row_save(int dtype, const ActSave& s, cudaStream_t st) {
  NormFwd a{};
  a.rows = s.rows; a.cols = s.cols; a.x_stride = s.x_stride; a.groups = 1;
  a.x = s.x; a.codes = s.codes; a.scales = s.scales;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    if (a.cols > 16384 || a.cols % 8 || a.x_stride % 8 || !aligned_to(a.x, 16) ||
        !aligned_to(a.codes, 8) || (sizeof(T) == 4 && a.cols > 8192))
      return cudaErrorNotSupported;
    return s.fmt == kFmtInt8 ? fwd<T, kFmtInt8, false>(a, true, st)
                             : fwd<T, kFmtE4m3, false>(a, true, st);
  });
}

}  // namespace bl
