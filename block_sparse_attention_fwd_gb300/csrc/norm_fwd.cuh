// Kernels of the root-mean-square norm's forward (norm.cuh), which also save rows
// in 8 bits.
#pragma once

#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// The same for rows whose chunks are whole and aligned: a block takes rows
// gridDim.x apart, and x and r of the next S - 1 of them are on their way to
// shared memory meanwhile, each thread's chunks into places of its own.  Loading
// straight into registers instead leaves the memory idle while a row is reduced.
// Bound by HBM: 32760 x 5120 bf16 in 100 us, with the residual in 196 us
// (6.8 TB/s), with the residual to e4m3 in 175 us (6.7 TB/s; issue slots are 74%
// busy there).  FMT8: 0 without the 8-bit output, else its format.  NORM = false
// only saves x in 8 bits: the same walk without the norm.
// ODD: rows of a 16-bit type that start anywhere.  Their aligned vectors go to
// the ring, and a chunk is shifted out of its own and the next thread's vector:
// one barrier more, and some 40 instructions a chunk and tensor (2561 columns: 23%
// of the copy rate element by element, 50% so, 63% with a residual).
template <typename T, int LPR, int NV, int FMT8, int S, bool NORM, bool ODD>
__global__ void __launch_bounds__(LPR ? 256 : 1024) norm_fwd_ring_kernel(NormFwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  static_assert(!ODD || CB == 16);
  __shared__ float buf[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const int nt = blockDim.x;
  const int64_t stride = (int64_t)gridDim.x * R.here;
  const int plane = NV * nt * CB;                    // bytes of x in a stage; r's follow
  uint8_t* const mine = ring + threadIdx.x * 16;
  auto fetch = [&](int s, int64_t row) {
    if (row < a.rows) {
      const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
      const T* r = static_cast<const T*>(a.r) + row * a.r_stride;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = R.t + k * R.step;
        uint8_t* p = mine + s * (NORM ? 2 : 1) * plane + k * nt * CB;
        if constexpr (ODD) {
          if (c * 8 < cols + 8) {
            copy_odd(p, x, c, cols);
            if (NORM && a.r) copy_odd(p + plane, r, c, cols);
          }
        } else if (c * 8 < cols) {
#pragma unroll
          for (int v = 0; v < CB / 16; ++v) {
            constexpr int E = 16 / sizeof(T);
            copy_chunk<CB>(p + v * nt * 16, x + c * 8 + v * E);
            if (NORM && a.r) copy_chunk<CB>(p + plane + v * nt * 16, r + c * 8 + v * E);
          }
        }
      }
    }
    copy_commit();
  };
  // a chunk out of the thread's place p, of a row at this address
  auto chunk = [&](const uint8_t* p, const T* row) {
    Chunk<T> c;
    if constexpr (ODD) {
      c = chunk_odd<T, LPR>(p, R.t, nt, row);
    } else {
#pragma unroll
      for (int v = 0; v < CB / 16; ++v)
        reinterpret_cast<uint4*>(&c)[v] = *reinterpret_cast<const uint4*>(p + v * nt * 16);
    }
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
      load_weight8<T, !ODD>(a.w, a.w_f32, col, cols - col, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
    }
  }
  int slot = 0, now = 0, fill = S - 1;
  for (int64_t row0 = first; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + R.mine;
    const bool in = LPR == 0 || row < a.rows;
    if constexpr (ODD) {
      // the next thread's vectors too have to be there, and every thread has to be
      // done with the stage that is filled next
      copy_wait<S - 2>();
      if constexpr (LPR) __syncwarp(); else __syncthreads();
      fetch(fill, row + (S - 1) * stride);
    } else {
      fetch(fill, row + (S - 1) * stride);
      copy_wait<S - 1>();
    }
    uint64_t h[NV][4], ss = 0;
    const int64_t at = row * cols + R.t * 8;
    auto write = [&](void* to, int k, const uint64_t (&f)[4], bool has) {
      if constexpr (ODD) {
        const int c = R.t + k * R.step;
        uint32_t words[4];
        pack_words<T>(f, words);
        store_anywhere<4>(reinterpret_cast<uint8_t*>(static_cast<T*>(to) + row * cols), c,
                          has ? min(cols - c * 8, 8) : 0, cols, lane_in_front(R), lane_behind(R),
                          words);
      } else {
        if (has) store8(static_cast<T*>(to) + at + k * R.step * 8, f);
      }
    };
    auto write_codes = [&](int k, const Codes& codes, bool has) {
      if constexpr (ODD) {
        const int c = R.t + k * R.step;
        store_anywhere<2>(a.codes + row * cols, c, has ? min(cols - c * 8, 8) : 0, cols,
                          lane_in_front(R), lane_behind(R), codes.w);
      } else {
        if (has) store_codes<true>(a.codes + at + k * R.step * 8, codes, 8);
      }
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool has = in && (R.t + k * R.step) * 8 < cols;
      if (has) {
        const uint8_t* p = mine + now * (NORM ? 2 : 1) * plane + k * nt * CB;
        unpack2(chunk(p, static_cast<const T*>(a.x) + row * a.x_stride), h[k]);
        if (NORM && a.r) {
          uint64_t r[4];
          unpack2(chunk(p + plane, static_cast<const T*>(a.r) + row * a.r_stride), r);
#pragma unroll
          for (int i = 0; i < 4; ++i) h[k][i] = fadd2(h[k][i], r[i]);
        }
        if constexpr (NORM) {
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = ffma2(h[k][i], h[k][i], ss);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[k][i] = 0;
      }
      if (NORM && a.h) write(a.h, k, h[k], has);
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
        if (a.y) write(a.y, k, h[k], has);
      }
    }
    if constexpr (FMT8 != 0) {
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int col = (R.t + k * R.step) * 8;
        const bool has = in && col < cols;
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(h[k][i], f[2 * i], f[2 * i + 1]);
        const float m = amax8(f);
        if (a.group) {
          const float scale = scale_of(lanes_amax(m, min(a.group / 8, LPR ? LPR : 32)), FMT8);
          write_codes(k, encode8<FMT8>(f, scale), has);
          if (has && (col & (a.group - 1)) == 0)
            a.scales[row * a.groups + (col >> a.shift)] = scale;
        } else {
          top = amax2(top, m);
        }
      }
      if (!a.group) {
        if constexpr (LPR != 0) {
          top = lanes_amax(top, LPR);
        } else {
          top = block_amax(top, buf, slot);
          slot ^= 1;
        }
        const float scale = scale_of(top, FMT8);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(h[k][i], f[2 * i], f[2 * i + 1]);
          write_codes(k, encode8<FMT8>(f, scale), in && (R.t + k * R.step) * 8 < cols);
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

// Launches the ring kernel on rows that it takes, else cudaErrorNotSupported.
template <typename T, int FMT8, bool NORM, bool ODD>
cudaError_t fwd_ring(const NormFwd& a, cudaStream_t st) {
  const Plan p = plan(a.cols, 1024, 64, ODD);
  cudaError_t e = cudaErrorNotSupported;
  if (p.threads > 1024) return e;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr (N <= 2) {
      const size_t stage = (size_t)N * p.threads * (NORM ? 2 : 1) * sizeof(Chunk<T>);
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_fwd_ring_kernel<T, L, N, FMT8, S, NORM, ODD>;
        const size_t smem = S * stage;
        e = allow_smem<k>();
        if (e != cudaSuccess) return;
        k<<<grid(a.rows, p.here, fwd_blocks(a.rows, p, NORM ? 64 : 48, smem)), p.threads, smem,
            st>>>(a);
        e = cudaGetLastError();
      };
      constexpr int MOST = NORM || ODD ? 3 : 2;
      if (L != 0 || N == 1 || MOST * stage <= kMaxSmem / 2)
        ring(Int<MOST>());
      else if (2 * stage <= kMaxSmem)
        ring(Int<L == 0 && N == 2 ? 2 : MOST>());
    }
  });
  return e;
}

}  // namespace

}  // namespace bl
