// Kernels of the norms' forward (norm.cuh), which also save rows in 8 bits.
#pragma once

#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// Threads of a block that holds a row, at most.  The layer norm, which keeps the bias too,
// needs more than the 64 registers that 1024 threads leave each.
constexpr int fwd_threads(bool layer) { return layer ? 512 : 1024; }
template <bool LN>
using FwdArgs = std::conditional_t<LN, LayerNormFwd, NormFwd>;
// Registers a thread (the launch counts on them).
constexpr int fwd_regs(bool layer, bool norm, int nv) {
  return !layer ? (norm ? 64 : 48) : nv == 1 ? 64 : nv == 2 ? 80 : 128;
}

// The same for rows whose chunks are whole and aligned: a block takes rows
// gridDim.x apart, and x and r of the next S - 1 of them are on their way to
// shared memory meanwhile, each thread's chunks into places of its own.  Loading
// straight into registers instead leaves the memory idle while a row is reduced.
// Bound by HBM: 32760 x 5120 bf16 in 100 us, with the residual in 196 us
// (6.8 TB/s), with the residual to e4m3 in 175 us (6.7 TB/s; issue slots are 74%
// busy there).  FMT8: 0 without the 8-bit output, else its format.  NORM = false
// only saves x in 8 bits: the same walk without the norm.  LN: the layer norm, whose
// squares are summed of centred elements.
// ODD: rows of a 16-bit type that start anywhere.  Their aligned vectors go to
// the ring, and a chunk is shifted out of its own and the next thread's vector:
// one barrier more, and some 40 instructions a chunk and tensor (2561 columns: 23%
// of the copy rate element by element, 50% so, 63% with a residual).
// Registers are bounded by the numbers of threads alone (768 for 80 of them, where a thread has
// two chunks of rows that start anywhere): under __maxnreg__, even with the same bound, the
// kernels take more of them and spill (layer norm of 32760 x 2561 bf16 with a residual: 225 us,
// 199 so).
template <typename T, int LPR, int NV, int FMT8, int S, bool NORM, bool ODD, bool LN>
__global__ void __launch_bounds__(LN && ODD && NV == 2 ? 768 : LPR ? 256 : fwd_threads(LN))
    norm_fwd_ring_kernel(FwdArgs<LN> a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  static_assert(!ODD || CB == 16);
  static_assert(NORM || !LN);
  __shared__ float buf[2][LN ? 64 : 32];
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
  uint64_t w[NV][4], b[LN ? NV : 1][4];              // pairs of fp32, like h
  if constexpr (NORM) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      float f[8];
      load_weight8<T, !ODD>(a.w, a.w_f32, col, cols - col, f);
      if constexpr (LN) {
        // y is 0 behind the row, where it has no part in a group's largest value
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= cols - col) f[i] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
      if constexpr (LN) {
        load_bias8<T, !ODD>(a.b, a.w_f32, col, cols - col, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) b[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
      }
    }
  }
  // LN: one over the elements of a row that the thread's warp holds, and those of the
  // warp whose number is the thread's lane
  float inv_part = inv_cols, inv_lane = 0.f, n_lane = 0.f;
  if constexpr (LN && LPR == 0) {
    auto held = [&](int warp) {
      int n = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int left = cols - (warp * 32 + k * R.step) * 8;
        n += left < 0 ? 0 : left < 256 ? left : 256;
      }
      return n;
    };
    const int mine_n = held(threadIdx.x >> 5), lane_n = held(threadIdx.x & 31);
    inv_part = mine_n ? 1.f / (float)mine_n : 0.f;
    if ((threadIdx.x & 31) < (blockDim.x >> 5)) {
      n_lane = (float)lane_n;
      inv_lane = lane_n ? 1.f / n_lane : 0.f;
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
          for (int i = 0; i < 4; ++i)
            ss = LN ? fadd2(h[k][i], ss) : ffma2(h[k][i], h[k][i], ss);
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
      float sum = s0 + s1, mean = 0.f;
      if constexpr (!LN) {
        sum = row_sum<LPR>(sum, buf, slot);
      } else {
        // the squares around the mean of the elements that the warp's lanes (LPR of them)
        // hold; over the block the parts' means are put right, so one barrier does
        constexpr int W = LPR ? LPR : 32;
        sum = lanes_sum(sum, W);
        mean = LPR ? mean_of(sum, inv_part, (float)cols) : sum * inv_part;
        ss = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int valid = in ? cols - (R.t + k * R.step) * 8 : 0;
          const float off = valid > 0 ? -mean : 0.f;     // h is 0 where there is no chunk
          const uint64_t mm = f2_pack(off, off);
          if (!ODD || valid >= 8 || valid <= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint64_t d = fadd2(h[k][i], mm);
              ss = ffma2(d, d, ss);
            }
          } else {                                       // the row's end: the warp that has it
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float lo, hi;
              f2_unpack(fadd2(h[k][i], mm), lo, hi);
              const uint64_t d = f2_pack(2 * i < valid ? lo : 0.f, 2 * i + 1 < valid ? hi : 0.f);
              ss = ffma2(d, d, ss);
            }
          }
        }
        f2_unpack(ss, s0, s1);
        float squares = lanes_sum(s0 + s1, W);
        if constexpr (LPR == 0) {
          const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
          if (lane == 0) {
            buf[slot][warp] = sum;
            buf[slot][32 + warp] = squares;
          }
          __syncthreads();
          const float part = lane < warps ? buf[slot][lane] : 0.f;
          squares = lane < warps ? buf[slot][32 + lane] : 0.f;
          mean = mean_of(lanes_sum(part, 32), inv_cols, (float)cols);
          const float off = part * inv_lane - mean;      // of the mean of warp `lane`
          squares = lanes_sum(fmaf(off * off, n_lane, squares), 32);
          slot ^= 1;
        }
        sum = squares;
        if (R.t == 0 && in && a.mean) a.mean[row] = mean;
      }
      const float rstd = rsqrtf(fmaf(sum, inv_cols, a.eps));
      if (R.t == 0 && in && a.rstd) a.rstd[row] = rstd;
      const uint64_t rr = f2_pack(rstd, rstd), mm = f2_pack(-mean, -mean);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const bool has = in && (R.t + k * R.step) * 8 < cols;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[k][i] = LN ? ffma2(fmul2(fadd2(h[k][i], mm), rr), w[k][i], b[LN ? k : 0][i])
                       : fmul2(fmul2(h[k][i], rr), w[k][i]);
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

// Launches the ring kernel on rows that it takes, else cudaErrorNotSupported.
template <typename T, int FMT8, bool NORM, bool ODD, bool LN>
cudaError_t fwd_ring(const FwdArgs<LN>& a, cudaStream_t st) {
  const Plan p = plan(a.cols, fwd_threads(LN), 64, ODD);
  cudaError_t e = cudaErrorNotSupported;
  if (p.threads > fwd_threads(LN)) return e;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    // layer_fwd_pairs takes aligned rows of one chunk a thread, but for a scale a row
    constexpr bool PAIRS = LN && !ODD && FMT8 == 0 && L == 0 && N == 1;
    if constexpr ((N <= 2 || (LN && L == 0)) && !PAIRS) {
      constexpr size_t UNIT = (size_t)N * (NORM ? 2 : 1) * sizeof(Chunk<T>);  // a thread's of a stage
      const size_t stage = p.threads * UNIT;
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_fwd_ring_kernel<T, L, N, FMT8, S, NORM, ODD, LN>;
        const size_t smem = S * stage;
        e = allow_smem<k>((int)kMaxSmem);
        if (e != cudaSuccess) return;
        k<<<grid(a.rows, p.here, fwd_blocks(a.rows, p, fwd_regs(LN, NORM, N), smem)), p.threads, smem,
            st>>>(a);
        e = cudaGetLastError();
      };
      constexpr int MOST = NORM || ODD ? 3 : 2, TOP = fwd_threads(LN);
      if constexpr (L != 0 || N == 1 || MOST * UNIT * TOP <= kMaxSmem / 2) {
        ring(Int<MOST>());
      } else {
        if constexpr (MOST * UNIT * fewest_threads(N, TOP) <= kMaxSmem / 2)
          if (MOST * stage <= kMaxSmem / 2) {
            ring(Int<MOST>());
            return;
          }
        if (2 * stage <= kMaxSmem) ring(Int<2>());
      }
    }
  });
  return e;
}

// Rows that the ring does not take, straight from global memory: fp32 that starts
// anywhere or is too wide, and 16-bit rows that start anywhere of more than 16376
// columns.  OUT8: with the 8-bit output, whose
// groups are neighbours, so those rows keep to chunks.
// (Arguments that are not marked constant cost registers: fp32 of 2561 columns 155 us, 144 so.)
template <typename T, int LPR, int NV, bool VEC, bool OUT8, bool LN>
__global__ void __launch_bounds__(LPR ? 256 : fwd_threads(LN))
    norm_fwd_kernel(const __grid_constant__ FwdArgs<LN> a) {
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
        s0 = LN ? s0 + h[k][i] : fmaf(h[k][i], h[k][i], s0);
        s1 = LN ? s1 + h[k][i + 1] : fmaf(h[k][i + 1], h[k][i + 1], s1);
      }
    }
    float ss = row_sum<LPR>(s0 + s1, buf, slot);
    if constexpr (LN) {
      const float mean = mean_of(ss, inv_cols, (float)cols);
      if (R.t == 0 && in && a.mean) a.mean[row] = mean;
      s0 = s1 = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          h[k][i] = col_of<SPREAD>(R, k, i) < here ? h[k][i] - mean : 0.f;
          h[k][i + 1] = col_of<SPREAD>(R, k, i + 1) < here ? h[k][i + 1] - mean : 0.f;
          s0 = fmaf(h[k][i], h[k][i], s0);
          s1 = fmaf(h[k][i + 1], h[k][i + 1], s1);
        }
      ss = row_sum<LPR>(s0 + s1, buf, slot);
    }
    const float rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
    if (R.t == 0 && in && a.rstd) a.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8];
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[i];
      if constexpr (LN) {
        if (a.b) {
          weight_unit<T, VEC, SPREAD>(a.b, a.w_f32, R, k, cols, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k][i] += w[i];
        }
      }
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

template <typename T, int FMT8, bool LN>
cudaError_t fwd(int dtype, const FwdArgs<LN>& a, bool vec, cudaStream_t st) {
  cudaError_t e = cudaErrorNotSupported;
  if constexpr (LN) {
    e = vec ? layer_fwd_pairs(dtype, a, st) : layer_fwd_odd(dtype, a, st);
  } else {
    if (!vec) e = fwd_odd(dtype, true, a, st);
  }
  if (vec && e == cudaErrorNotSupported) e = fwd_ring<T, FMT8, true, false, LN>(a, st);
  if (e != cudaErrorNotSupported) return e;
  const Plan p = plan(a.cols, fwd_threads(LN), 64);
  const unsigned g = grid(a.rows, p.here, kSMs * 32);
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    constexpr int MOST = LN ? 4 : 2;                  // chunks a thread of the widest rows
    if constexpr (N <= (L ? 2 : MOST) && (sizeof(T) == 4 || (L == 0 && N == MOST))) {
      constexpr bool WIDE = sizeof(T) == 4 && L == 0 && N == MOST;  // too wide for the ring
      if (vec && WIDE)
        norm_fwd_kernel<T, L, N, WIDE, FMT8 != 0, LN><<<g, p.threads, 0, st>>>(a);
      else
        norm_fwd_kernel<T, L, N, false, FMT8 != 0, LN><<<g, p.threads, 0, st>>>(a);
      e = cudaGetLastError();
    }
  });
  return e;
}

// The forward's launch on rows of any kind.
template <bool LN>
cudaError_t launch_fwd_of(int dtype, const FwdArgs<LN>& in, cudaStream_t st) {
  FwdArgs<LN> a = in;
  if (a.rows == 0) return cudaSuccess;
  a.shift = group_shift(a.group);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const size_t al = chunk_align(dtype);
    bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 && a.r_stride % 8 == 0 &&
               aligned_to(a.x, al) && aligned_to(a.r, al) && aligned_to(a.h, al) &&
               aligned_to(a.y, al) && aligned_to(a.w, a.w_f32 ? 32 : 16) && aligned_to(a.codes, 8);
    if constexpr (LN) vec = vec && aligned_to(a.b, a.w_f32 ? 32 : 16);
    const int fmt = a.codes ? a.fmt : 0;
    return fmt == 0          ? fwd<T, 0, LN>(dtype, a, vec, st)
           : fmt == kFmtInt8 ? fwd<T, kFmtInt8, LN>(dtype, a, vec, st)
                             : fwd<T, kFmtE4m3, LN>(dtype, a, vec, st);
  });
}

}  // namespace

}  // namespace bl
