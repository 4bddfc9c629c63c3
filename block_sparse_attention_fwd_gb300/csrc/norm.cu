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
#include <atomic>

#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

// A row is held by LPR lanes of a warp (8, 16 or 32, each with NV chunks: up to
// 1024 columns) or by the whole block (LPR = 0).
template <int LPR>
struct Rows {
  int here, mine, t, step;      // rows of the block, this thread's; its first chunk and their distance
  __device__ __forceinline__ Rows() {
    if constexpr (LPR != 0) {
      here = blockDim.x / LPR;
      mine = threadIdx.x / LPR;
      t = threadIdx.x % LPR;
      step = LPR;
    } else {
      here = 1;
      mine = 0;
      t = threadIdx.x;
      step = blockDim.x;
    }
  }
};
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float (*buf)[32], int& slot) {
  if constexpr (LPR != 0) return lanes_sum(v, LPR);
  v = block_sum(v, buf, slot);
  slot ^= 1;
  return v;
}

// FMT8: 0 without the 8-bit output, else its format.
template <typename T, int LPR, int NV, bool VEC, int FMT8>
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
    float ss = 0.f;
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
      for (int i = 0; i < 8; ++i) ss = fmaf(h[k][i], h[k][i], ss);
    }
    ss = row_sum<LPR>(ss, buf, slot);
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
      if constexpr (FMT8 != 0) {
        float m = amax8(h[k]);
        if (a.group) {
          m = lanes_amax(m, min(a.group / 8, LPR ? LPR : 32));
          const float scale = scale_of(m, FMT8);
          store_codes<VEC>(a.codes + row * cols + col, encode8<FMT8>(h[k], scale), valid);
          if (valid > 0 && (col & (a.group - 1)) == 0)
            a.scales[row * a.groups + (col >> a.shift)] = scale;
        } else {
          top = amax2(top, m);
        }
      }
    }
    if constexpr (FMT8 != 0) {
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
          const int col = (R.t + k * R.step) * 8;
          const int valid = in ? cols - col : 0;
          store_codes<VEC>(a.codes + row * cols + col, encode8<FMT8>(h[k], scale), valid);
        }
        if (R.t == 0 && in) a.scales[row] = scale;
      }
    }
  }
}

// The same for rows whose chunks are whole and aligned, on a grid that fills the
// GPU once: a block takes rows gridDim.x apart, and x and r of the next S - 1
// of them are on their way to shared memory meanwhile, each thread's chunks into
// places of its own.  Loading straight into registers instead leaves the
// memory idle while a row is reduced.  NORM = false only saves x in 8 bits with
// one scale a row: the same walk without the norm.
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
    return ring + (s * NV + k) * nt * 2 * CB + threadIdx.x * 16;
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
  float w[NV][8];
  if constexpr (NORM) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      load_weight8<T, true>(a.w, a.w_f32, col, cols - col, w[k]);
    }
  }
  int slot = 0, now = 0;
  for (int64_t row0 = first; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    fetch(now == 0 ? S - 1 : now - 1, row + (S - 1) * stride);
    copy_wait<S - 1>();
    float h[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      if (in && col < cols) {
        const uint8_t* p = place(now, k);
        const Chunk<T> x = chunk(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = to_f32(x.e[i]);
        if (NORM && a.r) {
          const Chunk<T> r = chunk(p + nt * CB);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k][i] += to_f32(r.e[i]);
          if (a.h) store8<T, true>(static_cast<T*>(a.h) + row * cols + col, h[k], 8);
        }
        if constexpr (NORM) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(h[k][i], h[k][i], ss);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = 0.f;
      }
    }
    float rstd = 1.f;
    if constexpr (NORM) {
      ss = row_sum<LPR>(ss, buf, slot);
      rstd = rsqrtf(fmaf(ss, inv_cols, a.eps));
      if (R.t == 0 && in && a.rstd) a.rstd[row] = rstd;
    }
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      const int valid = in && col < cols ? 8 : 0;
      if constexpr (NORM) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[k][i];
        if (a.y) store8<T, true>(static_cast<T*>(a.y) + row * cols + col, h[k], valid);
      }
      if constexpr (FMT8 != 0) {
        float m = amax8(h[k]);
        if (NORM && a.group) {
          m = lanes_amax(m, min(a.group / 8, LPR ? LPR : 32));
          const float scale = scale_of(m, FMT8);
          store_codes<true>(a.codes + row * cols + col, encode8<FMT8>(h[k], scale), valid);
          if (valid > 0 && (col & (a.group - 1)) == 0)
            a.scales[row * a.groups + (col >> a.shift)] = scale;
        } else {
          top = amax2(top, m);
        }
      }
    }
    if constexpr (FMT8 != 0) {
      if (!NORM || !a.group) {
        if constexpr (LPR != 0) {
          top = lanes_amax(top, LPR);
        } else {
          top = block_amax(top, buf, slot);
          slot ^= 1;
        }
        const float scale = scale_of(top, FMT8);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int col = (R.t + k * R.step) * 8;
          store_codes<true>(a.codes + row * cols + col, encode8<FMT8>(h[k], scale),
                            in && col < cols ? 8 : 0);
        }
        if (R.t == 0 && in) a.scales[row] = scale;
      }
    }
    now = now == S - 1 ? 0 : now + 1;
  }
}

// The end of a backward block: its threads' sums of g_w over the block's rows
// go to the block's row of a.partial.
template <int LPR, int NV, bool VEC>
__device__ __forceinline__ void write_partial(const NormBwd& a, const Rows<LPR>& R,
                                              const float (&acc)[NV][8], float* part) {
  const int cols = (int)a.cols;
  float* out = a.partial + (int64_t)blockIdx.x * cols;
  if constexpr (LPR != 0) {
    // the block's row slots are added in their order
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        part[R.mine * (LPR * NV * 8) + (R.t + k * LPR) * 8 + i] = acc[k][i];
    __syncthreads();
    for (int col = threadIdx.x; col < cols; col += blockDim.x) {
      float s = 0.f;
      for (int r = 0; r < R.here; ++r) s += part[r * (LPR * NV * 8) + col];
      out[col] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      store8<float, VEC>(out + col, acc[k], cols - col);
    }
  }
}

// Registers a thread of the backward may take (the launch counts on them).
constexpr int bwd_regs(int lpr, int nv) { return nv >= 3 ? 128 : nv == 2 ? 96 : lpr ? 64 : 72; }

// The backward of rows whose chunks are whole and aligned: one pass over the
// rows.  A block takes rows gridDim.x apart and keeps its sums of g_w in
// registers; g_y, h (or its codes and scales) and g_h of the next S - 1 rows are
// on their way to shared memory meanwhile, each thread's chunks into places of
// its own.  With v = g_y rstd the formulas need the fewest operations,
//   g_w += v h,  d = sum of (w v) h,  g_x = w v - (rstd^2 d / cols) h + g_h,
// on packed pairs of fp32.
template <typename T, int LPR, int NV, int FMT, int S>
__global__ void __launch_bounds__(LPR ? 256 : 512) __maxnreg__(bwd_regs(LPR, NV))
    norm_bwd_ring_kernel(NormBwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  constexpr int HB = FMT ? 12 : CB;                  // of h's: codes and a scale
  constexpr bool KEEP_W = NV <= 2;                   // the weight stays in registers
  __shared__ float buf[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const int nt = blockDim.x;
  const int64_t stride = (int64_t)gridDim.x * R.here;
  // [stage][k]: nt chunks of g_y, of g_h, of h (FMT: codes, then scales)
  const int k_bytes = nt * (2 * CB + HB), stage_bytes = NV * k_bytes;
  uint8_t* const mine = ring + threadIdx.x * 16;
  bool has[NV];                                      // whether the thread has a chunk k
#pragma unroll
  for (int k = 0; k < NV; ++k) has[k] = (R.t + k * R.step) * 8 < cols;

  auto fetch = [&](uint8_t* stage, int64_t row) {
    if (row < a.rows) {
      const int64_t at = row * cols + R.t * 8;
      const T* gy = static_cast<const T*>(a.g_y) + at;
      const T* gh = static_cast<const T*>(a.g_h) + at;
      const T* h = static_cast<const T*>(a.h) + at;
      const uint8_t* codes = a.codes + at;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!has[k]) continue;
        uint8_t* p = stage + k * k_bytes;
        const int off = k * R.step * 8;
#pragma unroll
        for (int v = 0; v < CB / 16; ++v) {
          constexpr int E = 16 / sizeof(T);
          copy_async<16>(p + v * nt * 16, gy + off + v * E);
          if (a.g_h) copy_async<16>(p + nt * CB + v * nt * 16, gh + off + v * E);
          if constexpr (FMT == 0) copy_async<16>(p + nt * 2 * CB + v * nt * 16, h + off + v * E);
        }
        if constexpr (FMT != 0) {
          copy_async<8>(p + nt * 2 * CB - (int)threadIdx.x * 8, codes + off);
          copy_async<4>(p + nt * (2 * CB + 8) - (int)threadIdx.x * 12,
                        a.scales + row * a.groups + ((R.t * 8 + off) >> a.shift));
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
  auto load_h = [&](const uint8_t* p, uint64_t (&h)[4]) {
    if constexpr (FMT == 0) {
      unpack2(chunk(p + nt * 2 * CB), h);
    } else {
      const uint2 raw =
          *reinterpret_cast<const uint2*>(p + nt * 2 * CB - (int)threadIdx.x * 8);
      const float s =
          *reinterpret_cast<const float*>(p + nt * (2 * CB + 8) - (int)threadIdx.x * 12);
      float f[8];
      decode8<FMT>(Codes{{raw.x, raw.y}}, f);
      const uint64_t ss = f2_pack(s, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = fmul2(f2_pack(f[2 * i], f[2 * i + 1]), ss);
    }
  };
  auto load_w = [&](int k, uint64_t (&w)[4]) {
    float f[8];
    const int col = (R.t + k * R.step) * 8;
    load_weight8<T, true>(a.w, a.w_f32, col, has[k] ? 8 : 0, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_pack(f[2 * i], f[2 * i + 1]);
  };

  const int64_t first = (int64_t)blockIdx.x * R.here;
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(mine + s * stage_bytes, first + s * stride + R.mine);
  uint64_t acc[NV][4], w[KEEP_W ? NV : 1][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = 0;
    if constexpr (KEEP_W) load_w(k, w[k]);
  }
  int slot = 0, now = 0, fill = S - 1;
  float rstd = first + R.mine < a.rows ? a.rstd[first + R.mine] : 0.f;
  for (int64_t row0 = first; row0 < a.rows; row0 += stride) {
    const int64_t row = row0 + R.mine;
    const bool in = LPR == 0 || row < a.rows;
    fetch(mine + fill * stage_bytes, row + (S - 1) * stride);
    const float rstd_next = row + stride < a.rows ? a.rstd[row + stride] : 0.f;
    copy_wait<S - 1>();
    const uint8_t* stage = mine + now * stage_bytes;
    uint64_t wv[NV][4], h[NV][4], dot = 0;
    const uint64_t rr = f2_pack(rstd, rstd);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in || !has[k]) continue;
      const uint8_t* p = stage + k * k_bytes;
      uint64_t g[4];
      unpack2(chunk(p), g);
      load_h(p, h[k]);
      if constexpr (!KEEP_W) load_w(k, w[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t v = fmul2(g[i], rr);
        acc[k][i] = ffma2(v, h[k][i], acc[k][i]);
        wv[k][i] = fmul2(v, w[KEEP_W ? k : 0][i]);
        dot = ffma2(wv[k][i], h[k][i], dot);
      }
    }
    float d0, d1;
    f2_unpack(dot, d0, d1);
    const float d = row_sum<LPR>(d0 + d1, buf, slot);
    const float c = -(d * inv_cols) * (rstd * rstd);
    const uint64_t cc = f2_pack(c, c);
    T* out = static_cast<T*>(a.g_x) + row * cols + R.t * 8;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in || !has[k]) continue;
      uint64_t g[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = ffma2(h[k][i], cc, wv[k][i]);
      if (a.g_h) {
        uint64_t e[4];
        unpack2(chunk(stage + k * k_bytes + nt * CB), e);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = fadd2(g[i], e[i]);
      }
      store8(out + k * R.step * 8, g);
    }
    rstd = rstd_next;
    now = now == S - 1 ? 0 : now + 1;
    fill = fill == S - 1 ? 0 : fill + 1;
  }
  if (a.partial) {
    float sum[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) f2_unpack(acc[k][i], sum[k][2 * i], sum[k][2 * i + 1]);
    write_partial<LPR, NV, true>(a, R, sum, reinterpret_cast<float*>(ring));
  }
}

// The backward of any other rows, straight from global memory.
template <typename T, int LPR, int NV, bool VEC, int FMT>
__global__ void __launch_bounds__(LPR ? 256 : 512) norm_bwd_kernel(NormBwd a) {
  __shared__ float buf[2][32];
  __shared__ float part[LPR ? 256 * 8 * NV : 1];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  float acc[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = 0.f;
  int slot = 0;
  auto load_unit = [&](int64_t row, int col, int valid, float rstd, float (&u)[8]) {
    if constexpr (FMT == 0) {
      const Chunk<T> h = load8<T, VEC>(static_cast<const T*>(a.h) + row * cols + col, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = to_f32(h.e[i]) * rstd;
    } else {
      const Codes c = load_codes<VEC>(a.codes + row * cols + col, valid);
      const float s = valid > 0 ? a.scales[row * a.groups + (col >> a.shift)] : 0.f;
      decode8<FMT>(c, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = u[i] * s * rstd;
    }
  };
  for (int64_t row0 = (int64_t)blockIdx.x * R.here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * R.here) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    const float rstd = in ? a.rstd[row] : 0.f;
    Chunk<T> gy[NV];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int col = (R.t + k * R.step) * 8;
      const int valid = in ? cols - col : 0;
      gy[k] = load8<T, VEC>(static_cast<const T*>(a.g_y) + row * cols + col, valid);
      float w[8], u[8];
      load_unit(row, col, valid, rstd, u);
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
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
      const int col = (R.t + k * R.step) * 8;
      const int valid = in ? cols - col : 0;
      float w[8], u[8], g[8];
      load_unit(row, col, valid, rstd, u);             // from the caches
      load_weight8<T, VEC>(a.w, a.w_f32, col, cols - col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = rstd * (to_f32(gy[k].e[i]) * w[i] - u[i] * c);
      if (a.g_h) {
        const Chunk<T> e = load8<T, VEC>(static_cast<const T*>(a.g_h) + row * cols + col, valid);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += to_f32(e.e[i]);
      }
      store8<T, VEC>(static_cast<T*>(a.g_x) + row * cols + col, g, valid);
    }
  }
  if (a.partial) write_partial<LPR, NV, VEC>(a, R, acc, part);
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

// Lanes a row (0: the block), chunks a thread and threads of a launch over rows
// of `cols` columns.  Up to warp_chunks chunks a warp holds whole rows and needs
// no barrier; beyond, a block of as few threads as hold the row with two chunks
// each, one chunk up to 1024 columns, where blocks are small.
struct Plan {
  int lpr, nv, threads, here;
};
Plan plan(int64_t cols, int max_threads, int warp_chunks) {
  const int chunks = (int)((cols + 7) / 8);
  Plan p;
  if (chunks <= warp_chunks) {
    p.lpr = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    p.nv = (chunks + 31) / 32;
    p.threads = 256;
    p.here = 256 / p.lpr;
  } else {
    p.lpr = 0;
    p.nv = chunks <= 128 ? 1 : chunks <= 2 * max_threads ? 2 : 4;
    p.threads = ((chunks + p.nv - 1) / p.nv + 31) / 32 * 32;
    p.here = 1;
  }
  return p;
}

constexpr int kSMs = 152;
constexpr size_t kMaxSmem = 220 * 1024;

// Blocks that are resident at once: `regs` a thread, `smem` bytes a block.
int resident(int threads, int regs, size_t smem) {
  int n = 65536 / (regs * threads);
  const int by_smem = (int)(kMaxSmem / (smem + 1536));
  if (n > by_smem) n = by_smem;
  if (n > 2048 / threads) n = 2048 / threads;
  if (n < 1) n = 1;
  return kSMs * n;
}
unsigned grid(int64_t rows, int here, int most) {
  const int64_t blocks = (rows + here - 1) / here;
  return (unsigned)(blocks < most ? blocks : most);
}

// Calls f(lanes a row, chunks a thread) as compile-time constants.
template <int N> struct Int { static constexpr int value = N; };
template <typename F>
void with_plan(const Plan& p, F&& f) {
  if (p.lpr == 8) f(Int<8>(), Int<1>());
  else if (p.lpr == 16) f(Int<16>(), Int<1>());
  else if (p.lpr == 32 && p.nv == 1) f(Int<32>(), Int<1>());
  else if (p.lpr == 32 && p.nv == 2) f(Int<32>(), Int<2>());
  else if (p.lpr == 32) f(Int<32>(), Int<3>());
  else if (p.nv == 1) f(Int<0>(), Int<1>());
  else if (p.nv == 2) f(Int<0>(), Int<2>());
  else f(Int<0>(), Int<4>());
}

// Raises a kernel's limit of dynamic shared memory, once a device.
template <auto* KERNEL>
cudaError_t allow_smem() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kMaxSmem);
  if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return e;
}

template <typename T, int FMT8, bool NORM>
cudaError_t fwd(const NormFwd& a, bool vec, cudaStream_t st) {
  const Plan p = plan(a.cols, 1024, 64);
  cudaError_t e = cudaSuccess;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr (N <= 2) {
      const size_t stage = (size_t)N * p.threads * 2 * sizeof(Chunk<T>);
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_fwd_ring_kernel<T, L, N, FMT8, S, NORM>;
        const size_t smem = S * stage;
        e = allow_smem<k>();
        if (e == cudaSuccess)
          k<<<grid(a.rows, p.here, resident(p.threads, 64, smem)), p.threads, smem, st>>>(a);
      };
      if (vec && 3 * stage <= kMaxSmem / 2)
        ring(Int<3>());
      else if (vec && 2 * stage <= kMaxSmem)
        ring(Int<2>());
      else if constexpr (NORM)
        norm_fwd_kernel<T, L, N, false, FMT8>
            <<<grid(a.rows, p.here, kSMs * 32), p.threads, 0, st>>>(a);
      else
        e = cudaErrorNotSupported;
    }
  });
  return e == cudaSuccess ? cudaGetLastError() : e;
}

template <typename T, int FMT>
cudaError_t bwd(const NormBwd& a, bool vec, int* blocks, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 96);
  cudaError_t e = cudaSuccess;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    constexpr int S = L == 0 && N == 4 ? 2 : 3;
    constexpr int CB = (int)sizeof(Chunk<T>);
    size_t smem = (size_t)S * N * p.threads * (2 * CB + (FMT ? 12 : CB));
    const size_t part = L ? (size_t)256 * 8 * N * 4 : 0;
    if (smem < part) smem = part;
    const bool ring = vec && smem <= kMaxSmem;
    *blocks = grid(a.rows, p.here, resident(p.threads, bwd_regs(L, N), ring ? smem : 0));
    if (ring) {
      constexpr auto* k = norm_bwd_ring_kernel<T, L, N, FMT, S>;
      e = allow_smem<k>();
      if (e == cudaSuccess) k<<<*blocks, p.threads, smem, st>>>(a);
    } else {
      norm_bwd_kernel<T, L, N, false, FMT><<<*blocks, p.threads, 0, st>>>(a);
    }
  });
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t cols) {
  const Plan p = plan(cols, 512, 96);
  return (int)grid(rows, p.here, resident(p.threads, bwd_regs(p.lpr, p.nv), 0));
}

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

cudaError_t launch_norm_bwd(int dtype, const NormBwd& in, void* g_w, cudaStream_t st) {
  NormBwd a = in;
  a.shift = group_shift(a.group);
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && aligned_to(a.g_y, 16) && aligned_to(a.h, 16) &&
                     aligned_to(a.g_h, 16) && aligned_to(a.g_x, 16) && aligned_to(a.w, 16) &&
                     aligned_to(a.codes, 8) && aligned_to(a.partial, 16);
    int blocks = 0;
    if (a.rows > 0) {
      const cudaError_t e = !a.codes              ? bwd<T, 0>(a, vec, &blocks, st)
                            : a.fmt == kFmtInt8   ? bwd<T, kFmtInt8>(a, vec, &blocks, st)
                                                  : bwd<T, kFmtE4m3>(a, vec, &blocks, st);
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
