// Kernels of the root-mean-square norm's backward (norm.cuh).
#pragma once

#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// The end of a backward block: its threads' sums of g_w over the block's rows
// go to the block's row of a.partial.
template <int LPR, int NV, bool VEC, bool SPREAD = false>
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
        part[R.mine * (LPR * NV * 8) + col_of<SPREAD>(R, k, i)] = acc[k][i];
    __syncthreads();
    for (int col = threadIdx.x; col < cols; col += blockDim.x) {
      float s = 0.f;
      for (int r = 0; r < R.here; ++r) s += part[r * (LPR * NV * 8) + col];
      out[col] = s;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) store_unit<float, VEC, SPREAD>(out, R, k, cols, acc[k]);
  }
}

// Registers a thread of the backward may take (the launch counts on them).
// SPREAD, with an address an element, takes more.
constexpr int bwd_regs(int lpr, int nv, bool spread = false) {
  return nv >= 3  ? 128
         : spread ? (nv == 1 ? 104 : 128)
         : nv == 2 ? 96
         : lpr     ? 64
                   : 72;
}

// The backward of rows whose chunks are whole and aligned: one pass over the
// rows.  A block takes rows gridDim.x apart and keeps its sums of g_w in
// registers; g_y, h (or its codes and scales) and g_h of the next S - 1 rows are
// on their way to shared memory meanwhile, each thread's chunks into places of
// its own.  With u = h rstd (of 8 bits: the codes by the product of scale and
// rstd),
//   g_w += g_y u,  c = mean of (w g_y) u,  g_x = rstd (w g_y - c u) + g_h,
// on packed pairs of fp32.  No product on the way is much larger or smaller than
// a result, so rows and gradients of any size stay within fp32's range; rstd^2
// does not (rows below 5e-20).  Bound by HBM: 32760 x 5120 bf16 with g_h in 192
// us (7.0 TB/s), h from int8 in 180 us (6.6 TB/s).  The same pass with loads into
// registers took 354 and 719 us; with the ring but scalar arithmetic, 245
// instructions a chunk, 240 and 255 us.  The weight that does not stay in
// registers is loaded in front of the row's chunks (fp32, 75000 x 640: 129 us, 140
// behind them).
// ODD: rows of a 16-bit type that start anywhere, as in the forward (2561 columns:
// 24% of the copy rate element by element, 51% so), or of fp32, SPREAD.
template <typename T, int LPR, int NV, int FMT, int S, bool ODD>
__global__ void __launch_bounds__(LPR ? 256 : 512) __maxnreg__(bwd_regs(LPR, NV, ODD && sizeof(T) == 4))
    norm_bwd_ring_kernel(NormBwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  constexpr int HB = FMT ? 12 : CB;                  // of h's: codes and a scale
  constexpr bool KEEP_W = NV <= 2;                   // the weight stays in registers
  constexpr bool SHIFT = ODD && CB == 16, SPREAD = ODD && CB != 16;
  static_assert(!SPREAD || FMT == 0);
  __shared__ float buf[2][32];
  extern __shared__ __align__(16) uint8_t ring[];
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  const int nt = blockDim.x;
  const int64_t stride = (int64_t)gridDim.x * R.here;
  // a stage: planes of NV * nt chunks of g_y, of g_h, of h (FMT: of codes, then of
  // scales)
  const int plane = NV * nt * CB, stage_bytes = 2 * plane + NV * nt * HB;
  bool has[NV];                                      // whether the thread has a chunk k
#pragma unroll
  for (int k = 0; k < NV; ++k) has[k] = col_of<SPREAD>(R, k, 0) < cols;

  // `place`: the thread's first 16 bytes of a stage; its codes and scales lie
  // 8 and 12 bytes a thread less far
  auto codes_at = [&](auto* place, int k) {
    return place + 2 * plane + k * nt * 8 - (int)threadIdx.x * 8;
  };
  auto scale_at = [&](auto* place, int k) {
    return place + 2 * plane + NV * nt * 8 + k * nt * 4 - (int)threadIdx.x * 12;
  };
  auto fetch = [&](uint8_t* place, int64_t row) {
    if (row < a.rows) {
      const int64_t at = row * cols + (ODD ? 0 : R.t * 8);
      const T* gy = static_cast<const T*>(a.g_y) + at;
      const T* gh = static_cast<const T*>(a.g_h) + at;
      const T* h = static_cast<const T*>(a.h) + at;
      const uint8_t* codes = a.codes + at;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint8_t* p = place + k * nt * CB;
        if constexpr (SPREAD) {
          uint8_t* all = place - threadIdx.x * 16;
          copy_spread(all, gy, R, k, nt, cols);
          if (a.g_h) copy_spread(all + plane, gh, R, k, nt, cols);
          copy_spread(all + 2 * plane, h, R, k, nt, cols);
        } else if constexpr (SHIFT) {
          const int c = R.t + k * R.step;
          if (c * 8 >= cols + 8) continue;
          copy_odd(p, gy, c, cols);
          if (a.g_h) copy_odd(p + plane, gh, c, cols);
          if constexpr (FMT == 0)
            copy_odd(p + 2 * plane, h, c, cols);
          else
            copy_odd8(codes_at(place, k), codes, c, cols);
        } else {
          if (!has[k]) continue;
          const int off = k * R.step * 8;
#pragma unroll
          for (int v = 0; v < CB / 16; ++v) {
            constexpr int E = 16 / sizeof(T);
            copy_chunk<CB>(p + v * nt * 16, gy + off + v * E);
            if (a.g_h) copy_chunk<CB>(p + plane + v * nt * 16, gh + off + v * E);
            if constexpr (FMT == 0) copy_chunk<CB>(p + 2 * plane + v * nt * 16, h + off + v * E);
          }
          if constexpr (FMT != 0) copy_async<8>(codes_at(place, k), codes + off);
        }
        if constexpr (FMT != 0)
          if (has[k])
            copy_async<4>(scale_at(place, k),
                          a.scales + row * a.groups + (((R.t + k * R.step) * 8) >> a.shift));
      }
    }
    copy_commit();
  };
  // chunk k out of the thread's place in a plane, of a row of this tensor
  auto chunk = [&](const uint8_t* place, int k, const void* tensor, int64_t row) {
    const uint8_t* p = place + k * nt * CB;
    Chunk<T> c;
    if constexpr (SPREAD) {
      c = chunk_spread(place - threadIdx.x * 16, k, nt);
    } else if constexpr (SHIFT) {
      c = chunk_odd<T, LPR>(p, R.t, nt, static_cast<const T*>(tensor) + row * cols);
    } else {
#pragma unroll
      for (int v = 0; v < CB / 16; ++v)
        reinterpret_cast<uint4*>(&c)[v] = *reinterpret_cast<const uint4*>(p + v * nt * 16);
    }
    return c;
  };
  auto load_u = [&](const uint8_t* place, int k, int64_t row, float rstd, uint64_t (&u)[4]) {
    if constexpr (FMT == 0) {
      const uint64_t rr = f2_pack(rstd, rstd);
      unpack2(chunk(place + 2 * plane, k, a.h, row), u);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = fmul2(u[i], rr);
    } else {
      const float s = *reinterpret_cast<const float*>(scale_at(place, k)) * rstd;
      Codes codes;
      if constexpr (SHIFT) {
        codes = codes_odd<LPR>(codes_at(place, k), R.t, nt, a.codes + row * cols);
      } else {
        const uint2 raw = *reinterpret_cast<const uint2*>(codes_at(place, k));
        codes = Codes{{raw.x, raw.y}};
      }
      float f[8];
      decode8<FMT>(codes, f);
      const uint64_t ss = f2_pack(s, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = fmul2(f2_pack(f[2 * i], f[2 * i + 1]), ss);
    }
  };
  auto load_w = [&](int k, uint64_t (&w)[4]) {
    float f[8];
    weight_unit<T, !ODD, SPREAD>(a.w, a.w_f32, R, k, cols, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f2_pack(f[2 * i], f[2 * i + 1]);
  };

  uint8_t* const mine = ring + threadIdx.x * 16;
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
    if constexpr (SHIFT) {
      copy_wait<S - 2>();
      if constexpr (LPR) __syncwarp(); else __syncthreads();
    }
    fetch(mine + fill * stage_bytes, row + (S - 1) * stride);
    // behind the fetch: in front of it the copies waited for this load (153 -> 171 us)
    const float rstd_next = row + stride < a.rows ? a.rstd[row + stride] : 0.f;
    if constexpr (!SHIFT) copy_wait<S - 1>();
    const uint8_t* place = mine + now * stage_bytes;
    uint64_t wg[NV][4], u[NV][4], dot = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in || !has[k]) continue;
      if constexpr (!KEEP_W) load_w(k, w[0]);
      uint64_t g[4];
      unpack2(chunk(place, k, a.g_y, row), g);
      load_u(place, k, row, rstd, u[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[k][i] = ffma2(g[i], u[k][i], acc[k][i]);
        wg[k][i] = fmul2(g[i], w[KEEP_W ? k : 0][i]);
        dot = ffma2(wg[k][i], u[k][i], dot);
      }
    }
    float d0, d1;
    f2_unpack(dot, d0, d1);
    const float c = -(row_sum<LPR>(d0 + d1, buf, slot) * inv_cols);
    const uint64_t cc = f2_pack(c, c), rr = f2_pack(rstd, rstd);
    T* out = static_cast<T*>(a.g_x) + row * cols + (ODD ? 0 : R.t * 8);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      uint32_t words[4] = {0, 0, 0, 0};
      if (in && has[k]) {
        uint64_t g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = ffma2(u[k][i], cc, wg[k][i]);
        if (a.g_h) {
          uint64_t e[4];
          unpack2(chunk(place + plane, k, a.g_h, row), e);
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = ffma2(g[i], rr, e[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) g[i] = fmul2(g[i], rr);
        }
        if constexpr (SPREAD) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(g[i], f[2 * i], f[2 * i + 1]);
          store_unit<T, false, true>(out, R, k, cols, f);
        } else if constexpr (SHIFT) {
          pack_words<T>(g, words);
        } else {
          store8(out + k * R.step * 8, g);
        }
      }
      if constexpr (SHIFT) {
        const int c = R.t + k * R.step;
        store_anywhere<4>(reinterpret_cast<uint8_t*>(out), c,
                          in && has[k] ? min(cols - c * 8, 8) : 0, cols, lane_in_front(R),
                          lane_behind(R), words);
      }
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
    write_partial<LPR, NV, !ODD, SPREAD>(a, R, sum, reinterpret_cast<float*>(ring));
  }
}

// Launches the ring kernel on rows that it takes, else cudaErrorNotSupported.
// *blocks: its blocks, which are the rows of partial sums.
template <typename T, int FMT, bool ODD>
cudaError_t bwd_ring(const NormBwd& a, int* blocks, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 96, ODD && sizeof(T) == 2);
  cudaError_t e = cudaErrorNotSupported;
  if (p.threads > 512) return e;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    constexpr int CB = (int)sizeof(Chunk<T>);
    // fp32 that a warp holds: 4-byte copies cost more than the ring gains (129
    // columns: 72% of the copy rate straight from global memory, 29% so)
    if constexpr (!(ODD && CB != 16 && L != 0)) {
      const size_t stage = (size_t)N * p.threads * (2 * CB + (FMT ? 12 : CB));
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_bwd_ring_kernel<T, L, N, FMT, S, ODD>;
        size_t smem = S * stage;
        if constexpr (L != 0) {                          // the block's sums of g_w go there too
          if (smem < (size_t)256 * 8 * N * 4) smem = (size_t)256 * 8 * N * 4;
        }
        *blocks = (int)grid(a.rows, p.here, resident(p.threads, bwd_regs(L, N, ODD && CB != 16), smem));
        e = allow_smem<k>();
        if (e != cudaSuccess) return;
        k<<<*blocks, p.threads, smem, st>>>(a);
        e = cudaGetLastError();
      };
      constexpr int MOST = N == 4 ? 2 : 3;               // stages
      if (MOST * stage <= kMaxSmem) {
        ring(Int<MOST>());
        return;
      }
      if constexpr (L == 0 && N == 2)
        if (2 * stage <= kMaxSmem) ring(Int<2>());
    }
  });
  return e;
}

}  // namespace

}  // namespace bl
