// Kernels of the norms' backward (norm.cuh).
#pragma once

#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// The end of a backward block: its threads' sums of g_w (g_b) over the block's rows
// go to the block's row of `partial`.
template <int LPR, int NV, bool VEC, bool SPREAD = false>
__device__ __forceinline__ void write_partial(const NormBwd& a, float* partial, const Rows<LPR>& R,
                                              const float (&acc)[NV][8], float* part) {
  const int cols = (int)a.cols;
  float* out = partial + (int64_t)blockIdx.x * cols;
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
// SPREAD, with an address an element, takes more, and so does the layer norm, with
// the sums of g_b (262144 x 128 bf16: 59 us with 88, two blocks an SM, 46 with 64).
constexpr int bwd_regs(int lpr, int nv, bool spread = false, bool layer = false) {
  return layer    ? (nv >= 2 || spread ? 128 : lpr ? 64 : 88)
         : nv >= 3  ? 128
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
// LN: the layer norm's, u = (h - mean) rstd and g_x = rstd (w g_y - mean of w g_y - c u)
// + g_h, with g_b beside g_w.  With three chunks a thread and more, u and w g_y do not
// stay in registers over the row's sum but are formed again from the ring (RELOAD).
template <typename T, int LPR, int NV, int FMT, int S, bool ODD, bool LN>
__global__ void __launch_bounds__(LPR ? 256 : 512)
    __maxnreg__(bwd_regs(LPR, NV, ODD && sizeof(T) == 4, LN))
    norm_bwd_ring_kernel(NormBwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>);          // bytes of a chunk
  constexpr int HB = FMT ? 12 : CB;                  // of h's: codes and a scale
  constexpr bool KEEP_W = NV <= 2;                   // the weight stays in registers
  constexpr bool SHIFT = ODD && CB == 16, SPREAD = ODD && CB != 16;
  constexpr bool RELOAD = LN && (NV >= 3 || (SPREAD && NV == 2));
  static_assert(!SPREAD || FMT == 0);
  __shared__ float buf[2][LN ? 64 : 32];
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
  auto load_u = [&](const uint8_t* place, int k, int64_t row, float mean, float rstd,
                    uint64_t (&u)[4]) {
    const uint64_t rr = f2_pack(rstd, rstd), mm = f2_pack(-mean, -mean);
    if constexpr (FMT == 0) {
      unpack2(chunk(place + 2 * plane, k, a.h, row), u);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = fmul2(LN ? fadd2(u[i], mm) : u[i], rr);
    } else {
      const float s = *reinterpret_cast<const float*>(scale_at(place, k)) * (LN ? 1.f : rstd);
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
      for (int i = 0; i < 4; ++i) {
        u[i] = f2_pack(f[2 * i], f[2 * i + 1]);
        u[i] = LN ? fmul2(ffma2(u[i], ss, mm), rr) : fmul2(u[i], ss);
      }
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
  uint64_t acc[NV][4], acc_b[LN ? NV : 1][4], w[KEEP_W ? NV : 1][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[k][i] = acc_b[LN ? k : 0][i] = 0;
    if constexpr (KEEP_W) load_w(k, w[k]);
  }
  int slot = 0, now = 0, fill = S - 1;
  float rstd = first + R.mine < a.rows ? a.rstd[first + R.mine] : 0.f;
  float mean = LN && first + R.mine < a.rows ? a.mean[first + R.mine] : 0.f;
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
    const float mean_next = LN && row + stride < a.rows ? a.mean[row + stride] : 0.f;
    if constexpr (!SHIFT) copy_wait<S - 1>();
    const uint8_t* place = mine + now * stage_bytes;
    uint64_t wg[RELOAD ? 1 : NV][4], u[RELOAD ? 1 : NV][4], dot = 0, all = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!in || !has[k]) continue;
      constexpr auto at = [](int k) { return RELOAD ? 0 : k; };
      if constexpr (!KEEP_W) load_w(k, w[0]);
      uint64_t g[4];
      unpack2(chunk(place, k, a.g_y, row), g);
      load_u(place, k, row, mean, rstd, u[at(k)]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[k][i] = ffma2(g[i], u[at(k)][i], acc[k][i]);
        if constexpr (LN) acc_b[k][i] = fadd2(g[i], acc_b[k][i]);
        wg[at(k)][i] = fmul2(g[i], w[KEEP_W ? k : 0][i]);
        dot = ffma2(wg[at(k)][i], u[at(k)][i], dot);
        if constexpr (LN) all = fadd2(wg[at(k)][i], all);
      }
    }
    float d0, d1;
    f2_unpack(dot, d0, d1);
    float c, flat = 0.f;
    if constexpr (LN) {
      float a0, a1;
      f2_unpack(all, a0, a1);
      const float2 sums = row_sum2<LPR>(make_float2(d0 + d1, a0 + a1), buf, slot);
      c = -(sums.x * inv_cols);
      flat = -(sums.y * inv_cols);
    } else {
      c = -(row_sum<LPR>(d0 + d1, buf, slot) * inv_cols);
    }
    const uint64_t cc = f2_pack(c, c), rr = f2_pack(rstd, rstd), ff = f2_pack(flat, flat);
    T* out = static_cast<T*>(a.g_x) + row * cols + (ODD ? 0 : R.t * 8);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      uint32_t words[4] = {0, 0, 0, 0};
      if (in && has[k]) {
        uint64_t g[4];
        if constexpr (RELOAD) {
          if constexpr (!KEEP_W) load_w(k, w[0]);
          unpack2(chunk(place, k, a.g_y, row), g);
          load_u(place, k, row, mean, rstd, u[0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) wg[0][i] = fmul2(g[i], w[KEEP_W ? k : 0][i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = ffma2(u[RELOAD ? 0 : k][i], cc, wg[RELOAD ? 0 : k][i]);
          if constexpr (LN) g[i] = fadd2(g[i], ff);
        }
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
    mean = mean_next;
    now = now == S - 1 ? 0 : now + 1;
    fill = fill == S - 1 ? 0 : fill + 1;
  }
  if (a.partial) {
    float sum[NV][8];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) f2_unpack(acc[k][i], sum[k][2 * i], sum[k][2 * i + 1]);
    write_partial<LPR, NV, !ODD, SPREAD>(a, a.partial, R, sum, reinterpret_cast<float*>(ring));
    if constexpr (LN) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) f2_unpack(acc_b[k][i], sum[k][2 * i], sum[k][2 * i + 1]);
      write_partial<LPR, NV, !ODD, SPREAD>(a, a.partial + (int64_t)gridDim.x * cols, R, sum,
                                           reinterpret_cast<float*>(ring));
    }
  }
}

// Launches the ring kernel on rows that it takes, else cudaErrorNotSupported.
// *blocks: its blocks, which are the rows of partial sums.
template <typename T, int FMT, bool ODD, bool LN>
cudaError_t bwd_ring(const NormBwd& a, int* blocks, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 96, ODD && sizeof(T) == 2);
  cudaError_t e = cudaErrorNotSupported;
  if (p.threads > 512) return e;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    constexpr int CB = (int)sizeof(Chunk<T>);
    // fp32 that a warp holds: 4-byte copies cost more than the ring gains (129
    // columns: 72% of the copy rate straight from global memory, 29% so)
    constexpr size_t UNIT = (size_t)N * (2 * CB + (FMT ? 12 : CB));    // a thread's of a stage
    // layer_bwd_rows takes aligned rows of up to two chunks a thread wherever three stages fit
    constexpr bool REST = LN && !ODD && L == 0 && N <= 2;
    if constexpr (!(ODD && CB != 16 && L != 0) && !(REST && (N == 1 || CB == 16 || FMT != 0))) {
      const size_t stage = p.threads * UNIT;
      auto ring = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        constexpr auto* k = norm_bwd_ring_kernel<T, L, N, FMT, S, ODD, LN>;
        size_t smem = S * stage;
        if constexpr (L != 0) {                          // the block's sums of g_w go there too
          if (smem < (size_t)256 * 8 * N * 4) smem = (size_t)256 * 8 * N * 4;
        }
        *blocks = (int)grid(a.rows, p.here,
                            resident(p.threads, bwd_regs(L, N, ODD && CB != 16, LN), smem));
        e = allow_smem<k>((int)kMaxSmem);
        if (e != cudaSuccess) return;
        k<<<*blocks, p.threads, smem, st>>>(a);
        e = cudaGetLastError();
      };
      constexpr int MOST = N == 4 ? 2 : 3;               // stages
      if constexpr (!REST)
        if (MOST * stage <= kMaxSmem) {
          ring(Int<MOST>());
          return;
        }
      if constexpr (L == 0 && N == 2 && MOST * UNIT * 512 > kMaxSmem)
        if (2 * stage <= kMaxSmem) ring(Int<2>());
    }
  });
  return e;
}

// The backward of rows that the ring does not take, straight from global memory: fp32
// that starts anywhere and is held by a warp or comes in 8 bits (IN8) or is too wide,
// and 16-bit rows that start anywhere of more than 16376 columns.
template <typename T, int LPR, int NV, bool VEC, bool IN8, bool LN>
__global__ void __launch_bounds__(LPR ? 256 : 512) norm_bwd_kernel(NormBwd a) {
  __shared__ float buf[2][LN ? 64 : 32];
  __shared__ float part[LPR ? 256 * 8 * NV : 1];
  constexpr bool SPREAD = !VEC && !IN8;
  const Rows<LPR> R;
  const int cols = (int)a.cols;
  const float inv_cols = 1.f / (float)cols;
  float acc[NV][8], acc_b[LN ? NV : 1][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[k][i] = acc_b[LN ? k : 0][i] = 0.f;
  int slot = 0;
  auto unit_of = [&](int64_t row, int k, int here, float mean, float rstd, float (&u)[8]) {
    if constexpr (!IN8) {
      const Chunk<T> h =
          load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.h) + row * cols, R, k, here);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (LN ? to_f32(h.e[i]) - mean : to_f32(h.e[i])) * rstd;
    } else {
      const int col = (R.t + k * R.step) * 8, valid = here - col;
      const Codes c = load_codes<VEC>(a.codes + row * cols + col, valid);
      const float s = valid > 0 ? a.scales[row * a.groups + (col >> a.shift)] : 0.f;
      decode8(a.fmt, c, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (LN ? fmaf(u[i], s, -mean) : u[i] * s) * rstd;
    }
  };
  for (int64_t row0 = (int64_t)blockIdx.x * R.here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * R.here) {
    const int64_t row = row0 + R.mine;
    const bool in = row < a.rows;
    const int here = in ? cols : 0;
    const float rstd = in ? a.rstd[row] : 0.f;
    const float mean = LN && in ? a.mean[row] : 0.f;
    Chunk<T> gy[NV];
    float dot = 0.f, all = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      gy[k] = load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.g_y) + row * cols, R, k, here);
      float w[8], u[8];
      unit_of(row, k, here, mean, rstd, u);
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float g = to_f32(gy[k].e[i]);
        acc[k][i] = fmaf(g, u[i], acc[k][i]);
        dot = fmaf(g * w[i], u[i], dot);
        if constexpr (LN) {
          acc_b[k][i] += g;
          all = fmaf(g, w[i], all);
        }
      }
    }
    float c, flat = 0.f;
    if constexpr (LN) {
      const float2 sums = row_sum2<LPR>(make_float2(dot, all), buf, slot);
      c = sums.x * inv_cols;
      flat = sums.y * inv_cols;
    } else {
      c = row_sum<LPR>(dot, buf, slot) * inv_cols;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float w[8], u[8], g[8];
      unit_of(row, k, here, mean, rstd, u);                  // from the caches
      weight_unit<T, VEC, SPREAD>(a.w, a.w_f32, R, k, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        g[i] = to_f32(gy[k].e[i]) * w[i] - u[i] * c;
        g[i] = rstd * (LN ? g[i] - flat : g[i]);
      }
      if (a.g_h) {
        const Chunk<T> e =
            load_unit<T, VEC, SPREAD>(static_cast<const T*>(a.g_h) + row * cols, R, k, here);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += to_f32(e.e[i]);
      }
      store_unit<T, VEC, SPREAD>(static_cast<T*>(a.g_x) + row * cols, R, k, here, g);
    }
  }
  if (a.partial) {
    write_partial<LPR, NV, VEC, SPREAD>(a, a.partial, R, acc, part);
    if constexpr (LN)
      write_partial<LPR, NV, VEC, SPREAD>(a, a.partial + (int64_t)gridDim.x * cols, R, acc_b, part);
  }
}

// g_w[col] (of the second row of blocks, g_b) = sum of the blocks' partial sums, 32 columns a block, 32 slices of
// the partial rows side by side and then added in their order: no atomics, so
// the result does not vary.  4 us at 4096 columns, most of it the launch.
template <typename T>
__global__ void __launch_bounds__(1024) norm_gw_kernel(const float* __restrict__ partial, int parts,
                                                       int cols, void* g_w, void* g_b, bool f32) {
  __shared__ float s[32][33];
  if (blockIdx.y) {
    partial += (int64_t)parts * cols;
    g_w = g_b;
  }
  if (!g_w) return;
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

template <typename T, int FMT, bool LN>
cudaError_t bwd(int dtype, const NormBwd& a, bool vec, int* blocks, cudaStream_t st) {
  cudaError_t e = cudaErrorNotSupported;
  if constexpr (LN)
    if (vec) e = layer_bwd_rows(dtype, a, blocks, st);
  if (e != cudaErrorNotSupported) return e;
  e = vec  ? bwd_ring<T, FMT, false, LN>(a, blocks, st)
      : LN ? layer_bwd_odd(dtype, a, blocks, st)
           : bwd_odd(dtype, a, blocks, st);
  if (e != cudaErrorNotSupported) return e;
  const Plan p = plan(a.cols, 512, 96);
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    if constexpr ((L == 0 && N == 4) || (sizeof(T) == 4 && (FMT != 0 || L != 0))) {
      constexpr bool WIDE = sizeof(T) == 4 && L == 0 && N == 4;     // too wide for the ring
      *blocks = (int)grid(a.rows, p.here, resident(p.threads, bwd_regs(L, N, false, LN), 0));
      if (vec && WIDE)
        norm_bwd_kernel<T, L, N, WIDE, FMT != 0, LN><<<*blocks, p.threads, 0, st>>>(a);
      else
        norm_bwd_kernel<T, L, N, false, FMT != 0, LN><<<*blocks, p.threads, 0, st>>>(a);
      e = cudaGetLastError();
    }
  });
  return e;
}

// Rows of partial sums that the backward writes at most.
template <bool LN>
int bwd_parts_of(int64_t rows, int64_t cols) {
  // of either way to lay out the rows
  int most = 0;
  if (LN) {                                              // layer_bwd_rows
    const Plan p = plan(cols, 512, 96);
    if (!p.lpr) most = (int)grid(rows, 1, resident(p.threads, p.nv == 1 ? 72 : 96, 0));
  }
  for (bool odd : {false, true}) {
    const Plan p = plan(cols, 512, 96, odd);
    const int blocks =
        (int)grid(rows, p.here, resident(p.threads, bwd_regs(p.lpr, p.nv, false, LN), 0));
    if (blocks > most) most = blocks;
  }
  return most;
}

// The backward's launch on rows of any kind.
template <bool LN>
cudaError_t launch_bwd_of(int dtype, const NormBwd& in, void* g_w, void* g_b, cudaStream_t st) {
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
      const cudaError_t e = !a.codes              ? bwd<T, 0, LN>(dtype, a, vec, &blocks, st)
                            : a.fmt == kFmtInt8   ? bwd<T, kFmtInt8, LN>(dtype, a, vec, &blocks, st)
                                                  : bwd<T, kFmtE4m3, LN>(dtype, a, vec, &blocks, st);
      if (e != cudaSuccess) return e;
    }
    if (g_w || g_b) {
      norm_gw_kernel<T><<<dim3((unsigned)((a.cols + 31) / 32), g_b ? 2 : 1), 1024, 0, st>>>(
          a.partial, blocks, (int)a.cols, g_w, g_b, a.w_f32);
      return cudaGetLastError();
    }
    return cudaSuccess;
  });
}

}  // namespace

}  // namespace bl
