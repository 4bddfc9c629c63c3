// Backward of the root-mean-square norm (norm.cuh).
#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

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
// on packed pairs of fp32.  Bound by HBM: 32760 x 5120 bf16 with g_h in 192 us
// (7.0 TB/s), h from int8 in 179 us (6.6 TB/s).  The same pass with loads into
// registers took 354 and 719 us; with the ring but scalar arithmetic on u = h
// rstd, 245 instructions a chunk, 240 and 255 us.
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

// The backward of any other rows, straight from global memory.  IN8: h comes in
// 8 bits.
template <typename T, int LPR, int NV, bool VEC, bool IN8>
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
    if constexpr (!IN8) {
      const Chunk<T> h = load8<T, VEC>(static_cast<const T*>(a.h) + row * cols + col, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = to_f32(h.e[i]) * rstd;
    } else {
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
cudaError_t bwd(const NormBwd& a, bool vec, int* blocks, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 96);
  cudaError_t e = cudaSuccess;
  with_plan(p, [&](auto lpr, auto nv) {
    constexpr int L = decltype(lpr)::value, N = decltype(nv)::value;
    constexpr bool WIDE = sizeof(T) == 4 && L == 0 && N == 4;     // too wide for the ring
    constexpr int CB = (int)sizeof(Chunk<T>);
    const size_t stage = (size_t)N * p.threads * (2 * CB + (FMT ? 12 : CB));
    auto blocks_of = [&](size_t smem) {
      return (int)grid(a.rows, p.here, resident(p.threads, bwd_regs(L, N), smem));
    };
    auto ring = [&](auto stages) {
      constexpr int S = decltype(stages)::value;
      constexpr auto* k = norm_bwd_ring_kernel<T, L, N, FMT, S>;
      size_t smem = S * stage;
      if constexpr (L != 0) {                          // the block's sums of g_w go there too
        if (smem < (size_t)256 * 8 * N * 4) smem = (size_t)256 * 8 * N * 4;
      }
      *blocks = blocks_of(smem);
      e = allow_smem<k>();
      if (e == cudaSuccess) k<<<*blocks, p.threads, smem, st>>>(a);
    };
    constexpr int MOST = N == 4 ? 2 : 3;               // stages
    if (vec && MOST * stage <= kMaxSmem) {
      ring(Int<MOST>());
      return;
    }
    if constexpr (L == 0 && N == 2)
      if (vec && 2 * stage <= kMaxSmem) {
        ring(Int<2>());
        return;
      }
    *blocks = blocks_of(0);
    if (vec && WIDE)
      norm_bwd_kernel<T, L, N, WIDE, FMT != 0><<<*blocks, p.threads, 0, st>>>(a);
    else
      norm_bwd_kernel<T, L, N, false, FMT != 0><<<*blocks, p.threads, 0, st>>>(a);
  });
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

int norm_bwd_parts(int64_t rows, int64_t cols) {
  const Plan p = plan(cols, 512, 96);
  return (int)grid(rows, p.here, resident(p.threads, bwd_regs(p.lpr, p.nv), 0));
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
