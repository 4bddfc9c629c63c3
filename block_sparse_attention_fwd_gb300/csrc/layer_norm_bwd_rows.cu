// Backward of the layer norm on rows that a block holds, whose chunks are whole and aligned.
#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// As norm_bwd_ring_kernel (norm_bwd.cuh), with fewer registers and instructions, which is
// what bounds the layer norm there: the sums of g_b and the mean take 128 registers, one
// block of 320 threads an SM (32760 x 5120 bf16 with g_h: 241 us; 193 so, 102% of the copy
// rate; from int8 247, 70%).  Pointers walk with the
// rows, FULL (every thread has all of its chunks) needs no predicates, and u is formed
// again from the ring behind the row's sums instead of being kept.
template <typename T, int NV, int FMT, bool GH, bool FULL>
__global__ void __launch_bounds__(512) __maxnreg__(NV == 1 ? 72 : 96)
    layer_norm_bwd_rows_kernel(NormBwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>), HB = FMT ? 8 : CB, S = 3;
  __shared__ float2 buf[2][16];
  extern __shared__ __align__(16) uint8_t ring[];
  const int cols = (int)a.cols, nt = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const float inv_cols = 1.f / (float)cols;
  // a stage: planes of g_y, of g_h, of h (FMT: of codes)
  const int plane = NV * nt * CB, h_plane = (GH ? 2 : 1) * plane, stage = h_plane + NV * nt * HB;
  bool has[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) has[k] = FULL || (t + k * nt) * 8 < cols;
  const int64_t first = blockIdx.x, step = (int64_t)gridDim.x * cols;
  const T* fg = static_cast<const T*>(a.g_y) + first * cols + t * 8;
  const T* fe = static_cast<const T*>(a.g_h) + first * cols + t * 8;
  const T* fh = static_cast<const T*>(a.h) + first * cols + t * 8;
  const uint8_t* fc = a.codes + first * cols + t * 8;
  T* out = static_cast<T*>(a.g_x) + first * cols + t * 8;
  const float* scales = a.scales + first * a.groups;
  auto fetch = [&](int place, bool there) {
    if (there) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (!has[k]) continue;
        uint8_t* p = ring + place + k * nt * CB + t * 16;
#pragma unroll
        for (int v = 0; v < CB / 16; ++v) {
          constexpr int E = 16 / sizeof(T);
          copy_chunk<CB>(p + v * nt * 16, fg + k * nt * 8 + v * E);
          if constexpr (GH) copy_chunk<CB>(p + plane + v * nt * 16, fe + k * nt * 8 + v * E);
          if constexpr (FMT == 0)
            copy_chunk<CB>(p + h_plane + v * nt * 16, fh + k * nt * 8 + v * E);
        }
        if constexpr (FMT != 0)
          copy_async<8>(ring + place + h_plane + k * nt * 8 + t * 8, fc + k * nt * 8);
      }
    }
    fg += step;
    if constexpr (GH) fe += step;
    if constexpr (FMT == 0) fh += step;
    else fc += step;
    copy_commit();
  };
  auto chunk = [&](int at) {
    Chunk<T> c;
#pragma unroll
    for (int v = 0; v < CB / 16; ++v)
      reinterpret_cast<uint4*>(&c)[v] =
          *reinterpret_cast<const uint4*>(ring + at + t * 16 + v * nt * 16);
    return c;
  };
  // (h - mean) rstd
  auto load_u = [&](int place, int k, float scale, float rstd, float mean, uint64_t (&u)[4]) {
    const uint64_t rr = f2_pack(rstd, rstd), mm = f2_pack(-mean, -mean);
    if constexpr (FMT == 0) {
      unpack2(chunk(place + h_plane + k * nt * CB), u);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = fmul2(fadd2(u[i], mm), rr);
    } else {
      const uint2 raw =
          *reinterpret_cast<const uint2*>(ring + place + h_plane + k * nt * 8 + t * 8);
      float f[8];
      decode8<FMT>(Codes{{raw.x, raw.y}}, f);
      const uint64_t ss = f2_pack(scale, scale);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = fmul2(ffma2(f2_pack(f[2 * i], f[2 * i + 1]), ss, mm), rr);
    }
  };
  int64_t left = a.rows - first;                        // rows from this one on
  fetch(0, left > 0);
  fetch(stage, left > gridDim.x);
  uint64_t w[NV][4], acc[NV][4], acc_b[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int col = (t + k * nt) * 8;
    float f[8];
    load_weight8<T, true>(a.w, a.w_f32, col, cols - col, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
      acc[k][i] = acc_b[k][i] = 0;
    }
  }
  const bool part_lane = (lane & 15) < nt / 32;
  int slot = 0, place = 0;
  float rstd = left > 0 ? a.rstd[first] : 0.f, mean = left > 0 ? a.mean[first] : 0.f;
  for (; left > 0; left -= gridDim.x) {
    fetch(place >= stage ? place - stage : place + 2 * stage, left > 2 * (int64_t)gridDim.x);
    // behind the fetch, or the copies would wait for these loads
    const int64_t row = a.rows - left;
    const bool more = left > gridDim.x;
    const float rstd_next = more ? a.rstd[row + gridDim.x] : 0.f;
    const float mean_next = more ? a.mean[row + gridDim.x] : 0.f;
    float scale[NV];
    if constexpr (FMT != 0) {
#pragma unroll
      for (int k = 0; k < NV; ++k) scale[k] = has[k] ? scales[((t + k * nt) * 8) >> a.shift] : 0.f;
      scales += gridDim.x * a.groups;
    }
    copy_wait<S - 1>();
    uint64_t wg[NV][4], dot = 0, all = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has[k]) continue;
      uint64_t g[4], u[4];
      unpack2(chunk(place + k * nt * CB), g);
      load_u(place, k, FMT ? scale[k] : 0.f, rstd, mean, u);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[k][i] = ffma2(g[i], u[i], acc[k][i]);
        acc_b[k][i] = fadd2(g[i], acc_b[k][i]);
        wg[k][i] = fmul2(g[i], w[k][i]);
        dot = ffma2(wg[k][i], u[i], dot);
        all = fadd2(wg[k][i], all);
      }
    }
    float d0, d1, a0, a1;
    f2_unpack(dot, d0, d1);
    f2_unpack(all, a0, a1);
    float c = lanes_sum(d0 + d1, 32), flat = lanes_sum(a0 + a1, 32);
    if (lane == 0) buf[slot][warp] = make_float2(c, flat);
    __syncthreads();
    const float2 v = part_lane ? buf[slot][lane & 15] : make_float2(0.f, 0.f);
    c = lanes_sum(v.x, 16) * -inv_cols;
    flat = lanes_sum(v.y, 16) * -inv_cols;
    slot ^= 1;
    const uint64_t cc = f2_pack(c, c), rr = f2_pack(rstd, rstd), ff = f2_pack(flat, flat);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has[k]) continue;
      uint64_t g[4];
      load_u(place, k, FMT ? scale[k] : 0.f, rstd, mean, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = fadd2(ffma2(g[i], cc, ff), wg[k][i]);
      if constexpr (GH) {
        uint64_t e[4];
        unpack2(chunk(place + plane + k * nt * CB), e);
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = ffma2(g[i], rr, e[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = fmul2(g[i], rr);
      }
      store8(out + k * nt * 8, g);
    }
    out += step;
    rstd = rstd_next;
    mean = mean_next;
    place = place == 2 * stage ? 0 : place + stage;
  }
  if (a.partial) {
    float* p = a.partial + first * cols;
    float* pb = p + (int64_t)gridDim.x * cols;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (!has[k]) continue;
      store8(p + (t + k * nt) * 8, acc[k]);
      store8(pb + (t + k * nt) * 8, acc_b[k]);
    }
  }
}

template <typename T, int FMT>
cudaError_t rows_of(const NormBwd& a, int* blocks, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 96);
  cudaError_t e = cudaErrorNotSupported;
  if (p.lpr || p.nv > 2 || p.threads > 512) return e;
  auto go = [&](auto nv, auto gh, auto full) {
    constexpr int N = decltype(nv)::value;
    constexpr bool GH = decltype(gh)::value != 0;
    constexpr auto* k = layer_norm_bwd_rows_kernel<T, N, FMT, GH, decltype(full)::value != 0>;
    const size_t smem = (size_t)3 * N * p.threads * ((GH ? 2 : 1) * sizeof(Chunk<T>) +
                                                     (FMT ? 8 : sizeof(Chunk<T>)));
    if (smem > kMaxSmem) return;
    e = allow_smem<k>((int)kMaxSmem);
    if (e != cudaSuccess) return;
    *blocks = (int)grid(a.rows, 1, resident(p.threads, N == 1 ? 72 : 96, smem));
    k<<<*blocks, p.threads, smem, st>>>(a);
    e = cudaGetLastError();
  };
  auto of = [&](auto nv, auto gh) {
    a.cols == (int64_t)8 * p.nv * p.threads ? go(nv, gh, Int<1>()) : go(nv, gh, Int<0>());
  };
  if (a.g_h)
    p.nv == 1 ? of(Int<1>(), Int<1>()) : of(Int<2>(), Int<1>());
  else
    p.nv == 1 ? of(Int<1>(), Int<0>()) : of(Int<2>(), Int<0>());
  return e;
}

}  // namespace

namespace norm {

cudaError_t layer_bwd_rows(int dtype, const NormBwd& a, int* blocks, cudaStream_t st) {
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return !a.codes            ? rows_of<T, 0>(a, blocks, st)
           : a.fmt == kFmtInt8 ? rows_of<T, kFmtInt8>(a, blocks, st)
                               : rows_of<T, kFmtE4m3>(a, blocks, st);
  });
}

}  // namespace norm

}  // namespace bl
