// Forward of the layer norm on rows that a block holds, two at a time.
#include "norm.cuh"

namespace bl {

using namespace norm;

namespace {

// Registers a thread: two blocks of 320 threads an SM.  A few spilled ones cost more than a
// block less (32760 x 5120 to e4m3: 212 us with 8 bytes spilled at 80, 181 us at 96), so the
// 8-bit output, whose codes take their own, has one row at a time where a thread has two
// chunks of it.
constexpr int pair_regs(int nv) { return nv == 1 ? 64 : 96; }

// The layer norm of rows that a block holds, whose chunks are whole and aligned: two rows
// at a time.  One row's sums are a chain of shuffles and a barrier that the few blocks that
// fit beside weight and bias in registers do not hide (32760 x 5120 bf16: 143 us a row at a
// time, 102 so, 97% of the copy rate; with the residual 197, 100%; to e4m3 182, 95%).  A
// row's mean and squares come from one round of shuffles: each warp sums
// distances from the mean of its first lane's elements, and the squares around its own mean
// follow by sum d^2 - (sum d)^2 / n.  With a pivot p that is the mean of k of the n elements,
// whose mean is m, (sum d)^2 / n = n (p - m)^2, and what is left, at least k n / (n - k)
// (p - m)^2, is at most n / k - 1 = 31 times smaller (the k of one value, the others of
// another).  The warps' means are put together likewise, around the first warp's, which holds
// as many elements as any other of 16: at most 15 times.  So the squares, summed to within
// 64 2^-24 of themselves, give the variance within 64 (32 + 16) 2^-24 at worst, 2e-4.
// FULL: every thread has all of its chunks.
template <typename T, int NV, int RB, int FMT8, bool RES, bool FULL>
__global__ void __launch_bounds__(512) __maxnreg__(pair_regs(NV))
    layer_norm_pair_kernel(LayerNormFwd a) {
  constexpr int CB = (int)sizeof(Chunk<T>), TENSORS = RES ? 2 : 1;
  __shared__ float2 buf[2][RB][16];
  extern __shared__ __align__(16) uint8_t ring[];
  const int cols = (int)a.cols, nt = blockDim.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const float inv_cols = 1.f / (float)cols;
  const int plane = NV * nt * CB, stage = RB * TENSORS * plane;
  bool has[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) has[k] = FULL || (t + k * nt) * 8 < cols;
  // pointers that walk with the pairs, to the thread's first chunk
  const int64_t first_row = (int64_t)blockIdx.x * RB, step = (int64_t)gridDim.x * RB;
  const T* fx = static_cast<const T*>(a.x) + first_row * a.x_stride + t * 8;
  const T* fr = static_cast<const T*>(a.r) + first_row * a.r_stride + t * 8;
  const int64_t step_x = step * a.x_stride, step_r = step * a.r_stride, step_y = step * cols;
  T* py = static_cast<T*>(a.y) + first_row * cols + t * 8;
  T* ph = static_cast<T*>(a.h) + first_row * cols + t * 8;
  uint8_t* pc = a.codes + first_row * cols + t * 8;
  auto fetch = [&](int place, int64_t rows_left) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      if (rows_left <= 0) break;
      // the row behind the last is the last once more
      const T* x = fx + (rb && rows_left > 1 ? a.x_stride : 0);
      const T* r = fr + (rb && rows_left > 1 ? a.r_stride : 0);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint8_t* p = ring + place + rb * TENSORS * plane + k * nt * CB + t * 16;
        if (!has[k]) continue;
#pragma unroll
        for (int v = 0; v < CB / 16; ++v) {
          constexpr int E = 16 / sizeof(T);
          copy_chunk<CB>(p + v * nt * 16, x + k * nt * 8 + v * E);
          if constexpr (RES) copy_chunk<CB>(p + plane + v * nt * 16, r + k * nt * 8 + v * E);
        }
      }
    }
    fx += step_x;
    if constexpr (RES) fr += step_r;
    copy_commit();
  };
  auto chunk = [&](int place) {
    Chunk<T> c;
#pragma unroll
    for (int v = 0; v < CB / 16; ++v)
      reinterpret_cast<uint4*>(&c)[v] =
          *reinterpret_cast<const uint4*>(ring + place + t * 16 + v * nt * 16);
    return c;
  };
  int64_t left = a.rows - first_row;                     // rows of this pair and behind
  fetch(0, left);
  uint64_t w[NV][4], b[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int col = (t + k * nt) * 8;
    float f[8];
    load_weight8<T, true>(a.w, a.w_f32, col, cols - col, f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[k][i] = has[k] ? f2_pack(f[2 * i], f[2 * i + 1]) : 0;   // y is 0 behind the row
    load_bias8<T, true>(a.b, a.w_f32, col, cols - col, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[k][i] = f2_pack(f[2 * i], f[2 * i + 1]);
  }
  // elements of a row that a warp holds
  auto held = [&](int of) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int rest = cols - (of * 32 + k * nt) * 8;
      n += rest < 0 ? 0 : rest < 256 ? rest : 256;
    }
    return (float)n;
  };
  const float n_mine = held(warp), inv_mine = n_mine > 0.f ? 1.f / n_mine : 0.f;
  const float n_lane = (lane & 15) < nt / 32 ? held(lane & 15) : 0.f;
  int count = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) count += has[k] ? 8 : 0;
  const float mine_n = (float)count, inv_n = count ? 1.f / mine_n : 0.f;

  int slot = 0, place = 0;
  for (; left > 0; left -= step) {
    fetch(place ^ stage, left - step);
    copy_wait<1>();
    uint64_t h[RB][NV][4];
    float sum[RB], sq[RB];
    const bool two = left > 1;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      uint64_t s2 = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (has[k]) {
          const int at = place + rb * TENSORS * plane + k * nt * CB;
          unpack2(chunk(at), h[rb][k]);
          if constexpr (RES) {
            uint64_t r[4];
            unpack2(chunk(at + plane), r);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[rb][k][i] = fadd2(h[rb][k][i], r[i]);
            if (a.h && (rb == 0 || two)) store8(ph + rb * cols + k * nt * 8, h[rb][k]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[rb][k][i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fadd2(s2, h[rb][k][i]);
      }
      float s0, s1;
      f2_unpack(s2, s0, s1);
      sum[rb] = s0 + s1;
    }
    float pivot[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      pivot[rb] = __shfl_sync(0xffffffffu, sum[rb] * inv_n, 0);
      sum[rb] = fmaf(-mine_n, pivot[rb], sum[rb]);
      uint64_t q2 = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const float off = has[k] ? -pivot[rb] : 0.f;
        const uint64_t oo = f2_pack(off, off);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint64_t d = fadd2(h[rb][k][i], oo);
          q2 = ffma2(d, d, q2);
        }
      }
      float s0, s1;
      f2_unpack(q2, s0, s1);
      sq[rb] = s0 + s1;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], o);
        sq[rb] += __shfl_xor_sync(0xffffffffu, sq[rb], o);
      }
    if (lane == 0) {
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
        buf[slot][rb][warp] = make_float2(fmaf(sum[rb], inv_mine, pivot[rb]),
                                          fmaf(-sum[rb] * inv_mine, sum[rb], sq[rb]));
    }
    __syncthreads();
    float first[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      first[rb] = buf[slot][rb][0].x;
      const float2 v = n_lane > 0.f ? buf[slot][rb][lane & 15] : make_float2(first[rb], 0.f);
      const float d = v.x - first[rb];
      sum[rb] = n_lane * d;
      sq[rb] = fmaf(sum[rb], d, v.y);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        sum[rb] += __shfl_xor_sync(0xffffffffu, sum[rb], o);
        sq[rb] += __shfl_xor_sync(0xffffffffu, sq[rb], o);
      }
    slot ^= 1;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const bool in = rb == 0 || two;
      const float mean = fmaf(sum[rb], inv_cols, first[rb]);
      const float var = fmaf(-sum[rb] * inv_cols, sum[rb], sq[rb]) * inv_cols;
      const float rstd = rsqrtf((var < 0.f ? 0.f : var) + a.eps);
      if (t == 0 && in) {
        const int64_t row = a.rows - left + rb;
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
      const uint64_t rr = f2_pack(rstd, rstd), mm = f2_pack(-mean, -mean);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          h[rb][k][i] = ffma2(fmul2(fadd2(h[rb][k][i], mm), rr), w[k][i], b[k][i]);
        if ((FMT8 == 0 || a.y) && in && has[k]) store8(py + rb * cols + k * nt * 8, h[rb][k]);
        if constexpr (FMT8 != 0) {
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) f2_unpack(h[rb][k][i], f[2 * i], f[2 * i + 1]);
          const float scale = scale_of(lanes_amax(amax8(f), a.group / 8), FMT8);
          if (in && has[k]) {
            const int col = (t + k * nt) * 8;
            store_codes<true>(pc + rb * cols + k * nt * 8, encode8<FMT8>(f, scale), 8);
            if ((col & (a.group - 1)) == 0)
              a.scales[(a.rows - left + rb) * a.groups + (col >> a.shift)] = scale;
          }
        }
      }
    }
    py += step_y;
    if constexpr (RES) ph += step_y;
    if constexpr (FMT8 != 0) pc += step_y;
    place ^= stage;
  }
}

// Launches the kernel of pairs of rows on rows that it takes, else cudaErrorNotSupported.
template <typename T, int FMT8>
cudaError_t pairs_of(const LayerNormFwd& a, cudaStream_t st) {
  const Plan p = plan(a.cols, 512, 64);
  cudaError_t e = cudaErrorNotSupported;
  if (p.lpr || p.nv > 2 || p.threads > 512 || (FMT8 && !a.group)) return e;
  const size_t row = (size_t)p.nv * p.threads * sizeof(Chunk<T>);
  auto go = [&](auto nv, auto res, auto full) {
    constexpr int N = decltype(nv)::value;
    constexpr bool RES = decltype(res)::value != 0;
    constexpr int RB = FMT8 && N == 2 ? 1 : 2;
    constexpr auto* k = layer_norm_pair_kernel<T, N, RB, FMT8, RES, decltype(full)::value != 0>;
    const size_t smem = 2 * RB * (RES ? 2 : 1) * row;
    e = allow_smem<k>((int)kMaxSmem);
    if (e != cudaSuccess) return;
    const int64_t pairs = (a.rows + RB - 1) / RB;
    k<<<grid(pairs, 1, fwd_blocks(pairs, p, pair_regs(N), smem)), p.threads, smem, st>>>(a);
    e = cudaGetLastError();
  };
  if (a.r && 8 * row > kMaxSmem / 2) return e;
  auto of = [&](auto nv, auto res) {
    a.cols == (int64_t)8 * p.nv * p.threads ? go(nv, res, Int<1>()) : go(nv, res, Int<0>());
  };
  if (a.r)
    p.nv == 1 ? of(Int<1>(), Int<1>()) : of(Int<2>(), Int<1>());
  else
    p.nv == 1 ? of(Int<1>(), Int<0>()) : of(Int<2>(), Int<0>());
  return e;
}

}  // namespace

namespace norm {

cudaError_t layer_fwd_pairs(int dtype, const LayerNormFwd& a, cudaStream_t st) {
  const int fmt = a.codes ? a.fmt : 0;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    return fmt == 0          ? pairs_of<T, 0>(a, st)
           : fmt == kFmtInt8 ? pairs_of<T, kFmtInt8>(a, st)
                             : pairs_of<T, kFmtE4m3>(a, st);
  });
}

}  // namespace norm

}  // namespace bl
