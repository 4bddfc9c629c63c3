// Norms of rows: the root-mean-square norm, with the residual's addition in front, an
// output in 8 bits and the backward pass:
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = (h rstd) w
//
// and, for the gradients g_y of y and g_h of h (the residual stream's own),
//   u = h rstd,  c = mean(w g_y u),
//   g_x = g_r = rstd (w g_y - u c) + g_h,   g_w = sum over rows of g_y u.
//
// Layer norm:
//
//   h = x + r,  m = mean(h),  rstd = 1 / sqrt(mean((h - m)^2) + eps),
//   y = (h - m) rstd w + b,  and with u = (h - m) rstd, c = mean(w g_y u),
//   g_x = g_r = rstd (w g_y - mean(w g_y) - u c) + g_h,
//   g_w = sum over rows of g_y u,  g_b = sum over rows of g_y.
//
// Sums run in fp32; y comes from the unrounded h, so it is rounded once.
// The passes are bound by HBM: each input read once, each output written once.
//
// This file has what the forward (norm_fwd.cu) and the backward (norm_bwd.cu)
// share: how rows are laid over threads, and how launches are sized.
#pragma once

#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace bl {
namespace norm {

// A row is held by LPR lanes of a warp (8, 16 or 32, each with NV chunks) or by the
// whole block (LPR = 0).
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
// The 8 elements of a row that a thread has in its unit k.  Chunks: 8 neighbours.
// SPREAD: R.step apart, so that the lanes of an access have neighbouring elements:
// for rows that start anywhere, where a chunk would take 8 accesses that each
// touch a sector a lane.  fp32, 32760 x 2561: forward 45 -> 68% of the copy rate, 87%
// with a residual; straight from global memory, as 4-byte copies to the ring wait
// on their own number (54 and 52%).  Backward 63% on the ring, 33% without.
template <bool SPREAD, int LPR>
__device__ __forceinline__ int col_of(const Rows<LPR>& R, int k, int i) {
  return SPREAD ? (k * 8 + i) * R.step + R.t : (R.t + k * R.step) * 8 + i;
}
template <typename T, bool VEC, bool SPREAD, int LPR>
__device__ __forceinline__ Chunk<T> load_unit(const T* __restrict__ row, const Rows<LPR>& R, int k,
                                              int cols) {
  if constexpr (!SPREAD) {
    const int col = col_of<false>(R, k, 0);
    return load8<T, VEC>(row + col, cols - col);
  } else {
    Chunk<T> c;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = col_of<true>(R, k, i);
      c.e[i] = col < cols ? row[col] : from_f32<T>(0.f);
    }
    return c;
  }
}
template <typename T, bool VEC, bool SPREAD, int LPR>
__device__ __forceinline__ void store_unit(T* __restrict__ row, const Rows<LPR>& R, int k, int cols,
                                           const float (&f)[8]) {
  if constexpr (!SPREAD) {
    const int col = col_of<false>(R, k, 0);
    store8<T, VEC>(row + col, f, cols - col);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = col_of<true>(R, k, i);
      if (col < cols) row[col] = from_f32<T>(f[i]);
    }
  }
}
template <typename T, bool VEC, bool SPREAD, int LPR>
__device__ __forceinline__ void weight_unit(const void* w, bool f32, const Rows<LPR>& R, int k,
                                            int cols, float (&f)[8]) {
  if constexpr (!SPREAD) {
    const int col = col_of<false>(R, k, 0);
    load_weight8<T, VEC>(w, f32, col, cols - col, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = col_of<true>(R, k, i);
      f[i] = !w            ? 1.f
             : col >= cols ? 0.f
             : f32         ? static_cast<const float*>(w)[col]
                           : to_f32(static_cast<const T*>(w)[col]);
    }
  }
}

// The same through a plane of shared memory, fp32: element i of unit k lies
// 4 bytes a thread apart from its neighbours', and those behind the row are zero.
template <int LPR>
__device__ __forceinline__ void copy_spread(uint8_t* plane, const float* row, const Rows<LPR>& R,
                                            int k, int nt, int cols) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int col = col_of<true>(R, k, i);
    copy_async<4>(plane + ((k * 8 + i) * nt + (int)threadIdx.x) * 4, row + (col < cols ? col : 0),
                  col < cols ? 4 : 0);
  }
}
__device__ __forceinline__ Chunk<float> chunk_spread(const uint8_t* plane, int k, int nt) {
  Chunk<float> c;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c.e[i] = *reinterpret_cast<const float*>(plane + ((k * 8 + i) * nt + (int)threadIdx.x) * 4);
  return c;
}

// Whether the lane in front (behind) of this one's holds the chunk in front
// (behind): not across the ends of a warp or, with LPR, of a row's lanes.
template <int LPR>
__device__ __forceinline__ bool lane_in_front(const Rows<LPR>& R) {
  return LPR ? R.t > 0 : (threadIdx.x & 31) > 0;
}
template <int LPR>
__device__ __forceinline__ bool lane_behind(const Rows<LPR>& R) {
  return LPR ? R.t < LPR - 1 : (threadIdx.x & 31) < 31;
}

template <int LPR, int N>
__device__ __forceinline__ float row_sum(float v, float (*buf)[N], int& slot) {
  if constexpr (LPR != 0) return lanes_sum(v, LPR);
  v = block_sum(v, buf, slot);
  slot ^= 1;
  return v;
}

// Two sums at once (32 + 32 partial sums a slot of buf).
template <int LPR>
__device__ __forceinline__ float2 row_sum2(float2 v, float (*buf)[64], int& slot) {
  v.x = lanes_sum(v.x, LPR ? LPR : 32);
  v.y = lanes_sum(v.y, LPR ? LPR : 32);
  if constexpr (LPR == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    float* b = buf[slot];
    if (lane == 0) {
      b[warp] = v.x;
      b[32 + warp] = v.y;
    }
    __syncthreads();
    v.x = lanes_sum(lane < warps ? b[lane] : 0.f, 32);
    v.y = lanes_sum(lane < warps ? b[32 + lane] : 0.f, 32);
    slot ^= 1;
  }
  return v;
}

// sum / n, inv = fl(1 / n), to within a rounding: a row of one number whose sum is exact has
// that number for its mean, and what is taken from it leaves 0.
__device__ __forceinline__ float mean_of(float sum, float inv, float n) {
  const float mean = sum * inv;
  return fmaf(fmaf(-mean, n, sum), inv, mean);
}

// Lanes a row (0: the block), chunks a thread and threads of a launch over rows
// of `cols` columns.  Up to warp_chunks chunks a warp holds whole rows and needs
// no barrier; beyond, a block of as few threads as hold the row with two chunks
// each, one chunk up to 1024 columns, where blocks are small.
struct Plan {
  int lpr, nv, threads, here;
};
inline Plan plan(int64_t cols, int max_threads, int warp_chunks, bool odd = false) {
  // rows that start anywhere need a place for one vector more
  const int chunks = (int)((cols + 7) / 8) + (odd ? 1 : 0);
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

// The fewest threads of such a block with nv chunks each, two or four.
constexpr int fewest_threads(int nv, int max_threads) {
  return ((nv == 4 ? 2 * max_threads : 128) / nv + 32) / 32 * 32;
}

constexpr int kSMs = 152;
constexpr size_t kMaxSmem = 220 * 1024;

// Blocks that are resident at once: `regs` a thread, `smem` bytes a block.
inline int resident(int threads, int regs, size_t smem) {
  int n = 65536 / (regs * threads);
  const int by_smem = (int)(kMaxSmem / (smem + 1536));
  if (n > by_smem) n = by_smem;
  if (n > 2048 / threads) n = 2048 / threads;
  if (n < 1) n = 1;
  return kSMs * n;
}
inline unsigned grid(int64_t rows, int here, int most) {
  const int64_t blocks = (rows + here - 1) / here;
  return (unsigned)(blocks < most ? blocks : most);
}

// Blocks of the forward's ring kernel.  One block for each that is resident runs them all
// in step: the reads of all blocks and then their writes come in bursts.  Eight
// times as many, as far as a block keeps about six rows, take turns out of step and
// work on neighbouring rows: 5120 columns 84 -> 99% of the copy rate without and
// 90 -> 101% with a residual, 128 columns 83 -> 96%; blocks of fewer rows lose it
// again to filling their rings (4096 rows of 4096: 87 -> 70% at eight times).
inline int fwd_blocks(int64_t rows, const Plan& p, int regs, size_t smem) {
  const int once = resident(p.threads, regs, smem);
  int64_t times = rows / ((int64_t)once * p.here * 6);
  if (times > 8) times = 8;
  if (times < 1) times = 1;
  return (int)(once * times);
}

// The ring kernels for rows that start anywhere (norm_fwd_odd.cu: 16-bit types;
// norm_bwd_odd.cu: those, and fp32 that a block holds, without 8 bits);
// cudaErrorNotSupported for others and where a row is too wide.
cudaError_t fwd_odd(int dtype, bool norm, const NormFwd& a, cudaStream_t st);
cudaError_t bwd_odd(int dtype, const NormBwd& a, int* blocks, cudaStream_t st);
// The layer norm's.
cudaError_t layer_fwd_odd(int dtype, const LayerNormFwd& a, cudaStream_t st);
// The layer norm's forward, two rows at a time (layer_norm_pairs.cu), where it takes the
// rows: whole aligned chunks, held by a block with two chunks a thread at most, and no
// scale a row.
cudaError_t layer_fwd_pairs(int dtype, const LayerNormFwd& a, cudaStream_t st);
// Its backward on such rows (layer_norm_bwd_rows.cu).
cudaError_t layer_bwd_rows(int dtype, const NormBwd& a, int* blocks, cudaStream_t st);
cudaError_t layer_bwd_odd(int dtype, const NormBwd& a, int* blocks, cudaStream_t st);

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

}  // namespace norm
}  // namespace bl
