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
//
// This file has what the forward (norm_fwd.cu) and the backward (norm_bwd.cu)
// share: how rows are laid over threads, and how launches are sized.
#pragma once

#include <atomic>
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
// touch a sector a lane.  fp32, 32760 x 2561: forward 45 -> 64% of the copy rate, 83%
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

template <int LPR>
__device__ __forceinline__ float row_sum(float v, float (*buf)[32], int& slot) {
  if constexpr (LPR != 0) return lanes_sum(v, LPR);
  v = block_sum(v, buf, slot);
  slot ^= 1;
  return v;
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

// The ring kernels for rows that start anywhere (norm_fwd_odd.cu: 16-bit types;
// norm_bwd_odd.cu: those, and fp32 that a block holds, without 8 bits);
// cudaErrorNotSupported for others and where a row is too wide.
cudaError_t fwd_odd(int dtype, bool norm, const NormFwd& a, cudaStream_t st);
cudaError_t bwd_odd(int dtype, const NormBwd& a, int* blocks, cudaStream_t st);

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

}  // namespace norm
}  // namespace bl
