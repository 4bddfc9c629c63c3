// Dropout from a counter-based generator, with a residual's addition behind it:
//
//   y_i = x_i / (1 - p) where element i is kept, else 0;  y_i += r_i
//
// Element i (its place in the dense tensor, whatever the strides) is kept iff word
// i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers:
// as easy as 1, 2, 3", SC 2011) of the counter (i / 4, offset) and the key `seed` is at
// least round(p 2^32).  The mask is a function of i, so it is never stored: the
// gradient is the same call on g_y.
//
// A thread forms the two counters' words of 8 neighbouring elements: 40 wide products
// and as many three-input xors for them, while the elements' own loads are under way.
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

struct Key {
  uint32_t k0, k1, o0, o1;
  __device__ __forceinline__ explicit Key(const int64_t* state) {
    const uint64_t seed = (uint64_t)__ldg(reinterpret_cast<const long long*>(state));
    const uint64_t offset = (uint64_t)__ldg(reinterpret_cast<const long long*>(state) + 1);
    k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
    o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
  }
};

__device__ __forceinline__ void philox(const Key& key, uint64_t j, uint32_t (&w)[4]) {
  uint32_t a = (uint32_t)j, b = (uint32_t)(j >> 32), c = key.o0, d = key.o1;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)a * 0xD2511F53u, q = (uint64_t)c * 0xCD9E8D57u;
    a = (uint32_t)(q >> 32) ^ b ^ k0;
    b = (uint32_t)q;
    c = (uint32_t)(p >> 32) ^ d ^ k1;
    d = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = a, w[1] = b, w[2] = c, w[3] = d;
}

__device__ __forceinline__ float drop(const Dropout& a, uint32_t word, float x, float r) {
  return (word >= a.threshold && !a.all ? x * a.scale : 0.f) + r;
}

// Dense tensors: chunks of 8 elements back to back, U of them a thread, 256 apart.  The
// last chunk may be cut, and without VEC none needs to be aligned.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(256) dropout_kernel(Dropout a) {
  const int64_t total = a.rows * a.cols;
  const int64_t c0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.r);
  Chunk<T> cx[U], cr[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = (c0 + u * 256) * 8;
    const int valid = (int)min(max(total - at, (int64_t)0), (int64_t)8);
    if (VEC && valid == 8) {
      cx[u] = load8<T, true>(x + at, 8);
      if (r) cr[u] = load8<T, true>(r + at, 8);
    } else {
      cx[u] = load8<T, false>(x + at, valid);
      if (r) cr[u] = load8<T, false>(r + at, valid);
    }
  }
  const Key key(a.state);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = (c0 + u * 256) * 8;
    if (at >= total) return;
    const int valid = (int)min(total - at, (int64_t)8);
    uint32_t w[2][4];
    philox(key, (uint64_t)at / 4, w[0]);
    philox(key, (uint64_t)at / 4 + 1, w[1]);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = drop(a, w[i / 4][i % 4], to_f32(cx[u].e[i]), r ? to_f32(cr[u].e[i]) : 0.f);
    T* y = static_cast<T*>(a.y) + at;
    if (VEC && valid == 8)
      store8<T, true>(y, f, 8);
    else
      store8<T, false>(y, f, valid);
  }
}

// Rows apart: a thread takes the four elements of a counter, each at its own place.
template <typename T>
__global__ void __launch_bounds__(256) dropout_rows_kernel(Dropout a) {
  const int64_t total = a.rows * a.cols;
  const int64_t step = (int64_t)gridDim.x * 256 * 4;
  const Key key(a.state);
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < total; at += step) {
    uint32_t w[4];
    philox(key, (uint64_t)at / 4, w);
    int64_t row = at / a.cols, col = at - row * a.cols;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at + i >= total) break;
      const float x = to_f32(static_cast<const T*>(a.x)[row * a.x_stride + col]);
      const float r = a.r ? to_f32(static_cast<const T*>(a.r)[row * a.r_stride + col]) : 0.f;
      static_cast<T*>(a.y)[at + i] = from_f32<T>(drop(a, w[i], x, r));
      if (++col == a.cols) {
        col = 0;
        ++row;
      }
    }
  }
}

__global__ void next_kernel(int64_t* state, int64_t* used) {
  const int64_t seed = state[0], offset = state[1];
  used[0] = seed;
  used[1] = offset;
  state[1] = (int64_t)((uint64_t)offset + 1);
}

}  // namespace

cudaError_t launch_dropout(int dtype, const Dropout& a, cudaStream_t st) {
  const int64_t total = a.rows * a.cols;
  if (total == 0) return cudaSuccess;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    if (a.rows > 1 && (a.x_stride != a.cols || (a.r && a.r_stride != a.cols))) {
      const int64_t blocks = (total + 1023) / 1024;
      dropout_rows_kernel<T><<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, st>>>(a);
      return cudaGetLastError();
    }
    const size_t al = chunk_align(dtype);
    constexpr int U = 2;
    const unsigned g = (unsigned)((total + 2048 * U - 1) / (2048 * U));
    if (aligned_to(a.x, al) && aligned_to(a.r, al) && aligned_to(a.y, al))
      dropout_kernel<T, true, U><<<g, 256, 0, st>>>(a);
    else
      dropout_kernel<T, false, U><<<g, 256, 0, st>>>(a);
    return cudaGetLastError();
  });
}

cudaError_t launch_dropout_next(int64_t* state, int64_t* used, cudaStream_t st) {
  next_kernel<<<1, 1, 0, st>>>(state, used);
  return cudaGetLastError();
}

}  // namespace bl
