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
// A thread forms the two counters' words of 8 neighbouring elements, 35 wide products and
// some 40 three-input xors, while the elements' own loads are under way.  With a residual
// that hides behind HBM (32760 x 5120 bf16 in 154 us, 96% of the copy rate; fp32 98%
// without one too); two bytes in and out an element do not suffice for it (16384 x 4096 bf16
// in 58 us, 68%: the multipliers 67% busy and dispatch in the way).
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

constexpr int kRuns = 32;      // blocks an SM: they take turns out of step

// The generator of a call: the rounds' keys, kept in registers (formed anew for every
// counter they cost 36 of some 200 instructions a chunk), and what the first two rounds
// make of the words that many counters share, the offset and the counter's upper half.
struct Philox {
  static constexpr uint32_t kM0 = 0xD2511F53u, kM1 = 0xCD9E8D57u;
  uint32_t k0[10], k1[10], o0, o1;
  uint32_t b1, p2_hi, p2_lo;
  __device__ __forceinline__ explicit Philox(const int64_t* state) {
    const uint64_t seed = (uint64_t)__ldg(reinterpret_cast<const long long*>(state));
    const uint64_t offset = (uint64_t)__ldg(reinterpret_cast<const long long*>(state) + 1);
    o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      k0[r] = (uint32_t)seed + r * 0x9E3779B9u;
      k1[r] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
      asm volatile("" : "+r"(k0[r]), "+r"(k1[r]));
    }
  }
  // For the counters with this upper half.
  __device__ __forceinline__ void upper(uint32_t high) {
    const uint64_t q = (uint64_t)o0 * kM1;
    const uint64_t p = (uint64_t)((uint32_t)(q >> 32) ^ high ^ k0[0]) * kM0;
    b1 = (uint32_t)q;
    p2_hi = (uint32_t)(p >> 32);
    p2_lo = (uint32_t)p;
  }
  // The four words of the counter whose lower half times kM0 is p.
  __device__ __forceinline__ void words(uint64_t p, uint32_t (&w)[4]) const {
    uint64_t q = (uint64_t)((uint32_t)(p >> 32) ^ o1 ^ k1[0]) * kM1;
    uint32_t a = (uint32_t)(q >> 32) ^ b1 ^ k0[1], b = (uint32_t)q;
    uint32_t c = p2_hi ^ (uint32_t)p ^ k1[1], d = p2_lo;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
      p = (uint64_t)a * kM0, q = (uint64_t)c * kM1;
      a = (uint32_t)(q >> 32) ^ b ^ k0[r];
      b = (uint32_t)q;
      c = (uint32_t)(p >> 32) ^ d ^ k1[r];
      d = (uint32_t)p;
    }
    w[0] = a, w[1] = b, w[2] = c, w[3] = d;
  }
};

// Two neighbours of a chunk as fp32.
template <typename T>
__device__ __forceinline__ void two(const Chunk<T>& c, int i, float& lo, float& hi) {
  lo = to_f32(c.e[2 * i]);
  hi = to_f32(c.e[2 * i + 1]);
}
// (byte moves and masks: the shift would go to the multipliers, which are the bound)
template <>
__device__ __forceinline__ void two(const Chunk<__nv_bfloat16>& c, int i, float& lo, float& hi) {
  const uint32_t w = reinterpret_cast<const uint32_t*>(&c)[i];
  lo = __uint_as_float(__byte_perm(w, 0, 0x1044));
  hi = __uint_as_float(w & 0xffff0000u);
}

// Two elements: what is dropped is 0 before its product, so infinities go too.  ALL: all
// are, p = 1 or within 2^-33 of it.
template <bool ALL>
__device__ __forceinline__ uint64_t drop2(const Dropout& a, uint32_t w0, uint32_t w1, float x0,
                                          float x1, uint64_t scale, bool add, uint64_t r) {
  const uint64_t x = f2_pack(!ALL && w0 >= a.threshold ? x0 : 0.f,
                             !ALL && w1 >= a.threshold ? x1 : 0.f);
  return add ? ffma2(x, scale, r) : fmul2(x, scale);
}

// Dense tensors: chunks of 8 elements back to back.  A block walks runs of U times
// 256 chunks, gridDim.x runs apart; the next run's loads are under way while this one's
// words are formed.
template <typename T, bool ADD, bool ALL>
__global__ void __launch_bounds__(256) dropout_kernel(Dropout a) {
  constexpr int U = sizeof(T) == 2 ? 2 : 1;
  const int64_t total = a.rows * a.cols, chunks = total / 8;
  const T* __restrict__ x = static_cast<const T*>(a.x);
  const T* __restrict__ r = static_cast<const T*>(a.r);
  int64_t c0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * (256 * U);
  Chunk<T> cx[U], cr[ADD ? U : 1];
  auto load = [&](int64_t at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = at + u * 256;
      cx[u] = load8<T, true>(x + c * 8, c < chunks ? 8 : 0);
      if constexpr (ADD) cr[u] = load8<T, true>(r + c * 8, c < chunks ? 8 : 0);
    }
  };
  load(c0);
  Philox gen(a.state);
  const uint64_t scale = f2_pack(a.scale, a.scale);
  for (; c0 < chunks; c0 += step) {
    Chunk<T> nx[U], nr[ADD ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nx[u] = cx[u];
      if constexpr (ADD) nr[u] = cr[u];
    }
    load(c0 + step);
    // the run's counters share their upper half: 2 * 256 * U is a power of two
    gen.upper((uint32_t)((uint64_t)c0 >> 31));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + u * 256;
      uint32_t w[2][4];
      const uint64_t p = (uint64_t)((uint32_t)c * 2) * Philox::kM0;
      gen.words(p, w[0]);
      gen.words(p + Philox::kM0, w[1]);
      uint64_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x0, x1, r0 = 0.f, r1 = 0.f;
        two(nx[u], i, x0, x1);
        if constexpr (ADD) two(nr[u], i, r0, r1);
        out[i] = drop2<ALL>(a, w[i / 2][2 * i % 4], w[i / 2][2 * i % 4 + 1], x0, x1, scale, ADD,
                            f2_pack(r0, r1));
      }
      if (c < chunks) store8(static_cast<T*>(a.y) + c * 8, out);
    }
  }
  // what is left behind the chunks
  const int64_t at = chunks * 8 + threadIdx.x;
  if (blockIdx.x == 0 && at < total) {
    gen.upper((uint32_t)((uint64_t)chunks >> 31));
    uint32_t w[4];
    gen.words((uint64_t)(uint32_t)(at / 4) * Philox::kM0, w);
    const uint32_t word = at % 4 < 2 ? (at % 4 ? w[1] : w[0]) : at % 4 == 2 ? w[2] : w[3];
    float lo, hi;
    f2_unpack(drop2<ALL>(a, word, 0, to_f32(x[at]), 0.f, scale, ADD,
                         f2_pack(ADD ? to_f32(r[at]) : 0.f, 0.f)),
              lo, hi);
    static_cast<T*>(a.y)[at] = from_f32<T>(lo);
  }
}

// Elements wherever they lie (rows apart, tensors that start anywhere): a thread takes the
// four of a counter, each at its own place.
template <typename T, bool ALL>
__global__ void __launch_bounds__(256) dropout_rows_kernel(Dropout a) {
  const int64_t total = a.rows * a.cols;
  const int64_t step = (int64_t)gridDim.x * 256 * 4;
  Philox gen(a.state);
  const uint64_t scale = f2_pack(a.scale, a.scale);
  for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; at < total; at += step) {
    uint32_t w[4];
    gen.upper((uint32_t)(at >> 34));
    gen.words((uint64_t)(uint32_t)(at / 4) * Philox::kM0, w);
    int64_t row = at / a.cols, col = at - row * a.cols;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (at + i >= total) break;
      const float x = to_f32(static_cast<const T*>(a.x)[row * a.x_stride + col]);
      const float r = a.r ? to_f32(static_cast<const T*>(a.r)[row * a.r_stride + col]) : 0.f;
      float lo, hi;
      f2_unpack(drop2<ALL>(a, w[i], 0, x, 0.f, scale, a.r != nullptr, f2_pack(r, 0.f)), lo, hi);
      static_cast<T*>(a.y)[at + i] = from_f32<T>(lo);
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
    const bool dense = a.rows == 1 || (a.x_stride == a.cols && (!a.r || a.r_stride == a.cols));
    const size_t al = chunk_align(dtype);
    if (dense && total >= 8 && aligned_to(a.x, al) && aligned_to(a.r, al) && aligned_to(a.y, al)) {
      constexpr int U = sizeof(T) == 2 ? 2 : 1;
      const int64_t runs = (total / 8 + 256 * U - 1) / (256 * U), most = 152 * kRuns;
      const unsigned g = (unsigned)(runs < most ? runs : most);
      if (a.all)
        a.r ? dropout_kernel<T, true, true><<<g, 256, 0, st>>>(a)
            : dropout_kernel<T, false, true><<<g, 256, 0, st>>>(a);
      else
        a.r ? dropout_kernel<T, true, false><<<g, 256, 0, st>>>(a)
            : dropout_kernel<T, false, false><<<g, 256, 0, st>>>(a);
    } else {
      const int64_t blocks = (total + 1023) / 1024;
      const unsigned g = (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
      a.all ? dropout_rows_kernel<T, true><<<g, 256, 0, st>>>(a)
            : dropout_rows_kernel<T, false><<<g, 256, 0, st>>>(a);
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_dropout_next(int64_t* state, int64_t* used, cudaStream_t st) {
  next_kernel<<<1, 1, 0, st>>>(state, used);
  return cudaGetLastError();
}

}  // namespace bl
