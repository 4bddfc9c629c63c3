// Saving in e4m3 for products in 8 bits (gemm8.cu): of a tensor [rows, cols], in one
// reading, with one scale for every
//   128 elements of a row        the codes that products over the columns read
//   128 elements of a column     those of products over the rows
//   128 x 128 elements           a weight's, which both kinds of product read
// in the format of rows.cuh.  And the loading of the last two.
//
// A block takes a tile of 128 x 128: a thread has a chunk of 8 columns of 8 rows, 16
// apart, so a row lies in 16 neighbouring lanes and a column in 16 threads of 8 warps.
// The tile waits in shared memory for its second use (in registers, where the compiler
// kept it as 64 fp32 numbers a thread, two blocks fit an SM: 16384 x 4096 bf16 to rows
// and columns in 74 us, 53 so: 75% of the copy rate, the issue slots 75% busy; rows or
// columns alone 89 and 84%, a weight's blocks 83%).
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

// 8 codes to a row of codes of which `valid` exist; WIDE: 8-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void put_codes(uint8_t* p, const Codes& c, int valid) {
  if (WIDE && valid >= 8)
    store_codes<true>(p, c, 8);
  else
    store_codes<false>(p, c, valid);
}

template <typename T, bool VEC, bool WIDE>
__global__ void __launch_bounds__(256) tile_save_kernel(TileSave a) {
  constexpr int CB = (int)sizeof(Chunk<T>);
  extern __shared__ __align__(16) uint8_t tile[];        // a thread's chunks in its own places
  __shared__ float part[8][128];
  __shared__ __align__(16) float col_scale[128];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t tiles_x = (a.cols + 127) / 128;
  const int64_t bx = blockIdx.x % tiles_x, by = blockIdx.x / tiles_x;
  const int64_t row0 = by * 128 + ty, col0 = bx * 128, col = col0 + tx * 8;
  const int valid = (int)min(max(a.cols - col, (int64_t)0), (int64_t)8);
  const int here = (int)min(max((a.rows - row0 + 15) / 16, (int64_t)0), (int64_t)8);  // rows
  uint8_t* const mine = tile + threadIdx.x * 16;
  {
    const T* x = static_cast<const T*>(a.x) + row0 * a.x_stride + col;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint8_t* p = mine + k * 256 * CB;
      if (VEC && k < here && valid) {
#pragma unroll
        for (int v = 0; v < CB / 16; ++v)
          copy_chunk<CB>(p + v * 256 * 16, x + v * (16 / (int)sizeof(T)));
      } else {
        const Chunk<T> c = load8<T, false>(x, !VEC && k < here ? valid : 0);
#pragma unroll
        for (int v = 0; v < CB / 16; ++v)
          *reinterpret_cast<uint4*>(p + v * 256 * 16) = reinterpret_cast<const uint4*>(&c)[v];
      }
      x += 16 * a.x_stride;
    }
    copy_commit();
    copy_wait<0>();
  }
  auto chunk = [&](int k, float (&f)[8]) {
    Chunk<T> c;
#pragma unroll
    for (int v = 0; v < CB / 16; ++v)
      reinterpret_cast<uint4*>(&c)[v] =
          *reinterpret_cast<const uint4*>(mine + k * 256 * CB + v * 256 * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(c.e[i]);
  };
  float top[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool rows = a.row_codes != nullptr, down = a.col_codes || a.block_codes;
  uint8_t* to = a.row_codes + row0 * a.row_stride + col;
#pragma unroll 2
  for (int k = 0; k < 8; ++k) {
    float f[8];
    chunk(k, f);
    if (rows) {
      const float scale = scale_of(lanes_amax(amax8(f), 16), kFmtE4m3);
      if (k < here) {
        put_codes<WIDE>(to, encode8<kFmtE4m3>(f, scale), valid);
        if (tx == 0) a.row_scales[(row0 + 16 * k) * tiles_x + bx] = scale;
      }
      to += 16 * a.row_stride;
    }
    if (down) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = amax2(top[i], f[i]);
    }
  }
  if (!down) return;
  if (a.block_codes) {
    const float m = lanes_amax(amax8(top), 32);
    if ((threadIdx.x & 31) == 0) part[0][threadIdx.x >> 5] = m;
    __syncthreads();
    const float scale = scale_of(lanes_amax(part[0][threadIdx.x & 7], 8), kFmtE4m3);
    if (threadIdx.x == 0) a.block_scales[by * tiles_x + bx] = scale;
    to = a.block_codes + row0 * a.block_stride + col;
#pragma unroll 4
    for (int k = 0; k < 8; ++k) {
      float f[8];
      chunk(k, f);
      if (k < here) put_codes<WIDE>(to, encode8<kFmtE4m3>(f, scale), valid);
      to += 16 * a.block_stride;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top[i] = amax2(top[i], __shfl_xor_sync(0xffffffffu, top[i], 16));
    if ((threadIdx.x & 16) == 0) part[threadIdx.x >> 5][tx * 8 + i] = top[i];
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    float m = part[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = amax2(m, part[w][threadIdx.x]);
    const float scale = scale_of(m, kFmtE4m3);
    col_scale[threadIdx.x] = scale;
    if (col0 + threadIdx.x < a.cols) a.col_scales[by * a.cols + col0 + threadIdx.x] = scale;
  }
  __syncthreads();
  float inv[8];
  uint32_t keep[2] = {0u, 0u};                           // codes 0 under a scale that is NaN
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float scale = col_scale[tx * 8 + i];
    inv[i] = __frcp_rn(scale);
    if (!isnan(scale)) keep[i / 4] |= 0xffu << (8 * (i % 4));
  }
  to = a.col_codes + row0 * a.col_stride + col;
#pragma unroll 4
  for (int k = 0; k < 8; ++k) {
    float f[8];
    chunk(k, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], inv[i]);
    Codes codes = encode8<kFmtE4m3>(f, 1.f);
    codes.w[0] &= keep[0];
    codes.w[1] &= keep[1];
    if (k < here) put_codes<WIDE>(to, codes, valid);
    to += 16 * a.col_stride;
  }
}

// (16384 x 4096 bf16: columns' groups 70 us, 43% of the copy rate, blocks 66 us.)
// Values of codes [rows, cols] whose scale lies at scales[(row / 128) * s_row + (col >> shift)
// * s_col]: columns' groups (shift 0) or blocks (7).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) tile_load_kernel(TileLoad a) {
  const int64_t per_row = (a.cols + 7) / 8, total = a.rows * per_row;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += step) {
    const int64_t row = x / per_row, col = (x - row * per_row) * 8;
    const int valid = (int)min(a.cols - col, (int64_t)8);
    const Codes c = load_codes<VEC>(a.codes + row * a.stride + col, valid);
    const float* s = a.scales + (row >> 7) * a.groups;
    float f[8];
    decode8<kFmtE4m3>(c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) f[i] *= s[(col + i) >> a.shift];
    store8<T, VEC>(static_cast<T*>(a.x) + row * a.cols + col, f, valid);
  }
}

// Rows of codes that start anywhere to rows `pitch` bytes apart (16-byte aligned), 16 bytes
// a thread out of the aligned words that cover them; two tensors in one launch, of which
// either may have no rows.
__global__ void __launch_bounds__(256) repitch_kernel(Repitch a, Repitch b) {
  const int64_t row_a = (a.cols + 15) / 16, row_b = (b.cols + 15) / 16;
  const int64_t in_a = a.rows * row_a, total = in_a + b.rows * row_b;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < total; x += step) {
    const bool first = x < in_a;
    const Repitch& t = first ? a : b;
    const int64_t per_row = first ? row_a : row_b, y = first ? x : x - in_a;
    const int64_t row = y / per_row, col = (y - row * per_row) * 16;
    const uint8_t* const begin = t.from + row * t.from_pitch;
    const uintptr_t at = reinterpret_cast<uintptr_t>(begin + col);
    const uintptr_t end = reinterpret_cast<uintptr_t>(begin + t.cols);
    const uint32_t* p = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
    uint32_t w[5], out[4];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = reinterpret_cast<uintptr_t>(p + i) < end ? __ldg(p + i) : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], (int)(at & 3) * 8);
    *reinterpret_cast<uint4*>(t.to + row * t.pitch + col) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
}

}  // namespace

cudaError_t launch_repitch(const Repitch& a, const Repitch& b, cudaStream_t st) {
  const int64_t pieces = a.rows * ((a.cols + 15) / 16) + b.rows * ((b.cols + 15) / 16);
  const int64_t blocks = (pieces + 255) / 256;
  repitch_kernel<<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, st>>>(a, b);
  return cudaGetLastError();
}

cudaError_t launch_tile_save(int dtype, const TileSave& a, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 && aligned_to(a.x, chunk_align(dtype));
    const bool wide = a.row_stride % 8 == 0 && a.col_stride % 8 == 0 && a.block_stride % 8 == 0 &&
                      aligned_to(a.row_codes, 8) && aligned_to(a.col_codes, 8) &&
                      aligned_to(a.block_codes, 8);
    const unsigned g = (unsigned)tiles;
    constexpr int smem = 128 * 128 * (int)sizeof(T);
    auto go = [&](auto v, auto w) {
      constexpr auto* k = tile_save_kernel<T, decltype(v)::value, decltype(w)::value>;
      const cudaError_t e = allow_smem<k>(smem);
      if (e != cudaSuccess) return e;
      k<<<g, 256, smem, st>>>(a);
      return cudaGetLastError();
    };
    if (vec && wide) return go(std::true_type(), std::true_type());
    return wide ? go(std::false_type(), std::true_type())
                : go(std::false_type(), std::false_type());
  });
}

cudaError_t launch_tile_load(int dtype, const TileLoad& a, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const int64_t blocks = (a.rows * ((a.cols + 7) / 8) + 255) / 256;
    const unsigned g = (unsigned)(blocks < 152 * 64 ? blocks : 152 * 64);
    if (a.cols % 8 == 0 && a.stride % 8 == 0 && aligned_to(a.codes, 8) &&
        aligned_to(a.x, chunk_align(dtype)))
      tile_load_kernel<T, true><<<g, 256, 0, st>>>(a);
    else
      tile_load_kernel<T, false><<<g, 256, 0, st>>>(a);
    return cudaGetLastError();
  });
}

}  // namespace bl
