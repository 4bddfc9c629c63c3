// Activations held in 8 bits between the forward and the backward: saving
// (one scale a group of 32, 64 or 128 elements of a row, or one a row),
// loading, and the expansion of an attention's q, k and v into its backward's
// workspace.  The format is in rows.cuh.  All passes are bound by HBM: x once
// in, one byte an element and the scales out, or the other way round.
#include <type_traits>

#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

constexpr int kExpandU = 2;

// Quotient and remainder by a divisor that does not change over a launch, in
// 32 bits wherever the dividend allows.
__device__ __forceinline__ void div_mod(int64_t x, int64_t d, int64_t& q, int64_t& r) {
  if ((uint64_t)x >> 32) {
    q = x / d;
    r = x - q * d;
  } else {
    const uint32_t qq = (uint32_t)x / (uint32_t)d;
    q = qq;
    r = (uint32_t)x - qq * (uint32_t)d;
  }
}

// Groups back to back in memory (every row a whole number of them): no rows,
// no division.  A lane holds 16 elements, so group / 16 = 2, 4 or 8
// neighbouring lanes hold a group; a thread takes U such pieces, 256 apart, and
// loads all of them before it works on any, which keeps U * 32 bytes of a
// 16-bit type in flight for each thread.  Bound by HBM: 168M bf16 elements to
// int8 in 73 us, 6.9 TB/s (one chunk of 8 a thread and divisions to find the
// row: 155 us).
template <typename T, int FMT, int U>
__global__ void __launch_bounds__(256) act_save_flat_kernel(const T* __restrict__ x,
                                                            uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales,
                                                            int64_t pieces, int shift) {
  const int lanes = 1 << shift;
  const int64_t p0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  Chunk<T> c[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
#pragma unroll
    for (int v = 0; v < 2; ++v) c[u][v] = load8<T, true>(x + p * 16 + v * 8, p < pieces ? 8 : 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
    float f[2][8];
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v][i] = to_f32(c[u][v].e[i]);
    const float scale = scale_of(lanes_amax(amax2(amax8(f[0]), amax8(f[1])), lanes), FMT);
    const Codes lo = encode8<FMT>(f[0], scale), hi = encode8<FMT>(f[1], scale);
    if (p < pieces) {
      reinterpret_cast<uint4*>(codes)[p] = make_uint4(lo.w[0], lo.w[1], hi.w[0], hi.w[1]);
      if ((p & (lanes - 1)) == 0) scales[p >> shift] = scale;
    }
  }
}

// Groups of `a.group` elements of rows of any width and stride: a.group / 8
// neighbouring lanes hold one, each lane one chunk.  A row takes a whole number
// of groups (the last may be cut).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) act_save_groups_kernel(ActSave a) {
  const int lanes = a.group / 8;                    // 4, 8 or 16
  const int64_t per_row = a.groups * lanes;         // chunks of a row, padded
  const int64_t total = a.rows * per_row;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t x0 = (int64_t)blockIdx.x * blockDim.x; x0 < total; x0 += stride) {
    const int64_t x = x0 + threadIdx.x;
    const bool in = x < total;
    int64_t row, j;
    div_mod(in ? x : 0, per_row, row, j);
    const int64_t col = j * 8;
    const int64_t left = in ? a.cols - col : 0;
    const int valid = (int)(left < 8 ? left : 8);
    const Chunk<T> c = load8<T, VEC>(static_cast<const T*>(a.x) + row * a.x_stride + col, valid);
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(c.e[i]);
    const float scale = scale_of(lanes_amax(amax8(f), lanes), a.fmt);
    store_codes<VEC>(a.codes + row * a.cols + col, encode8(a.fmt, f, scale), valid);
    if (in && (j & (lanes - 1)) == 0) a.scales[row * a.groups + j / lanes] = scale;
  }
}

// One scale a row: a warp (BLOCK: a block) goes over its row twice, for the
// maximum and for the codes; the second reading comes from the caches.  For rows
// that the row kernels of norm_fwd.cu do not take: fp32 that starts anywhere, and
// more than 16384 columns (16376 of 16-bit rows that start anywhere).
template <typename T, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(256) act_save_rows_kernel(ActSave a) {
  __shared__ float buf[2][32];
  const int t = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int step = BLOCK ? 256 : 32;
  const int rows_here = BLOCK ? 1 : 8;
  int slot = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * rows_here; row0 < a.rows;
       row0 += (int64_t)gridDim.x * rows_here) {
    const int64_t row = row0 + (BLOCK ? 0 : threadIdx.x >> 5);
    const int64_t cols = row < a.rows ? a.cols : 0;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    float m = 0.f;
#pragma unroll 4
    for (int64_t col = t * 8; col < cols; col += step * 8) {
      const int valid = (int)min((int64_t)8, cols - col);
      const Chunk<T> c = load8<T, VEC>(x + col, valid);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_f32(c.e[i]);
      m = amax2(m, amax8(f));
    }
    if constexpr (BLOCK) {
      m = block_amax(m, buf, slot);
      slot ^= 1;
    } else {
      __syncwarp();
      m = lanes_amax(m, 32);
    }
    const float scale = scale_of(m, a.fmt);
#pragma unroll 4
    for (int64_t col = t * 8; col < cols; col += step * 8) {
      const int valid = (int)min((int64_t)8, cols - col);
      const Chunk<T> c = load8<T, VEC>(x + col, valid);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = to_f32(c.e[i]);
      store_codes<VEC>(a.codes + row * a.cols + col, encode8(a.fmt, f, scale), valid);
    }
    if (t == 0 && row < a.rows) a.scales[row] = scale;
  }
}

// Rows of whole groups back to back in memory, as in the flat saving kernel.
// Bound by HBM: 168M codes to bf16 in 75 us, 6.7 TB/s (83 us with two 16-byte
// stores a piece).
template <typename T, int FMT, int U, bool W32>
__global__ void __launch_bounds__(256) act_load_flat_kernel(const uint8_t* __restrict__ codes,
                                                            const float* __restrict__ scales,
                                                            T* __restrict__ x, int64_t pieces,
                                                            int shift) {
  const int64_t p0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x;
  uint4 raw[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
    raw[u] = make_uint4(0u, 0u, 0u, 0u);
    scale[u] = 0.f;
    if (p < pieces) {
      raw[u] = __ldg(reinterpret_cast<const uint4*>(codes) + p);
      scale[u] = __ldg(scales + (p >> shift));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
    if (p >= pieces) return;
    const Codes c[2] = {{{raw[u].x, raw[u].y}}, {{raw[u].z, raw[u].w}}};
    float f[2][8];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      decode8<FMT>(c[v], f[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v][i] *= scale[u];
    }
    store16<T, W32>(x + p * 16, f);
  }
}

// Rows of any width: codes and values lie back to back whatever the width, so a
// thread still moves 8 of them with vector instructions (VEC).  WHOLE: the width
// is a multiple of 8, so the 8 share a scale; otherwise the scale is looked up
// anew where a row or a group begins.
template <typename T, bool VEC, bool WHOLE, int FMT>
__global__ void __launch_bounds__(256) act_load_kernel(ActLoad a) {
  const int64_t total = a.rows * a.cols;
  const int shift = group_shift(a.group);
  const int64_t stride = (int64_t)gridDim.x * 256 * 8;
  for (int64_t x = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; x < total; x += stride) {
    int64_t row, col;
    div_mod(x, a.cols, row, col);
    const int valid = (int)min((int64_t)8, total - x);
    const Codes c = VEC && valid == 8 ? load_codes<true>(a.codes + x, 8)
                                      : load_codes<false>(a.codes + x, valid);
    float f[8];
    decode8<FMT>(c, f);
    float scale = a.scales[row * a.groups + (col >> shift)];
    if constexpr (WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= scale;
    } else {
      // elements up to the next border, and those behind it
      int here = (int)min(min(((col >> shift) + 1) << shift, a.cols) - col, (int64_t)8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i == here && i < valid) {
          col += here;
          if (col == a.cols) {
            col = 0;
            ++row;
          }
          scale = a.scales[row * a.groups + (col >> shift)];
          here += (int)min(min(((col >> shift) + 1) << shift, a.cols) - col, (int64_t)8);
          col -= i;                                   // so that adding `here` leads on
        }
        f[i] *= scale;
      }
    }
    if (VEC && valid == 8)
      store8<T, true>(static_cast<T*>(a.x) + x, f, 8);
    else
      store8<T, false>(static_cast<T*>(a.x) + x, f, valid);
  }
}

// q, k and v of an attention, [tokens, heads, D] codes with one scale a
// (token, head), to bf16: pieces of 16 as in the flat loading kernel.  The blocks
// of the three tensors follow one another.  Bound by HBM and, at attention
// sizes, by the ramp up and down: 19M elements in 15 us.
template <int D, int FMT, bool W32>
__global__ void __launch_bounds__(256) expand_kernel(Expand a) {
  constexpr int PER_ROW = D / 16, U = kExpandU;
  int s = 0;
  int64_t blk = blockIdx.x;
  while (s < 2 && blk >= a.blocks[s]) blk -= a.blocks[s++];
  const int64_t pieces = a.rows[s] * PER_ROW;
  const int64_t p0 = blk * (256 * U) + threadIdx.x;
  uint4 raw[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
    if (p < pieces) {
      raw[u] = __ldg(reinterpret_cast<const uint4*>(a.codes[s]) + p);
      scale[u] = __ldg(a.scales[s] + p / PER_ROW);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t p = p0 + u * 256;
    if (p >= pieces) return;
    const Codes c[2] = {{{raw[u].x, raw[u].y}}, {{raw[u].z, raw[u].w}}};
    float f[2][8];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      decode8<FMT>(c[v], f[v]);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[v][i] *= scale[u];
    }
    store16<__nv_bfloat16, W32>(static_cast<__nv_bfloat16*>(a.out[s]) + p * 16, f);
  }
}

constexpr int64_t kMaxBlocks = 152 * 64;

unsigned blocks_for(int64_t units) {
  return (unsigned)(units < kMaxBlocks ? units : kMaxBlocks);
}

// Pieces of 16 elements a thread of the flat kernels.
constexpr int kFlatU = 2;

// Whether the flat kernels take rows of `cols` with this group: then the shift
// from a piece to its group.
int flat_shift(int64_t cols, int group) {
  if (!group || cols % group) return -1;
  return group_shift(group) - 4;
}

}  // namespace

cudaError_t launch_act_save(int dtype, const ActSave& in, cudaStream_t st) {
  ActSave a = in;
  if (a.rows == 0) return cudaSuccess;
  // one scale a row of 32, 64 or 128 elements is one scale a group
  if (!a.group && (a.cols == 32 || a.cols == 64 || a.cols == 128)) a.group = (int)a.cols;
  const bool flat = a.x_stride == a.cols && flat_shift(a.cols, a.group) >= 0 &&
                    aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 16);
  // whole rows, and groups of rows that are aligned at least
  if (!flat && (!a.group || (a.cols % 8 == 0 && a.x_stride % 8 == 0 &&
                             aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 8)))) {
    const cudaError_t e = launch_row_save(dtype, a, st);
    if (e != cudaErrorNotSupported) return e;
  }
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = a.cols % 8 == 0 && a.x_stride % 8 == 0 &&
                     aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 8);
    if (flat) {
      const int shift = flat_shift(a.cols, a.group);
      const int64_t pieces = a.rows * (a.cols / 16);
      const unsigned g = (unsigned)((pieces + 256 * kFlatU - 1) / (256 * kFlatU));
      auto* x = static_cast<const T*>(a.x);
      if (a.fmt == kFmtInt8)
        act_save_flat_kernel<T, kFmtInt8, kFlatU><<<g, 256, 0, st>>>(x, a.codes, a.scales, pieces,
                                                                     shift);
      else
        act_save_flat_kernel<T, kFmtE4m3, kFlatU><<<g, 256, 0, st>>>(x, a.codes, a.scales, pieces,
                                                                     shift);
    } else if (a.group) {
      const int64_t units = (a.rows * a.groups * (a.group / 8) + 255) / 256;
      if (vec)
        act_save_groups_kernel<T, true><<<blocks_for(units), 256, 0, st>>>(a);
      else
        act_save_groups_kernel<T, false><<<blocks_for(units), 256, 0, st>>>(a);
    } else {
      if constexpr (sizeof(T) == 4)
        if (a.cols <= 1024) {
          act_save_rows_kernel<T, false, false><<<blocks_for((a.rows + 7) / 8), 256, 0, st>>>(a);
          return cudaGetLastError();
        }
      if (vec)
        act_save_rows_kernel<T, true, true><<<blocks_for(a.rows), 256, 0, st>>>(a);
      else
        act_save_rows_kernel<T, false, true><<<blocks_for(a.rows), 256, 0, st>>>(a);
    }
    return cudaGetLastError();
  });
}

cudaError_t launch_act_load(int dtype, const ActLoad& in, cudaStream_t st) {
  ActLoad a = in;
  if (a.rows == 0) return cudaSuccess;
  if (!a.group && (a.cols == 32 || a.cols == 64 || a.cols == 128)) a.group = (int)a.cols;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    const bool vec = aligned_to(a.x, chunk_align(dtype)) && aligned_to(a.codes, 8);
    const int shift = aligned_to(a.x, 16) && aligned_to(a.codes, 16)
                          ? flat_shift(a.cols, a.group) : -1;
    if (shift >= 0) {
      const int64_t pieces = a.rows * (a.cols / 16);
      const unsigned g = (unsigned)((pieces + 256 * kFlatU - 1) / (256 * kFlatU));
      auto* x = static_cast<T*>(a.x);
      auto flat = [&](auto fmt, auto w32) {
        act_load_flat_kernel<T, decltype(fmt)::value, kFlatU, decltype(w32)::value>
            <<<g, 256, 0, st>>>(a.codes, a.scales, x, pieces, shift);
      };
      const std::integral_constant<int, kFmtInt8> i8;
      const std::integral_constant<int, kFmtE4m3> e4;
      if (aligned_to(a.x, 32))
        a.fmt == kFmtInt8 ? flat(i8, std::true_type()) : flat(e4, std::true_type());
      else
        a.fmt == kFmtInt8 ? flat(i8, std::false_type()) : flat(e4, std::false_type());
      return cudaGetLastError();
    }
    const unsigned g = blocks_for((a.rows * a.cols + 2047) / 2048);
    auto launch = [&](auto fmt) {
      constexpr int F = decltype(fmt)::value;
      if (!vec)
        act_load_kernel<T, false, false, F><<<g, 256, 0, st>>>(a);
      else if (a.cols % 8 == 0)
        act_load_kernel<T, true, true, F><<<g, 256, 0, st>>>(a);
      else
        act_load_kernel<T, true, false, F><<<g, 256, 0, st>>>(a);
    };
    if (a.fmt == kFmtInt8)
      launch(std::integral_constant<int, kFmtInt8>());
    else
      launch(std::integral_constant<int, kFmtE4m3>());
    return cudaGetLastError();
  });
}

cudaError_t launch_expand(int d, int fmt, const Expand& in, cudaStream_t st) {
  Expand a = in;
  int64_t blocks = 0;
  for (int s = 0; s < 3; ++s) {
    a.blocks[s] = (a.rows[s] * (d / 16) + 256 * kExpandU - 1) / (256 * kExpandU);
    blocks += a.blocks[s];
  }
  const unsigned g = (unsigned)blocks;
  bool w32 = true;
  for (int s = 0; s < 3; ++s) w32 = w32 && aligned_to(a.out[s], 32);
  auto launch = [&](auto dim, auto f) {
    constexpr int D = decltype(dim)::value, F = decltype(f)::value;
    if (w32)
      expand_kernel<D, F, true><<<g, 256, 0, st>>>(a);
    else
      expand_kernel<D, F, false><<<g, 256, 0, st>>>(a);
  };
  const std::integral_constant<int, kFmtInt8> i8;
  const std::integral_constant<int, kFmtE4m3> e4;
  if (d == 64) {
    const std::integral_constant<int, 64> dim;
    fmt == kFmtInt8 ? launch(dim, i8) : launch(dim, e4);
  } else {
    const std::integral_constant<int, 128> dim;
    fmt == kFmtInt8 ? launch(dim, i8) : launch(dim, e4);
  }
  return cudaGetLastError();
}

}  // namespace bl
