// Rows of a matrix in chunks of 8 consecutive elements, the unit that the row
// kernels (norm_fwd.cu, norm_bwd.cu, act8.cu) load, keep in registers and store: 16 bytes of
// a 16-bit type, 32 of fp32, 8 of codes.  With VEC a chunk is whole and
// aligned and moves in one or two vector instructions; otherwise element by
// element under a count of valid elements (odd widths, views whose rows start
// anywhere).
//
// Also the 8-bit format: a group of consecutive elements of a row shares one
// fp32 scale,
//   scale = amax * fl32(1 / qmax), at least 2^-126 and at most the largest
//           number whose product with qmax is finite; qmax = 127 (int8) or 448
//           (e4m3),
//   code  = round to nearest even of fl32(x * fl32(1 / scale)),
//   value = code * scale.
// The bounds keep 1 / scale and every value finite, so an all-zero group needs
// no case of its own.  A NaN or an infinity in the group makes the scale NaN (codes
// 0): the whole group loads as NaN instead of as a wrong number.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace bl {

constexpr int kFmtInt8 = 1, kFmtE4m3 = 2;
// The largest fp32 numbers whose products with 127 and 448 are finite.
constexpr float kTopInt8 = 0x1.020406p+121f, kTopE4m3 = 0x1.249248p+119f;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

template <typename T>
struct alignas(16) Chunk {
  T e[8];
};
struct alignas(8) Codes {
  uint32_t w[2];
};

// 16 or 32 bytes in one instruction each way (32: 32-byte aligned).  Two 16-byte
// stores of a lane, 32 bytes apart from lane to lane, write every 32-byte sector
// in two halves.
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[4]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 8 elements at p, of which `valid` exist (the others read as zero).
template <typename T, bool VEC>
__device__ __forceinline__ Chunk<T> load8(const T* __restrict__ p, int valid) {
  Chunk<T> c;
  if constexpr (VEC) {
    uint32_t(&w)[sizeof(c) / 4] = *reinterpret_cast<uint32_t(*)[sizeof(c) / 4]>(&c);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(c) / 4); ++i) w[i] = 0;
    if (valid > 0) load_words(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c.e[i] = i < valid ? p[i] : from_f32<T>(0.f);
  }
  return c;
}

// Two values rounded to T, in one 32-bit word (two words of fp32).
template <typename T> struct Pair;
template <> struct Pair<float> {
  float2 v;
  __device__ __forceinline__ Pair(float a, float b) : v(make_float2(a, b)) {}
};
template <> struct Pair<__half> {
  __half2 v;
  __device__ __forceinline__ Pair(float a, float b) : v(__floats2half2_rn(a, b)) {}
};
template <> struct Pair<__nv_bfloat16> {
  __nv_bfloat162 v;
  __device__ __forceinline__ Pair(float a, float b) : v(__floats2bfloat162_rn(a, b)) {}
};

template <typename T>
__device__ __forceinline__ Chunk<T> pack8(const float (&f)[8]) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<Pair<T>*>(&c)[i] = Pair<T>(f[2 * i], f[2 * i + 1]);
  return c;
}

// The chunk as four packed pairs of fp32 (f2_* in common.cuh).
template <typename T>
__device__ __forceinline__ void unpack2(const Chunk<T>& c, uint64_t (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(to_f32(c.e[2 * i]), to_f32(c.e[2 * i + 1]));
}
template <typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, const uint64_t (&f)[4]) {
  Chunk<T> c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f[i], lo, hi);
    reinterpret_cast<Pair<T>*>(&c)[i] = Pair<T>(lo, hi);
  }
  store_words(p, *reinterpret_cast<const uint32_t(*)[sizeof(c) / 4]>(&c));
}

// Four pairs rounded to a 16-bit type.
template <typename T>
__device__ __forceinline__ void pack_words(const uint64_t (&f)[4], uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f[i], lo, hi);
    const Pair<T> p(lo, hi);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* __restrict__ p, const float (&f)[8], int valid) {
  const Chunk<T> c = pack8<T>(f);
  if constexpr (VEC) {
    if (valid > 0) store_words(p, *reinterpret_cast<const uint32_t(*)[sizeof(c) / 4]>(&c));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = c.e[i];
  }
}

// 16 values rounded to T and written to 16 consecutive elements, 32-byte aligned
// with W32, 16-byte aligned without.
template <typename T, bool W32>
__device__ __forceinline__ void store16(T* __restrict__ p, const float (&f)[2][8]) {
  if constexpr (W32 && sizeof(T) == 2) {
    struct alignas(16) { Chunk<T> c[2]; } both = {{pack8<T>(f[0]), pack8<T>(f[1])}};
    store_words(p, *reinterpret_cast<const uint32_t(*)[8]>(&both));
  } else if constexpr (W32 || sizeof(T) == 2) {
    store8<T, true>(p, f[0], 8);
    store8<T, true>(p + 8, f[1], 8);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      reinterpret_cast<float4*>(p)[v] = make_float4(f[v / 2][4 * (v % 2)], f[v / 2][4 * (v % 2) + 1],
                                                    f[v / 2][4 * (v % 2) + 2],
                                                    f[v / 2][4 * (v % 2) + 3]);
  }
}

template <bool VEC>
__device__ __forceinline__ Codes load_codes(const uint8_t* __restrict__ p, int valid) {
  Codes c{{0u, 0u}};
  if constexpr (VEC) {
    if (valid > 0) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      c.w[0] = v.x;
      c.w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) c.w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  }
  return c;
}

template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, Codes c, int valid) {
  if constexpr (VEC) {
    if (valid > 0) *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = (uint8_t)(c.w[i / 4] >> (8 * (i % 4)));
  }
}

// Codes as floats (without the scale).  int8: the byte with its sign bit
// flipped is placed in the low mantissa bits of 2^23, so one add takes off
// 2^23 + 128 and leaves the exact integer; that is full-rate arithmetic where
// an integer-to-float conversion is not.
template <int FMT>
__device__ __forceinline__ void decode8(const Codes& c, float (&f)[8]) {
  if constexpr (FMT == kFmtInt8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t flipped = c.w[i / 4] ^ 0x80808080u;
      const uint32_t bits = __byte_perm(flipped, 0x4b000000u, 0x7650 + (i % 4));
      f[i] = __uint_as_float(bits) - 8388736.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t two = (uint16_t)(c.w[i / 2] >> (16 * (i % 2)));
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3);
      const float2 v = __half22float2(__half2(h));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}

// Largest magnitude of 8 values, NaN if there is one among them; the sign of
// the result is arbitrary (a maximum of magnitudes in one instruction).
__device__ __forceinline__ float amax2(float a, float b) {
  float d;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float amax8(const float (&f)[8]) {
  return amax2(amax2(amax2(f[0], f[1]), amax2(f[2], f[3])),
               amax2(amax2(f[4], f[5]), amax2(f[6], f[7])));
}

// The scale of a group whose largest magnitude is |amax|.
__device__ __forceinline__ float scale_of(float amax, int fmt) {
  const bool i8 = fmt == kFmtInt8;
  const float a = fabsf(amax);
  float s = fmaxf(__fmul_rn(a, i8 ? 1.f / 127.f : 1.f / 448.f), 1.17549435e-38f);
  s = fminf(s, i8 ? kTopInt8 : kTopE4m3);
  return a <= 3.402823466e38f ? s : __uint_as_float(0x7fffffffu);
}

// The codes of 8 values of a group with this scale.  |x / scale| stays below
// qmax (1 + 2^-21), which rounds to qmax, so nothing is clamped.  int8: adding
// 1.5 * 2^23 rounds to an integer (ties to even) and leaves its two's
// complement in the low mantissa byte.
template <int FMT>
__device__ __forceinline__ Codes encode8(const float (&f)[8], float scale) {
  Codes c{{0u, 0u}};
  const float inv = __frcp_rn(scale);
  if constexpr (FMT == kFmtInt8) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      b[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], inv), 12582912.f));
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c.w[i] = __byte_perm(__byte_perm(b[4 * i], b[4 * i + 1], 0x0040),
                           __byte_perm(b[4 * i + 2], b[4 * i + 3], 0x0040), 0x5410);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = make_float2(__fmul_rn(f[2 * i], inv), __fmul_rn(f[2 * i + 1], inv));
      c.w[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3)
                    << (16 * (i % 2));
    }
  }
  if (isnan(scale)) c = Codes{{0u, 0u}};
  return c;
}

__device__ __forceinline__ Codes encode8(int fmt, const float (&f)[8], float scale) {
  return fmt == kFmtInt8 ? encode8<kFmtInt8>(f, scale) : encode8<kFmtE4m3>(f, scale);
}
__device__ __forceinline__ void decode8(int fmt, const Codes& c, float (&f)[8]) {
  if (fmt == kFmtInt8)
    decode8<kFmtInt8>(c, f);
  else
    decode8<kFmtE4m3>(c, f);
}

// Over `width` neighbouring lanes (a power of two up to 32; uniform).
__device__ __forceinline__ float lanes_amax(float v, int width) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width) v = amax2(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int width) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum (largest magnitude) over the block: warp partials through one of two
// slots of `buf`, which the caller alternates, so that one barrier a reduction
// is enough: a slot is written again only after the barrier of the reduction
// in between.  Every thread gets the result, formed in the same order.
__device__ __forceinline__ float block_sum(float v, float (*buf)[32], int slot) {
  v = lanes_sum(v, 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[slot][warp] = v;
  __syncthreads();
  return lanes_sum(lane < warps ? buf[slot][lane] : 0.f, 32);
}
__device__ __forceinline__ float block_amax(float v, float (*buf)[32], int slot) {
  v = lanes_amax(v, 32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) buf[slot][warp] = v;
  __syncthreads();
  return lanes_amax(lane < warps ? buf[slot][lane] : 0.f, 32);
}

// Asynchronous copies of 4, 8 or 16 bytes from global to shared memory.  The
// row kernels give every thread its own places, which it fills for rows ahead
// and reads itself, so that waiting for its own copies is all it needs.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
                 : "memory");
}
// 16 bytes that share their 32-byte sector with another copy of the same thread:
// through L1, so that the sector comes once.
__device__ __forceinline__ void copy_async_half(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
// 16 bytes of a chunk of CB.
template <int CB>
__device__ __forceinline__ void copy_chunk(void* dst, const void* src) {
  if constexpr (CB == 16)
    copy_async<16>(dst, src);
  else
    copy_async_half(dst, src);
}
// The same for the first `size` bytes (0 to BYTES), the others become zero.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int size) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(size)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES),
                 "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Rows that start anywhere.  The aligned vectors that cover such a row are
// copied whole; chunk c of the row lies in vectors c and c + 1, shifted by the
// row's misalignment.  Writing, a lane's aligned vector is made of the end of the
// chunk of the lane in front and the beginning of its own.

// Bytes shift .. shift + 4 W of the 8 W bytes in w (4 W a power of two).
template <int W>
__device__ __forceinline__ void shift_bytes(uint32_t (&w)[2 * W], int shift, uint32_t (&out)[W]) {
#pragma unroll
  for (int step = W / 2; step > 0; step /= 2)
    if (shift & (4 * step)) {
#pragma unroll
      for (int i = 0; i + step < 2 * W; ++i) w[i] = w[i + step];
    }
  const int bits = (shift & 3) * 8;
#pragma unroll
  for (int i = 0; i < W; ++i) out[i] = __funnelshift_r(w[i], w[i + 1], bits);
}

// Copies aligned vector c of the row of `cols` 16-bit elements at `row` (c = 0
// holds its beginning); what lies behind the row's end becomes zero.  A vector may
// begin up to 14 bytes in front of the row, within the same aligned 16 bytes.
template <typename T>
__device__ __forceinline__ void copy_odd(void* place, const T* row, int c, int cols) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row);
  const uintptr_t from = (at & ~(uintptr_t)15) + (uintptr_t)c * 16, end = at + (uintptr_t)cols * 2;
  const int left = from < end ? (int)(end - from) : 0;
  copy_async<16>(place, reinterpret_cast<const void*>(left ? from : at & ~(uintptr_t)15),
                 left < 16 ? left : 16);
}

// The thread's chunk of a row that copy_odd brought to places `p`, one vector a
// thread and then, nt places on, the next chunks of the same threads; t is the
// thread's first chunk.
template <typename T, int LPR>
__device__ __forceinline__ Chunk<T> chunk_odd(const uint8_t* p, int t, int nt, const T* row) {
  // behind the last lane of a row comes its first lane's next place
  const uint8_t* next = LPR && t == LPR - 1 ? p + (nt - (LPR - 1)) * 16 : p + 16;
  const uint4 lo = *reinterpret_cast<const uint4*>(p), hi = *reinterpret_cast<const uint4*>(next);
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  Chunk<T> c;
  shift_bytes<4>(w, (int)(reinterpret_cast<uintptr_t>(row) & 15),
                 *reinterpret_cast<uint32_t(*)[4]>(&c));
  return c;
}

// The same for codes: vectors of 8 bytes.
__device__ __forceinline__ void copy_odd8(void* place, const uint8_t* row, int c, int cols) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(row);
  const uintptr_t from = (at & ~(uintptr_t)7) + (uintptr_t)c * 8, end = at + (uintptr_t)cols;
  const int left = from < end ? (int)(end - from) : 0;
  copy_async<8>(place, reinterpret_cast<const void*>(left ? from : at & ~(uintptr_t)7),
                left < 8 ? left : 8);
}
template <int LPR>
__device__ __forceinline__ Codes codes_odd(const uint8_t* p, int t, int nt, const uint8_t* row) {
  const uint8_t* next = LPR && t == LPR - 1 ? p + (nt - (LPR - 1)) * 8 : p + 8;
  const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(next);
  uint32_t w[4] = {lo.x, lo.y, hi.x, hi.y};
  Codes c;
  shift_bytes<2>(w, (int)(reinterpret_cast<uintptr_t>(row) & 7), c.w);
  return c;
}

// Writes the chunks (8 elements of W / 2 bytes) that the lanes hold to the row at
// `row`: chunk c, of which `valid` elements exist.  `front` and `behind`: whether
// the lane in front (behind) holds the chunk in front (behind), whose valid
// elements are then those of a row of `cols`.  The whole warp takes part.
template <int W>
__device__ __forceinline__ void store_anywhere(uint8_t* row, int c, int valid, int cols, bool front,
                                               bool behind, const uint32_t (&w)[W]) {
  constexpr int E = W / 2;                            // bytes of an element
  const int off = (int)(reinterpret_cast<uintptr_t>(row) & (4 * W - 1));
  const int k = off / E;                              // elements of the chunk in front
  uint32_t both[2 * W], out[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    both[i] = __shfl_up_sync(0xffffffffu, w[i], 1);
    both[W + i] = w[i];
  }
  uint8_t* p = row + c * (4 * W);
  const bool whole = valid >= 8 - k && (k == 0 || front);
  if (whole) {
    if (k == 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) out[i] = w[i];
    } else {
      shift_bytes<W>(both, 4 * W - off, out);
    }
    if constexpr (W == 4)
      *reinterpret_cast<uint4*>(p - off) = make_uint4(out[0], out[1], out[2], out[3]);
    else
      *reinterpret_cast<uint2*>(p - off) = make_uint2(out[0], out[1]);
  }
  // what no lane's vector holds, element by element
  const int next = min(cols - (c + 1) * 8, 8);        // valid elements of the chunk behind
  const int from = whole ? 8 - k : 0;
  const int to = behind && next >= 8 - k ? min(valid, 8 - k) : valid;
  if (from < to) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= from && i < to) {
        const uint32_t bits = w[i * E / 4] >> (8 * (i * E % 4));
        if constexpr (E == 2)
          reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)bits;
        else
          p[i] = (uint8_t)bits;
      }
  }
}

// A weight row of type T or fp32 (or none: ones).
template <typename T, bool VEC>
__device__ __forceinline__ void load_weight8(const void* w, bool f32, int64_t col, int valid,
                                             float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (f32) {
    const Chunk<float> c = load8<float, VEC>(static_cast<const float*>(w) + col, valid);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c.e[i];
  } else {
    const Chunk<T> c = load8<T, VEC>(static_cast<const T*>(w) + col, valid);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = to_f32(c.e[i]);
  }
}

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Bytes that a vector of 8 elements wants to be aligned to.
inline size_t chunk_align(int dtype) { return dtype == 2 ? 32 : 16; }

// Calls f with a null pointer of the element type that `dtype` (BL_BF16,
// BL_FP16, BL_FP32) names.
template <typename F>
cudaError_t with_type(int dtype, F&& f) {
  if (dtype == 0) return f((__nv_bfloat16*)nullptr);
  if (dtype == 1) return f((__half*)nullptr);
  return f((float*)nullptr);
}

// Shift from a column to its group (one group a row: any column to 0).
inline __host__ __device__ int group_shift(int group) {
  return group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 31;
}

inline int64_t groups_of(int64_t cols, int group) {
  return group ? (cols + group - 1) / group : 1;
}

}  // namespace bl
