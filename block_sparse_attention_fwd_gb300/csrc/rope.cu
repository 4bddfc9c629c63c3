// Rotary positions with several axes, on q and k in one launch, forward and
// inverse (the gradient's rotation).
//
// Pair p of the first 2 * pairs dimensions of a head belongs to one axis (the
// pairs are dealt to the axes in consecutive sections) and turns by the angle
// position[token][axis] * f_p:
//   (u, v) -> (u cos - v sin, u sin + v cos)
// with (u, v) = (x[2p], x[2p + 1]) interleaved, (x[p], x[p + pairs]) in
// halves; the dimensions behind 2 * pairs pass through.
//
// Angles.  f_p comes as a 64-bit fixed-point fraction of a turn,
// F_p = round(f_p / (2 pi) * 2^64), so position * F_p modulo 2^64 is the angle
// modulo one turn: an integer product keeps what an fp32 product loses (at
// position 10^6 and f = 1 half a step of the angle is 0.03 rad), without
// fp64, whose rate here is low, and without a table to read.  The upper 32
// bits, as a signed number of half turns, go to sincospi in fp32.
//
// The pass is bound by HBM: q and k once in, once out.  A group of lanes
// covers one head of one token with 16-byte vectors; a thread takes the same
// vector of U heads, so that the sines are formed once for U heads and U
// loads are in flight.
#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

__device__ __forceinline__ void turn(const Rope& a, const int32_t* pos, int p, float& c, float& s) {
  int axis = 0;
#pragma unroll
  for (int e = 0; e < 3; ++e) axis += p >= a.ends[e] ? 1 : 0;
  const uint64_t angle = (uint64_t)(int64_t)pos[axis] * a.freqs[p];
  sincospif((float)(int32_t)(angle >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  if (a.inverse) s = -s;
}

// VECW elements (16 bytes) of a head at a time.
template <typename T, int U, bool HALF>
__global__ void __launch_bounds__(256) rope_kernel(Rope a) {
  constexpr int W = 16 / sizeof(T);
  struct alignas(16) Vec { T e[W]; };
  const int lanes = a.lanes;                       // lanes a head
  const int here = 256 / lanes;                    // units a block
  const int g = threadIdx.x / lanes, lane = threadIdx.x % lanes;
  const int64_t unit = (int64_t)blockIdx.x * here + g;
  if (g >= here || unit >= a.units) return;
  const uint32_t per_token = a.q_units + a.k_units;
  const uint32_t token = (uint32_t)unit / per_token;
  uint32_t hc = (uint32_t)unit % per_token;
  const uint32_t b = token / (uint32_t)a.n, i = token % (uint32_t)a.n;
  const bool is_k = hc >= a.q_units;
  if (is_k) hc -= a.q_units;
  const int heads = is_k ? a.Hk : a.H;
  const int h0 = hc * U;
  const T* in = static_cast<const T*>(is_k ? a.k : a.q);
  T* out = static_cast<T*>(is_k ? a.k_out : a.q_out);
  const int64_t* si = is_k ? a.ks : a.qs;
  const int64_t* so = is_k ? a.kos : a.qos;
  in += b * si[0] + i * si[1] + h0 * si[2];
  out += b * so[0] + i * so[1] + h0 * so[2];
  const int32_t* pos = a.pos + b * a.pos_batch + (int64_t)i * a.axes;

  if constexpr (HALF) {
    const int turning = a.pairs / W;               // lanes that turn pairs
    if (lane < turning) {
      const int p0 = lane * W;
      Vec u[U], v[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (h0 + k < heads) {
          u[k] = *reinterpret_cast<const Vec*>(in + k * si[2] + p0);
          v[k] = *reinterpret_cast<const Vec*>(in + k * si[2] + p0 + a.pairs);
        }
      float c[W], s[W];
#pragma unroll
      for (int j = 0; j < W; ++j) turn(a, pos, p0 + j, c[j], s[j]);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (h0 + k < heads) {
#pragma unroll
          for (int j = 0; j < W; ++j) {
            const float x = to_f32(u[k].e[j]), y = to_f32(v[k].e[j]);
            u[k].e[j] = from_f32<T>(x * c[j] - y * s[j]);
            v[k].e[j] = from_f32<T>(x * s[j] + y * c[j]);
          }
          *reinterpret_cast<Vec*>(out + k * so[2] + p0) = u[k];
          *reinterpret_cast<Vec*>(out + k * so[2] + p0 + a.pairs) = v[k];
        }
    } else if (a.copy) {
      const int e0 = 2 * a.pairs + (lane - turning) * W;
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (h0 + k < heads)
          *reinterpret_cast<Vec*>(out + k * so[2] + e0) =
              *reinterpret_cast<const Vec*>(in + k * si[2] + e0);
    }
  } else {
    const int p0 = lane * (W / 2);
    if (p0 >= a.pairs && !a.copy) return;
    Vec u[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (h0 + k < heads) u[k] = *reinterpret_cast<const Vec*>(in + k * si[2] + 2 * p0);
    float c[W / 2], s[W / 2];
#pragma unroll
    for (int j = 0; j < W / 2; ++j)
      if (p0 + j < a.pairs) turn(a, pos, p0 + j, c[j], s[j]);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (h0 + k < heads) {
#pragma unroll
        for (int j = 0; j < W / 2; ++j)
          if (p0 + j < a.pairs) {
            const float x = to_f32(u[k].e[2 * j]), y = to_f32(u[k].e[2 * j + 1]);
            u[k].e[2 * j] = from_f32<T>(x * c[j] - y * s[j]);
            u[k].e[2 * j + 1] = from_f32<T>(x * s[j] + y * c[j]);
          }
        *reinterpret_cast<Vec*>(out + k * so[2] + 2 * p0) = u[k];
      }
  }
}

// Any head dim, stride and alignment: a thread turns one pair or copies one
// element of one head.
template <typename T>
__global__ void __launch_bounds__(256) rope_any_kernel(Rope a) {
  const int64_t per_head = a.pairs + (a.d - 2 * a.pairs);
  const int64_t per_token = (int64_t)(a.H + a.Hk) * per_head;
  const int64_t total = (int64_t)a.B * a.n * per_token;
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < total;
       x += (int64_t)gridDim.x * blockDim.x) {
    const int64_t token = x / per_token;
    const int rest = (int)(x % per_token);
    int h = rest / (int)per_head;
    const int p = rest % (int)per_head;
    const int64_t b = token / a.n, i = token % a.n;
    const bool is_k = h >= a.H;
    if (is_k) h -= a.H;
    const int64_t* si = is_k ? a.ks : a.qs;
    const int64_t* so = is_k ? a.kos : a.qos;
    const T* in = static_cast<const T*>(is_k ? a.k : a.q) + b * si[0] + i * si[1] + h * si[2];
    T* out = static_cast<T*>(is_k ? a.k_out : a.q_out) + b * so[0] + i * so[1] + h * so[2];
    if (p >= a.pairs) {
      const int e = a.pairs + p;
      if (a.copy) out[e] = in[e];
      continue;
    }
    const int e0 = a.half ? p : 2 * p, e1 = a.half ? p + a.pairs : 2 * p + 1;
    float c, s;
    turn(a, a.pos + b * a.pos_batch + i * a.axes, p, c, s);
    const float u = to_f32(in[e0]), v = to_f32(in[e1]);
    out[e0] = from_f32<T>(u * c - v * s);
    out[e1] = from_f32<T>(u * s + v * c);
  }
}

template <typename T, int U>
void rope_launch(Rope a, cudaStream_t st) {
  a.q_units = (a.H + U - 1) / U;
  a.k_units = (a.Hk + U - 1) / U;
  a.units = (int64_t)a.B * a.n * (a.q_units + a.k_units);
  constexpr int W = 16 / sizeof(T);
  a.lanes = a.half ? a.pairs / W + (a.d - 2 * a.pairs) / W : a.d / W;
  const int here = 256 / a.lanes;
  const unsigned g = (unsigned)((a.units + here - 1) / here);
  if (a.half)
    rope_kernel<T, U, true><<<g, 256, 0, st>>>(a);
  else
    rope_kernel<T, U, false><<<g, 256, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_rope(int dtype, const Rope& a, cudaStream_t st) {
  if (a.B == 0 || a.n == 0) return cudaSuccess;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    constexpr int W = 16 / sizeof(T);
    bool vec = a.d % W == 0 && a.d / W <= 256 && (!a.half || a.pairs % W == 0) &&
               (int64_t)a.B * a.n * (a.H + a.Hk) < (int64_t)1 << 31;
    for (int i = 0; i < 3; ++i)
      vec = vec && a.qs[i] % W == 0 && a.qos[i] % W == 0 &&
            (!a.Hk || (a.ks[i] % W == 0 && a.kos[i] % W == 0));
    vec = vec && aligned_to(a.q, 16) && aligned_to(a.q_out, 16) && aligned_to(a.k, 16) &&
          aligned_to(a.k_out, 16);
    if (!vec) {
      const int64_t total = (int64_t)a.B * a.n * (a.H + a.Hk) * (a.d - a.pairs);
      const int64_t blocks = (total + 255) / 256;
      rope_any_kernel<T><<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, st>>>(a);
    } else if ((int64_t)a.B * a.n * (a.H + a.Hk) >= 152 * 128) {
      rope_launch<T, 4>(a, st);
    } else {
      rope_launch<T, 1>(a, st);
    }
    return cudaGetLastError();
  });
}

}  // namespace bl
