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
// fp64, whose rate here is low, and without a table to read.  Its upper two
// bits, rounded, are the quadrant; the rest, |x| <= pi / 4, goes through the
// Taylor series of sine and cosine (to x^9 and x^8: the next terms are below
// 2^-25), within 1.7 * 2^-24 of the exact values; the general sincospi took the
// largest share of a pass over single heads (44 -> 36 us at 100000 tokens).
//
// The pass is bound by HBM: q and k once in, once out.  A block takes a tile of
// tokens.  It forms the tile's sines and cosines once, in shared memory, and
// then goes over the (token, head) units of the tile, 256 / lanes of them at a
// time, a group of lanes with 16-byte vectors on each; a thread has the vectors
// of U units in flight, the first of them from before the sines are formed.
// Measured: 40 + 40 heads of 128 at 32760 tokens in 208 us, 6.5 TB/s
// (interleaved), and 196 us, 6.8 TB/s (halves); each thread forming the sines of
// its own vectors took 328 and 244 us.
#include "kernels.h"
#include "rows.cuh"

namespace bl {

namespace {

// (cos, sin) of an angle in 2^-32 turns.
__device__ __forceinline__ float2 cos_sin(uint32_t angle) {
  const uint32_t quadrant = (angle + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(angle - (quadrant << 30)) * 1.46291807926716e-9f;   // 2 pi / 2^32
  const float x2 = x * x;
  float s = fmaf(x2, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(s, x2, 1.f / 120.f);
  s = fmaf(s, x2, -1.f / 6.f);
  s = fmaf(s * x2, x, x);
  float c = fmaf(x2, 1.f / 40320.f, -1.f / 720.f);
  c = fmaf(c, x2, 1.f / 24.f);
  c = fmaf(c, x2, -0.5f);
  c = fmaf(c, x2, 1.f);
  // a quarter turn takes (c, s) to (-s, c)
  const float a = quadrant & 1 ? s : c, b = quadrant & 1 ? c : s;
  return make_float2((quadrant + 1) & 2 ? -a : a, quadrant & 2 ? -b : b);
}

__device__ __forceinline__ int axis_of(const Rope& a, int p) {
  int axis = 0;
#pragma unroll
  for (int e = 0; e < 3; ++e) axis += p >= a.ends[e] ? 1 : 0;
  return axis;
}
// The angle at a position of a pair with frequency f, in 2^-32 turns.
__device__ __forceinline__ uint32_t angle_of(const Rope& a, const int32_t* pos, uint64_t f) {
  const uint32_t hi = (uint32_t)(((uint64_t)(int64_t)__ldg(pos) * f) >> 32);
  return a.inverse ? 0u - hi : hi;
}

template <typename T, int U, bool HALF>
__global__ void __launch_bounds__(256, 4) rope_kernel(Rope a) {
  constexpr int W = 16 / sizeof(T);
  constexpr int NV = HALF ? 2 : 1;                   // vectors of a unit a thread holds
  constexpr int NP = HALF ? W : W / 2;               // pairs in them
  struct alignas(16) Vec { T e[W]; };
  // (cos, sin) of the tile's tokens.  The pairs of a token lie in planes of two
  // pairs a lane, so that neighbouring lanes read neighbouring 16 bytes.
  extern __shared__ float4 table[];
  const int lanes = a.lanes, step = 256 / lanes;
  const int g = threadIdx.x / lanes, lane = threadIdx.x - g * lanes;
  const int per_token = a.H + a.Hk;
  const int64_t tok0 = (int64_t)blockIdx.x * a.tile;
  const int toks = (int)min((int64_t)a.tile, (int64_t)a.B * a.n - tok0);
  const int holders = (a.pairs + NP - 1) / NP;       // lanes that hold pairs
  const int planes = NP / 2;
  const int p0 = lane * NP;
  const bool turns = lane < holders;
  const bool works = g < step && (turns || a.copy);
  // the thread's elements of a head: HALF has two vectors, of the halves of its
  // pairs or next to each other behind them (the last may lack its second)
  const int e0 = HALF ? (turns ? p0 : 2 * a.pairs + (lane - holders) * 2 * W) : 2 * p0;
  const int second = turns ? a.pairs : W;
  const bool two = HALF && (turns || e0 + W < a.d);

  int tok = g / per_token, head = g - tok * per_token;      // the next unit's
  const int tok_step = step / per_token, head_step = step - tok_step * per_token;
  Vec v[U][NV];
  T* dst[U];
  int at[U];                                          // token of the tile, or -1
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = works && tok < toks ? tok : -1;
      if (at[u] >= 0) {
        const uint32_t t = (uint32_t)tok0 + tok;
        const bool is_k = head >= a.H;
        const int h = is_k ? head - a.H : head;
        const int64_t* si = is_k ? a.ks : a.qs;
        const int64_t* so = is_k ? a.kos : a.qos;
        const T* src = static_cast<const T*>(is_k ? a.k : a.q) + e0 + (int64_t)h * (int)si[2];
        dst[u] = static_cast<T*>(is_k ? a.k_out : a.q_out) + e0 + (int64_t)h * (int)so[2];
        if (a.flat) {                                 // the batches follow one another
          src += (int64_t)t * (int)si[1];
          dst[u] += (int64_t)t * (int)so[1];
        } else {
          const uint32_t b = t / (uint32_t)a.n, i = t - b * (uint32_t)a.n;
          src += b * si[0] + i * si[1];
          dst[u] += b * so[0] + i * so[1];
        }
        v[u][0] = *reinterpret_cast<const Vec*>(src);
        if constexpr (HALF)
          if (two) v[u][1] = *reinterpret_cast<const Vec*>(src + second);
      }
      tok += tok_step;
      head += head_step;
      if (head >= per_token) {
        head -= per_token;
        ++tok;
      }
    }
  };

  load();
  {
    // A thread keeps its place in a token's part of the table, so its pair, and
    // goes over the tokens `apart` at a time.
    const int places = planes * holders * 2;
    const int apart = places < 256 ? 256 / places : 1;
    const int t0 = threadIdx.x / places;
    for (int x = threadIdx.x - t0 * places; x < places && t0 < apart; x += 256) {
      const int plane = x / (2 * holders), rest = x - plane * 2 * holders;
      const int p = (rest >> 1) * NP + 2 * plane + (rest & 1);
      if (p >= a.pairs) continue;
      const uint64_t f = a.freqs[p];
      const int32_t* pos = a.pos + axis_of(a, p);
      float2* place = reinterpret_cast<float2*>(table) + x;
#pragma unroll 4
      for (int t = t0; t < toks; t += apart) {
        const uint32_t token = (uint32_t)tok0 + t;
        const uint32_t i = a.pos_flat ? token : token % (uint32_t)a.n;
        place[t * places] = cos_sin(angle_of(a, pos + (int64_t)i * a.axes, f));
      }
    }
  }
  __syncthreads();
  while (at[0] >= 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      if (turns) {
        const float4* cs = table + at[u] * planes * holders + lane;
#pragma unroll
        for (int j = 0; j < planes; ++j) {
          const float4 c = cs[j * holders];
          if constexpr (HALF) {
            const float x0 = to_f32(v[u][0].e[2 * j]), x1 = to_f32(v[u][0].e[2 * j + 1]);
            const float y0 = to_f32(v[u][1].e[2 * j]), y1 = to_f32(v[u][1].e[2 * j + 1]);
            reinterpret_cast<Pair<T>*>(&v[u][0])[j] =
                Pair<T>(x0 * c.x - y0 * c.y, x1 * c.z - y1 * c.w);
            reinterpret_cast<Pair<T>*>(&v[u][1])[j] =
                Pair<T>(x0 * c.y + y0 * c.x, x1 * c.w + y1 * c.z);
          } else {
            // the last vector may pass the last pair
            if (p0 + 2 * j < a.pairs) {
              const float x = to_f32(v[u][0].e[4 * j]), y = to_f32(v[u][0].e[4 * j + 1]);
              reinterpret_cast<Pair<T>*>(&v[u][0])[2 * j] =
                  Pair<T>(x * c.x - y * c.y, x * c.y + y * c.x);
            }
            if (p0 + 2 * j + 1 < a.pairs) {
              const float x = to_f32(v[u][0].e[4 * j + 2]), y = to_f32(v[u][0].e[4 * j + 3]);
              reinterpret_cast<Pair<T>*>(&v[u][0])[2 * j + 1] =
                  Pair<T>(x * c.z - y * c.w, x * c.w + y * c.z);
            }
          }
        }
      }
      *reinterpret_cast<Vec*>(dst[u]) = v[u][0];
      if constexpr (HALF)
        if (two) *reinterpret_cast<Vec*>(dst[u] + second) = v[u][1];
    }
    load();
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
    const float2 cs = 
        cos_sin(angle_of(a, a.pos + b * a.pos_batch + i * a.axes + axis_of(a, p), a.freqs[p]));
    const float c = cs.x, s = cs.y;
    const float u = to_f32(in[e0]), v = to_f32(in[e1]);
    out[e0] = from_f32<T>(u * c - v * s);
    out[e1] = from_f32<T>(u * s + v * c);
  }
}

// Tokens of a block's tile: four batches of U units for every thread, as far as
// there are tokens for four blocks an SM.  Half as many units cost 8% at 40 + 40
// heads of 128 (interleaved: 225 against 207 us), twice as many gain nothing.
int tile_tokens(int64_t tokens, int heads, int groups, int U) {
  int64_t tile = (4 * U * groups + heads - 1) / heads;
  if (tile > 128) tile = 128;
  const int64_t fill = tokens / (4 * 152);
  if (tile > fill) tile = fill;
  return tile < 1 ? 1 : (int)tile;
}

template <typename T, bool HALF>
cudaError_t rope_launch(Rope a, cudaStream_t st) {
  constexpr int W = 16 / sizeof(T);
  a.lanes = HALF ? a.pairs / W + ((a.d - 2 * a.pairs) / W + 1) / 2 : a.d / W;
  const int64_t tokens = (int64_t)a.B * a.n;
  a.flat = true;
  for (const int64_t* st : {a.qs, a.qos, a.ks, a.kos})
    a.flat = a.flat && (a.B == 1 || st[0] == (int64_t)a.n * st[1]);
  a.pos_flat = a.B == 1 || a.pos_batch != 0;
  constexpr int U = HALF ? 2 : 4;
  a.tile = tile_tokens(tokens, a.H + a.Hk, 256 / a.lanes, U);
  // the table of a tile stays within 32 KB
  constexpr int NP = HALF ? W : W / 2;
  const int padded = (a.pairs + NP - 1) / NP * NP;
  while (a.tile > 1 && (int64_t)a.tile * padded * 8 > 32768) a.tile /= 2;
  const size_t smem = (size_t)a.tile * padded * 8;
  const unsigned g = (unsigned)((tokens + a.tile - 1) / a.tile);
  rope_kernel<T, U, HALF><<<g, 256, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int dtype, const Rope& a, cudaStream_t st) {
  if (a.B == 0 || a.n == 0) return cudaSuccess;
  return with_type(dtype, [&](auto* z) {
    using T = std::remove_pointer_t<decltype(z)>;
    constexpr int W = 16 / sizeof(T);
    bool vec = a.d % W == 0 && a.d / W <= 256 && (!a.half || a.pairs % W == 0) &&
               (int64_t)a.B * a.n < (int64_t)1 << 31;
    for (int i = 0; i < 3; ++i)
      for (const int64_t* st : {a.qs, a.qos, a.ks, a.kos})
        vec = vec && st[i] % W == 0 && (i == 0 || st[i] < (int64_t)1 << 31);
    vec = vec && aligned_to(a.q, 16) && aligned_to(a.q_out, 16) && aligned_to(a.k, 16) &&
          aligned_to(a.k_out, 16);
    if (!vec) {
      const int64_t total = (int64_t)a.B * a.n * (a.H + a.Hk) * (a.d - a.pairs);
      const int64_t blocks = (total + 255) / 256;
      rope_any_kernel<T><<<(unsigned)(blocks < 152 * 64 ? blocks : 152 * 64), 256, 0, st>>>(a);
      return cudaGetLastError();
    }
    return a.half ? rope_launch<T, true>(a, st) : rope_launch<T, false>(a, st);
  });
}

}  // namespace bl
