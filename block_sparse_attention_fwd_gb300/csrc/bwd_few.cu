// The attention's backward from 8 bits for up to kFewTokens tokens, where the
// whole attention of a head is one tile: one launch.
//
//   P = exp(s Q K^T - LSE),  dP = dO V^T,  dS = P (dP - D),  D = rowsum(dO o O)
//   dV = P^T dO,  dK = s dS^T Q,  dQ = s dS K     (dK, dV summed over the group)
//
// At these lengths the tcgen05 path is bound by its launches (expansion, D pass,
// items, sums, dQ) and its seven tensor maps, and it rounds P and dS to bf16 for
// the tensor cores, an error that sums over few tokens do not average out (one
// token: 2^-8 at most of all of G_V).  Here the codes are read as they are, no
// workspace is needed but the status word, and P and dS enter their products as
// two bf16 parts each, P = hi + lo within 2^-16 of P.
//
// A block has 16 rows of one kind ("mine") and walks tiles of 16 rows of the
// other.  A key item (batch, kv head, 16 keys) goes over the group's heads and
// their queries and forms dK or dV, a query item (batch, head, 16 queries) over
// the keys and forms dQ.  S is formed three times for it and dP twice, but no sum
// crosses blocks, and a thread has one result's sums (dK and dV together: 242
// registers, 8 warps an SM).  All kinds are the same products,
//   S = A1 B1^T, dP = A2 B2^T, and acc += dS B1 (dQ, dK) or acc += P B2 (dV),
// with (A1, A2) = (K, V) and (B1, B2) = (Q, dO) or the other way round.  A warp takes every fourth tile by itself (no barriers) on
// mma.sync.m16n8k16, whose 16 rows fit where the 64 or 128 rows of a tcgen05
// instruction would stay empty: the accumulators of S are, in place, the A
// operand of the next product.  The warps' sums are added in their order at the
// end, so results do not vary.
//
// Measured (device time; the tcgen05 path at 65 tokens beside it), d = 128: 8/2
// heads causal, 1 token 4.1, 16 tokens 4.8, 64 tokens 13.0 us (19.2); 16 x 32/8
// heads causal, 64 tokens 44 us (57).  Bound by latency: loads, one tile's chain
// of products, the sums (0.44 instructions a cycle and scheduler, DRAM 5% busy).
// dK and dV in one item took 14.6 and 52 us; the same split on fp32
// multiply-adds, bound by its reads of shared memory, 49 and 174 us.  Beyond 64 tokens the
// pairs grow with n^2 and the tcgen05 path's one tile of 128 does not.
#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "tc.cuh"

namespace bl {

namespace {

constexpr int kRows = 16, kWarps = 4;

// 16 elements of a row of a tile's two tensors: k and v, or q and dO with what
// belongs to the query (o, LSE).
struct Part {
  uint4 x, y[2], o[2];
  float xs, ys, os, lse;
};

// Four 8 x 8 matrices whose rows the lanes point at.
__device__ __forceinline__ void ldm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values as bf16, and what that leaves of them as bf16.
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x, y);
  lo = pack_bf16(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
}

template <int D>
struct Smem {
  static constexpr int PITCH = D + 8;            // bf16; rows start 4 banks apart
  typedef __nv_bfloat16 Tile[kRows][PITCH];
  alignas(16) Tile a[2];
  // a warp's tiles, and then its fp32 sums of one result
  union alignas(16) {
    Tile b[2];
    float sum[kRows][D + 4];
  } w[kWarps];
  // LSE and D of the warps' queries; [kWarps]: of the block's own
  float lse[kWarps + 1][kRows], dd[kWarps + 1][kRows];
};

enum Kind { kDQ, kDK, kDV };

template <int D, int FMT, Kind KIND>
__device__ __forceinline__ void few_item(const BwdFew& a, Smem<D>& sm, int item, int tiles) {
  constexpr int LANES = D / 16;                  // of a row when loading
  constexpr int ROWS = 32 / LANES;               // of a warp's pass
  constexpr int PASSES = kRows / ROWS;
  constexpr int NT = D / 8;                      // 8-column tiles of a result
  constexpr bool KEYS = KIND != kDQ, DS = KIND != kDV;     // DS: needs dS
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.H / a.Hk, heads = KEYS ? a.Hk : a.H;
  const int mine = item % tiles, head = item / tiles % heads, b = item / tiles / heads;
  const int m0 = mine * kRows;
  const int hk = KEYS ? head : head / G;

  const int c16 = lane % LANES * 16;
  auto load_kv = [&](int r, Part& p) {
    p = Part{};
    if (r >= a.n) return;
    const int64_t at = ((int64_t)b * a.n + r) * a.Hk + hk;
    p.x = *reinterpret_cast<const uint4*>(a.k + at * D + c16);
    p.xs = a.k_scales[at];
    if (!DS) return;
    p.y[0] = *reinterpret_cast<const uint4*>(a.v + at * D + c16);
    p.ys = a.v_scales[at];
  };
  auto load_q = [&](int hq, int r, Part& p) {
    p = Part{};
    if (r >= a.n) return;
    const int64_t at = ((int64_t)b * a.n + r) * a.H + hq;
    p.x = *reinterpret_cast<const uint4*>(a.q + at * D + c16);
    p.xs = a.q_scales[at];
    const uint4* g = reinterpret_cast<const uint4*>(a.g_o + at * D + c16);
    p.y[0] = g[0];
    p.y[1] = g[1];
    p.lse = a.lse[((int64_t)b * a.H + hq) * a.n + r];
    if (!DS) return;
    if (a.o) {
      const uint4* o = reinterpret_cast<const uint4*>(a.o + at * D + c16);
      p.o[0] = o[0];
      p.o[1] = o[1];
    } else {
      p.o[0] = *reinterpret_cast<const uint4*>(a.o_codes + at * D + c16);
      p.os = a.o_scales[at];
    }
  };
  // 16 values of a checkpoint: they stand for bf16
  auto put_codes = [&](__nv_bfloat16* dst, const uint4& c, float scale) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      float f[8];
      decode8<FMT>(Codes{{w[2 * v], w[2 * v + 1]}}, f);
      reinterpret_cast<uint4*>(dst)[v] =
          make_uint4(pack_bf16(f[0] * scale, f[1] * scale), pack_bf16(f[2] * scale, f[3] * scale),
                     pack_bf16(f[4] * scale, f[5] * scale), pack_bf16(f[6] * scale, f[7] * scale));
    }
  };
  auto put_kv = [&](typename Smem<D>::Tile (&to)[2], int row, const Part& p) {
    put_codes(&to[0][row][c16], p.x, p.xs);
    if (DS) put_codes(&to[1][row][c16], p.y[0], p.ys);
  };
  auto put_q = [&](typename Smem<D>::Tile (&to)[2], int row, const Part& p, int slot) {
    put_codes(&to[0][row][c16], p.x, p.xs);
    float dot = 0.f;
    const uint32_t oc[4] = {p.o[0].x, p.o[0].y, p.o[0].z, p.o[0].w};
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      reinterpret_cast<uint4*>(&to[1][row][c16])[v] = p.y[v];
      if (!DS) continue;
      const uint32_t gw[4] = {p.y[v].x, p.y[v].y, p.y[v].z, p.y[v].w};
      const uint32_t ow[4] = {p.o[v].x, p.o[v].y, p.o[v].z, p.o[v].w};
      float o[8];
      if (a.o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[2 * i] = __uint_as_float(ow[i] << 16);
          o[2 * i + 1] = __uint_as_float(ow[i] & 0xffff0000u);
        }
      } else {
        decode8<FMT>(Codes{{oc[2 * v], oc[2 * v + 1]}}, o);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dot = fmaf(__uint_as_float(gw[i] << 16), o[2 * i], dot);
        dot = fmaf(__uint_as_float(gw[i] & 0xffff0000u), o[2 * i + 1], dot);
      }
    }
    if (DS) dot = lanes_sum(dot, LANES);
    if (c16 == 0) {
      sm.dd[slot][row] = a.o ? dot : dot * p.os;
      sm.lse[slot][row] = p.lse;
    }
  };

  if (warp < PASSES) {                                     // the block's own rows, a pass a warp
    const int row = warp * ROWS + lane / LANES;
    Part p;
    if (KEYS) {
      load_kv(m0 + row, p);
      put_kv(sm.a, row, p);
    } else {
      load_q(head, m0 + row, p);
      put_q(sm.a, row, p, kWarps);
    }
  }
  __syncthreads();

  // the tiles of the other kind that any pair of the item can be in
  int first = 0, last = tiles - 1;
  if (a.causal) (KEYS ? first : last) = mine;
  if (a.window) {
    if (KEYS) last = min(last, (int)(((int64_t)m0 + kRows - 1 + a.window - 1) / kRows));
    else first = max(0, m0 - a.window + 1) / kRows;
  }
  const int per_head = last - first + 1, units = KEYS ? per_head * G : per_head;

  auto& B = sm.w[warp].b;
  const uint32_t sA = (uint32_t)__cvta_generic_to_shared(&sm.a[0][0][0]);
  const uint32_t sB = (uint32_t)__cvta_generic_to_shared(&B[0][0][0]);
  constexpr uint32_t ROW = Smem<D>::PITCH * 2, TILE = kRows * ROW;      // bytes
  // rows that a lane points at: of A (and of B as [k][n], transposed), of B as [n][k]
  const uint32_t at_a = (lane & 15) * ROW + (lane >> 4) * 16;
  const uint32_t at_b = ((lane & 7) + (lane >> 4) * 8) * ROW + (lane >> 3 & 1) * 16;
  float acc[NT][4] = {};
  const int g4 = lane >> 2, t4 = lane & 3;
  for (int u = warp; u < units; u += kWarps) {
    const int h = KEYS ? head * G + u / per_head : head, o0 = (first + u % per_head) * kRows;
    const int64_t bh = (int64_t)b * a.H + h;
    // whether the list of the head keeps its one tile
    if (a.q_cnt && !(a.q_cnt[bh] == 1 && a.q_idx[bh] == 0)) continue;
    __syncwarp();                                          // the last tile has been read
#pragma unroll
    for (int p0 = 0; p0 < PASSES; p0 += 2) {
      Part p[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = o0 + (p0 + i) * ROWS + lane / LANES;
        if (KEYS) load_q(h, r, p[i]); else load_kv(r, p[i]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = (p0 + i) * ROWS + lane / LANES;
        if (KEYS) put_q(B, row, p[i], warp); else put_kv(B, row, p[i]);
      }
    }
    __syncwarp();
    float s[2][4] = {}, dp[2][4] = {};                     // S and dP of columns 0-7, 8-15
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t fa[4], fb[4];
      ldm(fa, sA + at_a + k * 32);
      ldm(fb, sB + at_b + k * 32);
      mma16(s[0], fa, fb[0], fb[1]);
      mma16(s[1], fa, fb[2], fb[3]);
      if constexpr (DS) {
        ldm(fa, sA + TILE + at_a + k * 32);
        ldm(fb, sB + TILE + at_b + k * 32);
        mma16(dp[0], fa, fb[0], fb[1]);
        mma16(dp[1], fa, fb[2], fb[3]);
      }
    }
    // P or dS, in two parts, where the next product takes them
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float e[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int m = g4 + 8 * r, o = 8 * t + 2 * t4 + j, c = 2 * r + j;
          const int key = KEYS ? m0 + m : o0 + o, query = KEYS ? o0 + o : m0 + m;
          const int slot = KEYS ? warp : kWarps, ql = KEYS ? o : m;
          const bool on = key < a.n && query < a.n && (!a.causal || query >= key) &&
                          (!a.window || query - key < a.window);
          e[j] = on ? exp2f(fmaf(s[t][c], a.scale * kLog2e, -(sm.lse[slot][ql] * kLog2e))) : 0.f;
          if (DS) e[j] = on ? e[j] * (dp[t][c] - sm.dd[slot][ql]) : 0.f;
        }
        split(e[0], e[1], hi[2 * t + r], lo[2 * t + r]);
      }
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      uint32_t fb[4];
      ldm_t(fb, sB + (DS ? 0 : TILE) + at_a + x * 32);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        mma16(acc[2 * x + t], hi, fb[2 * t], fb[2 * t + 1]);
        mma16(acc[2 * x + t], lo, fb[2 * t], fb[2 * t + 1]);
      }
    }
  }

  // the warps' sums, added in their order
  __nv_bfloat16* to = KIND == kDQ ? a.g_q : KIND == kDK ? a.g_k : a.g_v;
  const float by = DS ? a.scale : 1.f;
  __syncwarp();                                            // the warp's tiles have been read
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      *reinterpret_cast<float2*>(&sm.w[warp].sum[g4 + 8 * r][8 * x + 2 * t4]) =
          make_float2(acc[x][2 * r], acc[x][2 * r + 1]);
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * D / 4; i += kWarps * 32) {
    const int row = i / (D / 4), c = i % (D / 4) * 4, r = m0 + row;
    if (r >= a.n) continue;
    float4 f = *reinterpret_cast<const float4*>(&sm.w[0].sum[row][c]);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 g = *reinterpret_cast<const float4*>(&sm.w[w].sum[row][c]);
      f.x += g.x;
      f.y += g.y;
      f.z += g.z;
      f.w += g.w;
    }
    *reinterpret_cast<uint2*>(to + (((int64_t)b * a.n + r) * heads + head) * D + c) =
        make_uint2(pack_bf16(f.x * by, f.y * by), pack_bf16(f.z * by, f.w * by));
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32, 4) bwd_few_kernel(BwdFew a) {
  __shared__ Smem<D> sm;
  if (blockIdx.x == 0) {
    bool bad = false;
    if (a.q_cnt)
      for (int64_t x = threadIdx.x; x < (int64_t)a.B * a.H; x += kWarps * 32) {
        const int c = a.q_cnt[x];
        bad = bad || c < 0 || c > 1 || (c == 1 && a.q_idx[x] != 0);
      }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      a.status[0] = bad ? tc::kStatusCorrupt : 0;
      a.status[1] = 0;
    }
  }
  const int tiles = (a.n + kRows - 1) / kRows;
  const int key_items = a.B * a.Hk * tiles, item = (int)blockIdx.x;
  if (item < key_items)
    few_item<D, FMT, kDK>(a, sm, item, tiles);
  else if (item < 2 * key_items)
    few_item<D, FMT, kDV>(a, sm, item - key_items, tiles);
  else
    few_item<D, FMT, kDQ>(a, sm, item - 2 * key_items, tiles);
}

}  // namespace

cudaError_t launch_bwd_few(int d, int fmt, const BwdFew& a, cudaStream_t st) {
  const int tiles = (a.n + kRows - 1) / kRows;
  const int64_t items = (int64_t)a.B * (2 * (int64_t)a.Hk + a.H) * tiles;
  if (items > INT32_MAX) return cudaErrorNotSupported;
  const unsigned g = (unsigned)items;
  if (d == 64)
    fmt == kFmtInt8 ? bwd_few_kernel<64, kFmtInt8><<<g, kWarps * 32, 0, st>>>(a)
                    : bwd_few_kernel<64, kFmtE4m3><<<g, kWarps * 32, 0, st>>>(a);
  else
    fmt == kFmtInt8 ? bwd_few_kernel<128, kFmtInt8><<<g, kWarps * 32, 0, st>>>(a)
                    : bwd_few_kernel<128, kFmtE4m3><<<g, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace bl
