// Products of e4m3 codes with a scale for each block of 128 of the summed dim:
//
//   out[i, j] = sum over blocks b of sa(i, b) sb(j, b) * sum over k in b of A[i, k] B[j, k]
//
// The inner sums run on the tensor cores (tcgen05.mma kind::f8f6f4, fp32 in TMEM), one
// block of 128 at a time; the outer sum in fp32 registers, where the scales come in, so
// nothing is rounded to fewer than 32 bits before the result.
//
// A CTA has a tile of 128 x BN.  Warp roles:
//   warp 0      TMA producer: codes of A and B, 128 of the summed dim a stage.
//   warp 1      MMA issuer (one thread), TMEM owner: a block's product into one of NB
//               accumulators.
//   warps 2, 3  scales of the tile's rows and columns into a ring of shared memory.
//   warps 4-    accumulate: a thread has a row of up to 128 columns of the tile in
//               registers, reads the block's product from TMEM and adds it, scaled.
// Either operand may have the summed dim contiguous (K-major) or the other one
// (MN-major): the tiles in shared memory are alike, 128 rows of 128 bytes, and only
// the descriptors differ, so no operand is ever transposed in memory.
// Every mbarrier wait is bounded (tc.cuh); a tile that was given up is written as NaN.
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "tc.cuh"

namespace bl {

namespace {

using namespace tc;

constexpr int kSMs = 152;

template <int BN>
struct GCfg {
  static constexpr int NB = BN <= 64 ? 4 : 2;           // accumulators in TMEM
  static constexpr int COLS = NB * BN < 32 ? 32 : NB * BN;
  static constexpr int EPI = BN == 256 ? 8 : 4;         // accumulating warps
  static constexpr int THREADS = 128 + EPI * 32;
  static constexpr int CTAS = BN == 256 ? 1 : 2;        // on an SM
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : BN == 128 ? 3 : BN == 64 ? 4 : 5;
  static constexpr int NSC = 8;                         // stages of scales
  static constexpr int SC_FLOATS = 128 + BN;
  static constexpr int SMEM = NS * STAGE + NSC * SC_FLOATS * 4 + 1024;
  static constexpr int PER = BN / (EPI / 4);            // columns of a thread
};

template <int BN>
struct GBars {
  using C = GCfg<BN>;
  uint64_t full[C::NS], empty[C::NS], t_full[C::NB], t_empty[C::NB], s_full[C::NSC],
      s_empty[C::NSC];
};

// kind::f8f6f4 with e4m3 A and B (formats 0), fp32 accumulate, M = 128.
__device__ __forceinline__ uint32_t idesc_e4m3(int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier once this thread's copies so far are there (the barrier's
// count has the arrival already).
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" :::
                   "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, int rank) {
  uint32_t v;
  asm volatile(
      "{\n .reg .u32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n"
      " ld.shared::cluster.u32 %0, [a];\n}\n"
      : "=r"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// Tiles in groups of kGroup along i, j by j: a group's rows of A stay in L2 while B
// passes by.
constexpr int kGroup = 16;
__device__ __forceinline__ void tile_at(int t, int ti, int tj, int& i, int& j) {
  const int per = kGroup * tj, g = t / per, r = t - g * per;
  const int h = min(kGroup, ti - g * kGroup);
  j = r / h;
  i = g * kGroup + (r - j * h);
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, const uint64_t* acc, int n, bool wide) {
  if (wide && n >= 16) {
    float f[2][8];
#pragma unroll
    for (int c = 0; c < 8; ++c) f2_unpack(acc[c], f[c / 4][2 * (c % 4)], f[c / 4][2 * (c % 4) + 1]);
    store16<T, true>(p, f);
  } else {
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      float lo, hi;
      f2_unpack(acc[c / 2], lo, hi);
      if (c < n) p[c] = from_f32<T>(c % 2 ? hi : lo);
    }
  }
}

// COL: every column has a scale of its own; else every 128 share one.
template <int BN, bool COL, typename T>
__global__ void __launch_bounds__(GCfg<BN>::THREADS, GCfg<BN>::CTAS)
    gemm8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 Gemm8 g, uint64_t wait_ns) {
  using C = GCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  float* sc = reinterpret_cast<float*>(sm + C::NS * C::STAGE);
  __shared__ __align__(8) GBars<BN> bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail, s_loads;
  __shared__ uint64_t s_wait;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ti = (g.m + 127) / 128, tj = (g.n + BN - 1) / BN, tiles = ti * tj;
  const int nkb = (g.k + 127) / 128;
  // with splits, a cluster shares a tile: each CTA has a part of the summed dim
  const int rank = BN <= 128 ? blockIdx.x % g.splits : 0;
  const int first = BN <= 128 ? blockIdx.x / g.splits : blockIdx.x;
  const int step = BN <= 128 ? gridDim.x / g.splits : gridDim.x;
  const int kb0 = BN <= 128 ? (int)((int64_t)nkb * rank / g.splits) : 0;
  const int kb1 = BN <= 128 ? (int)((int64_t)nkb * (rank + 1) / g.splits) : nkb;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&bars.full[s], 1);
      mbar_init(&bars.empty[s], 1);
    }
    for (int s = 0; s < C::NB; ++s) {
      mbar_init(&bars.t_full[s], 1);
      mbar_init(&bars.t_empty[s], C::EPI);
    }
    for (int s = 0; s < C::NSC; ++s) {
      mbar_init(&bars.s_full[s], 64);
      mbar_init(&bars.s_empty[s], C::EPI);
    }
    s_fail = 0;
    s_loads = 0;
    s_wait = wait_ns;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&s_tmem, C::COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, int use, int ring) {   // for the phase of use `use` of a slot
    return mbar_wait_limited(bar, (use / ring) & 1, &s_wait);
  };
  auto failed = [&]() { return *(volatile int*)&s_fail != 0; };
  auto fail = [&]() { atomicOr(&s_fail, 1); };

  // the accumulating warps need registers, the others few; the shares add up to the
  // launch's (384 x 168, 256 x 128)
  if (warp < 4) {
  if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  if constexpr (BN == 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tm_a);
      prefetch_tmap(&tm_b);
      int it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        int i, j;
        tile_at(t, ti, tj, i, j);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::NS;
          ok = !failed() && (it < C::NS || wait(&bars.empty[s], it - C::NS, C::NS));
          if (!ok) break;
          uint8_t* a = sm + s * C::STAGE;
          mbar_expect_tx(&bars.full[s], C::STAGE);
          tma_load_2d(a, &tm_a, &bars.full[s], g.a_mn ? i * 128 : kb * 128,
                      g.a_mn ? kb * 128 : i * 128);
#pragma unroll
          for (int h = 0; h < (BN + 127) / 128; ++h)
            tma_load_2d(a + C::A_BYTES + h * 16384, &tm_b, &bars.full[s],
                        g.b_mn ? j * BN + h * 128 : kb * 128, g.b_mn ? kb * 128 : j * BN + h * 128);
          s_loads = it + 1;
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t id = idesc_e4m3(BN, g.a_mn, g.b_mn);
      const uint32_t step_a = g.a_mn ? 4096 : 32, step_b = g.b_mn ? 4096 : 32;
      int it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step)
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::NS, b = it % C::NB;
          ok = !failed() && (it < C::NB || wait(&bars.t_empty[b], it - C::NB, C::NB)) &&
               wait(&bars.full[s], it, C::NS);
          if (!ok) break;
          fence_after_sync();
          const uint32_t a = saddr(sm + s * C::STAGE);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + b * BN, sdesc_sw128(a + kk * step_a, 16384, 1024),
                   sdesc_sw128(a + C::A_BYTES + kk * step_b, 16384, 1024), id, kk > 0);
          mma_commit(&bars.empty[s]);
          mma_commit(&bars.t_full[b]);
        }
      if (!ok) {
        fail();
        // nothing may be in flight when the CTA ends: its MMAs, and then the copies
        if (it > 0) mbar_wait_poll(&bars.t_full[(it - 1) % C::NB], ((it - 1) / C::NB) & 1);
      }
    }
  } else {
    const int t0 = threadIdx.x - 64;
    int it = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int i, j;
      tile_at(t, ti, tj, i, j);
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::NSC;
        ok = __all_sync(0xffffffffu, !failed() && (it < C::NSC ||
                                                   wait(&bars.s_empty[s], it - C::NSC, C::NSC)));
        if (!ok) break;
        float* a = sc + s * C::SC_FLOATS;
#pragma unroll
        for (int e = t0; e < 128; e += 64) {
          const int row = min(i * 128 + e, g.m - 1);
          copy_async<4>(a + e, g.sa + (int64_t)(row >> g.sa_shift) * g.sa_i + kb * g.sa_b);
        }
        if constexpr (COL) {
#pragma unroll
          for (int e = t0; e < BN; e += 64) {
            const int col = min(j * BN + e, g.n - 1);
            copy_async<4>(a + 128 + e, g.sb + (int64_t)(col >> g.sb_shift) * g.sb_i + kb * g.sb_b);
          }
        } else if (t0 < (BN + 127) / 128) {
          const int col = min(j * BN + t0 * 128, g.n - 1);
          copy_async<4>(a + 128 + t0, g.sb + (int64_t)(col >> g.sb_shift) * g.sb_i + kb * g.sb_b);
        }
        copies_arrive(&bars.s_full[s]);
      }
    }
    if (!ok && lane == 0) fail();
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  } else {
  if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  if constexpr (BN == 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int r = q * 32 + lane, c0 = half * C::PER;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + c0;
    constexpr int CH = C::PER < 32 ? 16 : 32;            // columns at a time
    int it = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += step) {
      int i, j;
      tile_at(t, ti, tj, i, j);
      uint64_t acc[C::PER / 2];
#pragma unroll
      for (int c = 0; c < C::PER / 2; ++c) acc[c] = 0;
      for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
        const int b = it % C::NB, s = it % C::NSC;
        ok = __all_sync(0xffffffffu, !failed() && wait(&bars.s_full[s], it, C::NSC) &&
                                         wait(&bars.t_full[b], it, C::NB));
        if (!ok) break;
        fence_after_sync();
        const float* a = sc + s * C::SC_FLOATS;
        const float sa = a[r];
        const uint64_t one = COL ? 0 : f2_pack(sa * a[128 + half], sa * a[128 + half]);
        const uint64_t sa2 = f2_pack(sa, sa);
#pragma unroll
        for (int c = 0; c < C::PER; c += CH) {
          uint32_t x[CH];
          if constexpr (CH == 32)
            tmem_ld32(lanes + b * BN + c, x);
          else
            tmem_ld16(lanes + b * BN + c, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < CH; e += 2) {
            const uint64_t p = f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            uint64_t w = one;
            if constexpr (COL)
              w = fmul2(*reinterpret_cast<const uint64_t*>(a + 128 + c0 + c + e), sa2);
            acc[(c + e) / 2] = ffma2(p, w, acc[(c + e) / 2]);
          }
        }
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.t_empty[b]);
          mbar_arrive(&bars.s_empty[s]);
        }
      }
      if (!ok) {
        if (lane == 0) fail();
#pragma unroll
        for (int c = 0; c < C::PER / 2; ++c) acc[c] = f2_pack(NAN, NAN);
      }
      const int row = i * 128 + r, col = j * BN + c0;
      if (BN <= 128 && g.splits > 1) {
        // the MMAs have read all stages: the ring holds the partial tile, [column][129]
        float* part = reinterpret_cast<float*>(sm);
#pragma unroll
        for (int c = 0; c < C::PER; ++c) {
          float lo, hi;
          f2_unpack(acc[c / 2], lo, hi);
          part[c * 129 + r] = c % 2 ? hi : lo;
        }
      } else if (g.out_j == 1) {
        T* out = static_cast<T*>(g.out) + (int64_t)row * g.out_i + col;
        if (row < g.m) {
#pragma unroll
          for (int c = 0; c < C::PER; c += 16) store_row<T>(out + c, acc + c / 2, g.n - col - c, g.wide);
        }
      } else {
        T* out = static_cast<T*>(g.out) + row;
#pragma unroll
        for (int c = 0; c < C::PER; ++c) {
          float lo, hi;
          f2_unpack(acc[c / 2], lo, hi);
          if (row < g.m && col + c < g.n) out[(int64_t)(col + c) * g.out_j] = from_f32<T>(c % 2 ? hi : lo);
        }
      }
    }
  }
  if constexpr (BN <= 128) {
    if (g.splits > 1) {
      // every CTA adds its share of the tile's columns over the cluster, rank by rank
      __syncthreads();
      cluster_sync_all();
      int i, j;
      tile_at(first, ti, tj, i, j);
      const uint32_t part = saddr(sm);
      bool bad = false;
      for (int p = 0; p < g.splits; ++p) bad |= ld_cluster(saddr(&s_fail), p) != 0;
      const int e0 = (int)((int64_t)128 * BN * rank / g.splits);
      const int e1 = (int)((int64_t)128 * BN * (rank + 1) / g.splits);
      for (int e = e0 + threadIdx.x; e < e1; e += C::THREADS) {
        const int r = g.out_j == 1 ? e / BN : e & 127, c = g.out_j == 1 ? e % BN : e >> 7;
        const int row = i * 128 + r, col = j * BN + c;
        if (row >= g.m || col >= g.n) continue;
        float v = 0.f;
        for (int p = 0; p < g.splits; ++p)
          v += __uint_as_float(ld_cluster(part + (c * 129 + r) * 4, p));
        if (bad) v = NAN;
        static_cast<T*>(g.out)[(int64_t)row * g.out_i + (int64_t)col * g.out_j] = from_f32<T>(v);
      }
      cluster_sync_all();
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (failed() && threadIdx.x == 0)
    for (int s = 0; s < C::NS; ++s) {                  // the copies still in flight
      const int last = s_loads - 1 - ((s_loads - 1 - s) % C::NS + C::NS) % C::NS;
      if (s_loads > 0 && last >= 0) mbar_wait_poll(&bars.full[s], (last / C::NS) & 1);
    }
  if (warp == 1) tmem_free(tmem, C::COLS);
}

template <auto* KERNEL>
cudaError_t allow(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  e = cudaFuncSetAttribute((const void*)KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return e;
}

template <int BN, bool COL, typename T>
cudaError_t launch(const Gemm8& g, cudaStream_t st) {
  using C = GCfg<BN>;
  CUtensorMap ta, tb;
  const int box_b = g.b_mn ? 128 : BN < 128 ? BN : 128;
  if (!make_codes_map(&ta, g.a, g.a_mn ? g.m : g.k, g.a_mn ? g.k : g.m, g.a_pitch, 128) ||
      !make_codes_map(&tb, g.b, g.b_mn ? g.n : g.k, g.b_mn ? g.k : g.n, g.b_pitch, box_b))
    return cudaErrorInvalidValue;
  constexpr auto* k = gemm8_kernel<BN, COL, T>;
  cudaError_t e = allow<k>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((g.m + 127) / 128) * ((g.n + BN - 1) / BN);
  const int64_t most = kSMs * C::CTAS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.splits > 1 ? tiles * g.splits : tiles < most ? tiles : most));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (g.splits > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = g.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, k, ta, tb, g, wait_limit_ns());
}

// The operands' roles the other way round: out^T = B A^T.
Gemm8 swapped(const Gemm8& g) {
  Gemm8 s = g;
  s.m = g.n; s.n = g.m;
  s.a = g.b; s.b = g.a; s.a_pitch = g.b_pitch; s.b_pitch = g.a_pitch;
  s.a_mn = g.b_mn; s.b_mn = g.a_mn;
  s.sa = g.sb; s.sb = g.sa;
  s.sa_i = g.sb_i; s.sb_i = g.sa_i; s.sa_b = g.sb_b; s.sb_b = g.sa_b;
  s.sa_shift = g.sb_shift; s.sb_shift = g.sa_shift;
  s.out_i = g.out_j; s.out_j = g.out_i;
  return s;
}

template <typename T>
cudaError_t run(const Gemm8& in, cudaStream_t st) {
  Gemm8 g = in;
  const int nkb = (g.k + 127) / 128;
  g.wide = g.out_j == 1 && aligned_to(g.out, 32) && g.out_i * (int64_t)sizeof(T) % 32 == 0;
  // few rows: they become the columns of narrow tiles, and clusters share the summed dim
  const bool few = g.m <= 64 && !g.a_mn;
  const int64_t big = (int64_t)((g.m + 127) / 128) * ((g.n + 255) / 256);
  g.splits = 1;
  if (!few && big >= kSMs)
    return g.sb_shift == 7 ? launch<256, false, T>(g, st) : launch<256, true, T>(g, st);
  const int bn = !few ? 128 : g.m <= 16 ? 16 : g.m <= 32 ? 32 : 64;
  if (few) g = swapped(g);
  const int64_t tiles = (int64_t)((g.m + 127) / 128) * ((g.n + bn - 1) / bn);
  int64_t splits = 2 * kSMs / tiles;
  if (splits > 8) splits = 8;
  if (splits > nkb / 2) splits = nkb / 2;
  if (splits > 1) g.splits = (int)splits;
  if (bn == 128) return g.sb_shift == 7 ? launch<128, false, T>(g, st) : launch<128, true, T>(g, st);
  if (bn == 64) return launch<64, true, T>(g, st);
  if (bn == 32) return launch<32, true, T>(g, st);
  return launch<16, true, T>(g, st);
}

}  // namespace

cudaError_t launch_gemm8(int dtype, const Gemm8& g, cudaStream_t st) {
  return with_type(dtype, [&](auto* z) { return run<std::remove_pointer_t<decltype(z)>>(g, st); });
}

}  // namespace bl
