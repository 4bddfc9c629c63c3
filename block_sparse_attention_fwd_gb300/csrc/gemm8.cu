// Products of e4m3 codes with a scale for each block of 128 of the summed dim:
//
//   out[i, j] = sum over blocks b of sa(i, b) sb(j, b) * sum over k in b of A[i, k] B[j, k]
//
// The inner sums run on the tensor cores (tcgen05.mma kind::f8f6f4, fp32 in TMEM), one
// block of 128 at a time; the outer sum in fp32 registers, where the scales come in, so
// nothing is rounded to fewer than 32 bits before the result.
//
// A CTA has a tile of 128 x BN.  Warp roles:
//   warp 0        TMA producer: codes of A and B, 128 of the summed dim a stage.
//   ISSUERS more  MMA issuers (one thread each, turn by turn), warp 1 the TMEM's owner: a
//                 block's product into one of NB accumulators.
//   one more      scales of the tile's rows and columns into a ring of shared memory.
//   EPI more      accumulate: 32 rows of BN or BN / 2 columns of the tile in registers, to
//                 which a warp adds the block's product from TMEM, scaled.
// Either operand may have the summed dim contiguous (K-major) or the other one
// (MN-major): the tiles in shared memory are alike, 128 rows of 128 bytes, and only
// the descriptors differ, so no operand is ever transposed in memory.
// Every mbarrier wait is bounded (tc.cuh); a tile that was given up is written as NaN.
//
// 8192^3 in 409 us, 2.69 PFLOP/s (1.4 times the measured bf16 rate of the tensor cores), in
// bursts; run for seconds the GPU's power is the bound (2.3 PFLOP/s at 1390 W and 1810 MHz,
// the tensor cores 57% busy).  With a scale a column, g_w, 590 us, of which two packed fp32
// instructions for two elements of a product instead of one are some 310; no pipe is more than
// 52% busy (the warps' largest stalls are fixed latencies and reads of TMEM).  Few rows:
// 8 x 16384 x 16384 in 45 us, the weight at 5.9 TB/s; a call of 8 x 5120 x 5120 takes 11, of
// which 4 are the launch and the sum over the cluster.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "rows.cuh"
#include "tc.cuh"

namespace bl {

namespace {

using namespace tc;

constexpr int kSMs = 152;
constexpr int kMostSplits = 4;     // CTAs that share a tile's sum

template <int BN, bool COL>
struct GCfg {
  static constexpr int NB = BN == 256 ? 2 : 4;          // accumulators in TMEM
  static constexpr int COLS = NB * BN < 32 ? 32 : NB * BN;
  static constexpr int ISSUERS = BN == 256 ? 2 : 4;
  static constexpr int PRE = 2 + ISSUERS;               // warps in front of the accumulating
  static constexpr int EPI = BN >= 64 ? 8 : 4;          // accumulating warps
  static constexpr int THREADS = (PRE + EPI) * 32;
  static constexpr int CTAS = BN >= 64 ? 1 : 2;         // on an SM
  static constexpr int A_BYTES = 128 * 128, B_BYTES = BN * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int NS = BN == 256 ? 4 : BN == 128 ? 6 : BN == 64 ? 8 : 5;
  static constexpr int GROUP = 16;                      // see tile_at
  static constexpr int NSC = 8;                         // stages of scales
  static constexpr int SC_FLOATS = 128 + BN;
  static constexpr int SMEM = NS * STAGE + NSC * SC_FLOATS * 4 + 1024;
  static constexpr int PER = BN / (EPI / 4);            // columns of a thread
};

template <typename C>
struct GBars {
  uint64_t full[C::NS], empty[C::NS], t_full[C::NB], t_empty[C::NB], s_full[C::NSC],
      s_empty[C::NSC];
};

// kind::f8f6f4 with e4m3 A and B (formats 0), fp32 accumulate.
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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

// A bounded wait, which also ends when another role has given up.  Reading the global
// timer takes longer than most waits do, so it starts only behind a few looks, each of
// which suspends the thread for a while.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                             const int* given_up) {
  auto look = [&]() { return mbar_try(bar, parity); };
  if (look()) return true;
  if (limit_ns >= kSuspendHintNs)
    for (int i = 0; i < 4; ++i)
      if (look()) return true;
  const uint64_t t0 = globaltimer();
  for (;;) {
    if (look()) return true;
    if (*(const volatile int*)given_up || globaltimer() - t0 > limit_ns) return false;
  }
}

__device__ __forceinline__ uint4 ld_cluster4(uint32_t addr, int rank) {
  uint4 v;
  asm volatile(
      "{\n .reg .u32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n"
      " ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [a];\n}\n"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// 16 lanes x 32 columns: thread t gets, of group g of 8 columns, columns 2 (t % 4) and the
// next of lane t / 4 in x[4 g], x[4 g + 1], and of lane t / 4 + 8 in x[4 g + 2], x[4 g + 3].
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
        "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
        "=r"(x[14]), "=r"(x[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&x)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
        "=r"(x[7])
      : "r"(taddr));
}

// A warp's 32 rows x PER columns of the tile, pairs of columns.  With a scale a row and one
// for all columns a thread has a row; with a scale a column too, four rows (r / 4 and 8, 16,
// 24 on) of every fourth pair, so that it needs a quarter of the columns' scales: the
// shared memory that a thread would read them from is what feeds the MMAs (8192^3: 1250
// TFLOP/s with a row a thread).  Its loads of 16 lanes take longer than those of 32: with them
// y and g_x of 8192^3 take 510 us.
template <int PER, bool COL>
struct Acc {
  uint64_t v[PER / 2];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int c = 0; c < PER / 2; ++c) v[c] = f2_pack(x, x);
  }
  // += the product in TMEM, scaled
  __device__ __forceinline__ void add(uint32_t taddr, const float* sa, const float* sb, int lane) {
    if constexpr (!COL) {
      const float s = sa[lane] * sb[0];
      const uint64_t ss = f2_pack(s, s);
#pragma unroll
      for (int c = 0; c < PER; c += 32) {
        uint32_t x[32];
        tmem_ld32(taddr + c, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          v[(c + e) / 2] = ffma2(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), ss,
                                 v[(c + e) / 2]);
      }
    } else {
      constexpr int CH = PER < 32 ? 16 : 32;             // columns at a time
      constexpr int N = PER / CH * 2;                    // of 16 lanes
      float rows[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) rows[u] = sa[(lane >> 2) + 8 * u];
      // the next part is on its way while this one is added
      uint32_t x[2][CH / 2];
      auto load = [&](int n) {
        const uint32_t at = taddr + ((uint32_t)(16 * (n & 1)) << 16) + n / 2 * CH;
        if constexpr (CH == 32)
          tmem_ld_16x32(at, x[n & 1]);
        else
          tmem_ld_16x16(at, x[n & 1]);
      };
      load(0);
      uint64_t cols[CH / 8];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = n / 2 * CH, h = n & 1;
        if (h == 0) {
#pragma unroll
          for (int k = 0; k < CH / 8; ++k)
            cols[k] = *reinterpret_cast<const uint64_t*>(sb + c + k * 8 + (lane & 3) * 2);
        }
        tmem_ld_wait();
        if (n + 1 < N) load(n + 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint64_t row = f2_pack(rows[2 * h + u], rows[2 * h + u]);
#pragma unroll
          for (int k = 0; k < CH / 8; ++k) {
            uint64_t& to = v[(c / 8 + k) * 4 + 2 * h + u];
            to = ffma2(f2_pack(__uint_as_float(x[h][4 * k + 2 * u]),
                               __uint_as_float(x[h][4 * k + 2 * u + 1])),
                       fmul2(cols[k], row), to);
          }
        }
      }
    }
  }
  // Rows of the warp's part to `out`, whose rows are `pitch` apart and 32-byte aligned; `rows`
  // and `cols` of them exist.  Four neighbouring lanes exchange what they hold of 32 columns,
  // so that they write four groups of 8 columns of a row side by side.  (As the lanes have
  // them: with a scale a column pairs, half sectors and four times the stores, g_w of 1024
  // tokens x 4096 x 4096 in 37 us, 32 so, of 8 x 5120 x 5120 32 and 16.5; else a sector of each
  // of 32 rows a store, 32779 x 2880 x 48 to fp32 in 94 us, 68 so.)
  template <typename T>
  __device__ __forceinline__ void store(T* out, int64_t pitch, int rows, int cols,
                                        int lane) const {
    const bool odd = lane & 1, high = lane & 2;
    auto swap = [](auto& lo, auto& hi, bool up, int with) {  // up keeps hi, else lo
      const auto got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, with);
      lo = up ? got : lo;
      hi = up ? hi : got;
    };
    // p[k] of the four lanes' lane l to p[l] of lane k
    auto exchange = [&](auto& p0, auto& p1, auto& p2, auto& p3) {
      swap(p0, p1, odd, 1);
      swap(p2, p3, odd, 1);
      swap(p0, p2, high, 2);
      swap(p1, p3, high, 2);
    };
    auto halves = [](uint64_t x) {                       // a pair in 16 bits each
      float lo, hi;
      f2_unpack(x, lo, hi);
      const Pair<T> p(lo, hi);
      return *reinterpret_cast<const uint32_t*>(&p);
    };
    if constexpr (COL) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = (lane >> 2) + 8 * u;
#pragma unroll
        for (int c = 0; c < PER; c += 32) {
          const int col = c + (lane & 3) * 8;
          const bool in = r < rows && col < cols;
          T* const to = out + r * pitch + col;
          if constexpr (sizeof(T) == 4) {
            float x[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) f2_unpack(v[(c / 8 + k) * 4 + u], x[k], y[k]);
            exchange(x[0], x[1], x[2], x[3]);
            exchange(y[0], y[1], y[2], y[3]);
            const float f[8] = {x[0], y[0], x[1], y[1], x[2], y[2], x[3], y[3]};
            store8<T, true>(to, f, in ? 8 : 0);
          } else {
            uint32_t p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) p[k] = halves(v[(c / 8 + k) * 4 + u]);
            exchange(p[0], p[1], p[2], p[3]);
            if (in) store_words(to, p);
          }
        }
      }
    } else if constexpr (sizeof(T) == 4 && PER < 128) {
      // (exchanging costs registers that these tiles' few have not: 128 x 5120 x 5120 in 16.3 us
      // instead of 14.4)
      if (lane < rows) {
#pragma unroll
        for (int c = 0; c < PER; c += 8) {
          const uint64_t f[4] = {v[c / 2], v[c / 2 + 1], v[c / 2 + 2], v[c / 2 + 3]};
          if (c < cols) store8(out + lane * pitch + c, f);
        }
      }
    } else {
      constexpr int W = 2 * (int)sizeof(T);              // words of 8 elements
      T* const mine = out + (lane & ~3) * pitch + (lane & 3) * 8;
#pragma unroll
      for (int c = 0; c < PER; c += 32) {
        uint32_t w[4][W];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint64_t x = v[c / 2 + k * 4 + i];
            if constexpr (sizeof(T) == 4) {
              float lo, hi;
              f2_unpack(x, lo, hi);
              w[k][2 * i] = __float_as_uint(lo);
              w[k][2 * i + 1] = __float_as_uint(hi);
            } else {
              w[k][i] = halves(x);
            }
          }
#pragma unroll
        for (int i = 0; i < W; ++i) exchange(w[0][i], w[1][i], w[2][i], w[3][i]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((lane & ~3) + k < rows && c + (lane & 3) * 8 < cols)
            store_words(mine + k * pitch + c, w[k]);
      }
    }
  }
  // f(row, column, value, value of the next column) of the thread's pairs
  template <typename F>
  __device__ __forceinline__ void each(int lane, F&& f) const {
#pragma unroll
    for (int c = 0; c < PER / 2; ++c) {
      float lo, hi;
      f2_unpack(v[c], lo, hi);
      if constexpr (COL)
        f((lane >> 2) + 8 * (c & 3), (c >> 2) * 8 + (lane & 3) * 2, lo, hi);
      else
        f(lane, 2 * c, lo, hi);
    }
  }
};

// Tiles in groups of GROUP along i, j by j: a group's rows of A stay in L2 while B
// passes by.
template <int GROUP>
__device__ __forceinline__ void tile_at(int t, int ti, int tj, int& i, int& j) {
  const int per = GROUP * tj, g = t / per, r = t - g * per;
  const int h = min(GROUP, ti - g * GROUP);
  j = r / h;
  i = g * GROUP + (r - j * h);
}

// COL: every column has a scale of its own; else every 128 share one.
template <int BN, bool COL, typename T>
__global__ void __launch_bounds__(GCfg<BN, COL>::THREADS, GCfg<BN, COL>::CTAS)
    gemm8_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 Gemm8 g, uint64_t wait_ns) {
  using C = GCfg<BN, COL>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  float* sc = reinterpret_cast<float*>(sm + C::NS * C::STAGE);
  __shared__ __align__(8) GBars<C> bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail, s_loads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ti = (g.m + 127) / 128, tj = (g.n + BN - 1) / BN, tiles = ti * tj;
  const int nkb = (g.k + 127) / 128;
  // with splits, a cluster shares a tile: each CTA has a part of the summed dim
  const int share = BN <= 128 ? g.splits : 1;
  const int rank = blockIdx.x % share, first = blockIdx.x / share, step = gridDim.x / share;
  const int kb0 = (int)((int64_t)nkb * rank / share);
  const int kb1 = (int)((int64_t)nkb * (rank + 1) / share);

  // a stage of the summed dim's block kb of tile (i, j)
  auto load = [&](int s, int i, int j, int kb) {
    uint8_t* a = sm + s * C::STAGE;
    mbar_expect_tx(&bars.full[s], C::STAGE);
    const int row = i * 128, col = j * BN;
    tma_load_2d(a, &tm_a, &bars.full[s], g.a_mn ? row : kb * 128, g.a_mn ? kb * 128 : row);
#pragma unroll
    for (int h = 0; h < (BN + 127) / 128; ++h)
      tma_load_2d(a + C::A_BYTES + h * 16384, &tm_b, &bars.full[s],
                  g.b_mn ? col + h * 128 : kb * 128, g.b_mn ? kb * 128 : col + h * 128);
  };
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
      mbar_init(&bars.s_full[s], 32);
      mbar_init(&bars.s_empty[s], C::EPI);
    }
    s_fail = 0;
    s_loads = 0;
    fence_mbar_init();
    // the first stages are on their way while the rest of the CTA gets ready
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    int i, j;
    tile_at<C::GROUP>(first, ti, tj, i, j);
    for (int s = 0; s < C::NS && first < tiles && kb0 + s < kb1; ++s) load(s, i, j, kb0 + s);
  }
  if (warp == 1) tmem_alloc(&s_tmem, C::COLS);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t* bar, int use, int ring) {   // for the phase of use `use` of a slot
    return wait_bounded(saddr(bar), (use / ring) & 1, wait_ns, &s_fail);
  };
  auto failed = [&]() { return *(volatile int*)&s_fail != 0; };
  auto fail = [&]() { atomicOr(&s_fail, 1); };

  // The accumulating warps need registers, the others few; the shares are the launch's 384
  // x 168.  (Either share too small spills a few in its loop over the blocks, which costs a
  // quarter of the rate: g_w at 8192^3 in 763 us with 56 and 224.)
  if (warp < C::PRE) {
    if constexpr (BN == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0) {
      if (lane == 0) {
        int it = 0;
        bool ok = true;
        s_loads = min(C::NS, first < tiles ? kb1 - kb0 : 0);
        for (int t = first; ok && t < tiles; t += step) {
          int i, j;
          tile_at<C::GROUP>(t, ti, tj, i, j);
          for (int kb = kb0; kb < kb1; ++kb, ++it) {
            if (t == first && kb - kb0 < C::NS) continue;  // on their way
            const int s = it % C::NS;
            ok = it < C::NS || wait(&bars.empty[s], it - C::NS, C::NS);
            if (!ok) break;
            load(s, i, j, kb);
            s_loads = it + 1;
          }
        }
        if (!ok) fail();
      }
    } else if (warp <= C::ISSUERS) {
      // The issuers take turns: a look at a barrier behind MMAs returns only when those have
      // been taken up, some 100 clocks in which one issuer alone would leave the tensor core
      // idle (with two looks a block, 930 clocks a block of 512).
      const int total = first < tiles ? ((tiles - 1 - first) / step + 1) * (kb1 - kb0) : 0;
      if (lane == 0) {
        const uint32_t id = idesc_e4m3(128, BN, g.a_mn, g.b_mn);
        const uint32_t step_a = g.a_mn ? 4096 : 32, step_b = g.b_mn ? 4096 : 32;
        int it = warp - 1;
        for (; it < total; it += C::ISSUERS) {
          const int s = it % C::NS, b = it % C::NB;
          if (!((it < C::NB || wait(&bars.t_empty[b], it - C::NB, C::NB)) &&
                wait(&bars.full[s], it, C::NS)))
            break;
          fence_after_sync();
          const uint32_t a = saddr(sm + s * C::STAGE);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + b * BN, sdesc_sw128(a + kk * step_a, 16384, 1024),
                   sdesc_sw128(a + C::A_BYTES + kk * step_b, 16384, 1024), id, kk > 0);
          mma_commit(&bars.empty[s]);
          mma_commit(&bars.t_full[b]);
        }
        if (it < total) fail();
        // Nothing may be in flight when the CTA ends: the MMAs, and then the copies.  An issuer
        // that has issued all of its blocks waits too: the warps that give up may be the
        // accumulating ones, with its last products still under way.
        const int last = it - C::ISSUERS;
        if (last >= 0) mbar_wait_poll(&bars.t_full[last % C::NB], (last / C::NB) & 1);
      }
    } else {
      // Scales that lie side by side come 16 bytes a lane, others by pointers that walk with
      // the blocks.
      const bool a_run = g.sa_i == 1 && g.sa_shift == 0;
      const bool a_wide = a_run && aligned_to(g.sa, 16) && g.sa_b % 4 == 0;
      const bool b_wide = aligned_to(g.sb, 16) && g.sb_b % 4 == 0;
      auto run = [&](float* to, const float* from, int left, int count, bool wide) {
        if (wide) {
          for (int e = lane * 4; e < count; e += 128)
            copy_async<16>(to + e, from + (e < left ? e : 0), min(max(left - e, 0) * 4, 16));
        } else {
          for (int e = lane; e < count; e += 32)
            copy_async<4>(to + e, from + (e < left ? e : 0), e < left ? 4 : 0);
        }
      };
      int it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += step) {
        int i, j;
        tile_at<C::GROUP>(t, ti, tj, i, j);
        const float* pa[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = a_run ? i * 128 : min(i * 128 + lane + 32 * u, g.m - 1);
          pa[u] = g.sa + (int64_t)(row >> g.sa_shift) * g.sa_i + kb0 * g.sa_b;
        }
        // few columns: one a lane, or two; many: side by side; !COL: one for 128
        constexpr int PB = BN <= 64 ? (BN + 31) / 32 : 1;
        const float* pb[PB];
#pragma unroll
        for (int u = 0; u < PB; ++u) {
          const int col = j * BN + (!COL ? lane * 128 : BN <= 64 ? lane + 32 * u : 0);
          pb[u] = g.sb + (int64_t)(min(col, g.n - 1) >> g.sb_shift) * g.sb_i + kb0 * g.sb_b;
        }
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::NSC;
          ok = __all_sync(0xffffffffu,
                          it < C::NSC || wait(&bars.s_empty[s], it - C::NSC, C::NSC));
          if (!ok) break;
          float* a = sc + s * C::SC_FLOATS;
          if (a_run) {
            run(a, pa[0], g.m - i * 128, 128, a_wide);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) copy_async<4>(a + lane + 32 * u, pa[u]);
          }
          if constexpr (!COL) {
            if (lane < (BN + 127) / 128) copy_async<4>(a + 128 + lane, pb[0]);
          } else if constexpr (BN <= 64) {
#pragma unroll
            for (int u = 0; u < PB; ++u)
              if (lane + 32 * u < BN) copy_async<4>(a + 128 + lane + 32 * u, pb[u]);
          } else {
            run(a + 128, pb[0], g.n - j * BN, BN, b_wide);
          }
          copies_arrive(&bars.s_full[s]);
#pragma unroll
          for (int u = 0; u < 4; ++u) pa[u] += g.sa_b;
#pragma unroll
          for (int u = 0; u < PB; ++u) pb[u] += g.sb_b;
        }
      }
      if (!ok && lane == 0) fail();
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    if constexpr (BN == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int q = warp & 3, c0 = ((warp - C::PRE) >> 2) * C::PER;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + c0;
    int it = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += step) {
      int i, j;
      tile_at<C::GROUP>(t, ti, tj, i, j);
      Acc<C::PER, COL> acc;
      acc.fill(0.f);
      for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
        const int b = it % C::NB, s = it % C::NSC;
        ok = __all_sync(0xffffffffu,
                        wait(&bars.s_full[s], it, C::NSC) && wait(&bars.t_full[b], it, C::NB));
        if (!ok) break;
        fence_after_sync();
        const float* a = sc + s * C::SC_FLOATS;
        acc.add(lanes + b * BN, a + q * 32, a + 128 + (COL ? c0 : c0 / 128), lane);
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.t_empty[b]);
          mbar_arrive(&bars.s_empty[s]);
        }
      }
      if (!ok) {
        if (lane == 0) fail();
        acc.fill(NAN);
      }
      const int row = i * 128 + q * 32, col = j * BN + c0;
      if (BN <= 128 && g.splits > 1) {
        // the MMAs have read all stages: the ring holds the partial tile, the result's
        // contiguous dim along its rows
        if (g.out_j == 1) {
          float* part = reinterpret_cast<float*>(sm) + q * 32 * (BN + 4) + c0;
          acc.each(lane, [&](int r, int c, float lo, float hi) {
            *reinterpret_cast<float2*>(part + r * (BN + 4) + c) = make_float2(lo, hi);
          });
        } else {
          float* part = reinterpret_cast<float*>(sm) + q * 32 + c0 * 132;
          acc.each(lane, [&](int r, int c, float lo, float hi) {
            part[c * 132 + r] = lo;
            part[c * 132 + 132 + r] = hi;
          });
        }
      } else if (g.out_j == 1) {
        T* out = static_cast<T*>(g.out) + (int64_t)row * g.out_i + col;
        const int n = g.n - col;
        bool whole = false;
        if constexpr (C::PER >= 32) {
          whole = g.wide;
          if (whole) acc.store(out, g.out_i, g.m - row, n, lane);
        }
        if (!whole) {
          acc.each(lane, [&](int r, int c, float lo, float hi) {
            if (row + r >= g.m) return;
            T* p = out + r * g.out_i + c;
            if (g.pairs && c + 1 < n) {
              *reinterpret_cast<Pair<T>*>(p) = Pair<T>(lo, hi);
            } else {
              if (c < n) p[0] = from_f32<T>(lo);
              if (c + 1 < n) p[1] = from_f32<T>(hi);
            }
          });
        }
      } else {
        T* out = static_cast<T*>(g.out) + row + (int64_t)col * g.out_j;
        acc.each(lane, [&](int r, int c, float lo, float hi) {
          if (row + r >= g.m) return;
          if (col + c < g.n) out[c * g.out_j + r] = from_f32<T>(lo);
          if (col + c + 1 < g.n) out[(c + 1) * g.out_j + r] = from_f32<T>(hi);
        });
      }
    }
  }
  if constexpr (BN <= 128) {
    if (g.splits > 1) {
      // every CTA adds its share of the tile's columns over the cluster, rank by rank
      __syncthreads();
      cluster_sync_all();
      int i, j;
      tile_at<C::GROUP>(first, ti, tj, i, j);
      const uint32_t part = saddr(sm);
      bool bad = false;
      for (int p = 0; p < g.splits; ++p) bad |= ld_cluster(saddr(&s_fail), p) != 0;
      // four neighbours of the result's contiguous dim at a time, all ranks' under way at
      // once (one by one, a sum of 7 ranks at 128 x 5120 x 5120 took 60 us)
      const bool rows = g.out_j == 1;
      const int wide = rows ? BN : 128, pitch = wide + 4, quads = 128 * BN / 4;
      const int e0 = quads * rank / g.splits, e1 = quads * (rank + 1) / g.splits;
      for (int e = e0 + threadIdx.x; e < e1; e += 2 * C::THREADS) {
        uint4 v[2][kMostSplits];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int eu = e + u * C::THREADS, x = eu * 4 / wide, y = eu * 4 - x * wide;
#pragma unroll
          for (int p = 0; p < kMostSplits; ++p)
            if (p < g.splits && eu < e1) v[u][p] = ld_cluster4(part + (x * pitch + y) * 4, p);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int eu = e + u * C::THREADS, x = eu * 4 / wide, y = eu * 4 - x * wide;
          const int row = i * 128 + (rows ? x : y), col = j * BN + (rows ? y : x);
          if (eu >= e1 || row >= g.m || col >= g.n) continue;
          float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 0; p < kMostSplits; ++p)
            if (p < g.splits) {
              f[0] += __uint_as_float(v[u][p].x);
              f[1] += __uint_as_float(v[u][p].y);
              f[2] += __uint_as_float(v[u][p].z);
              f[3] += __uint_as_float(v[u][p].w);
            }
          T* out = static_cast<T*>(g.out) + (int64_t)row * g.out_i + (int64_t)col * g.out_j;
          const int left = rows ? g.n - col : g.m - row;
          if (g.quads && left >= 4) {
            if (bad) f[0] = f[1] = f[2] = f[3] = NAN;
            reinterpret_cast<Pair<T>*>(out)[0] = Pair<T>(f[0], f[1]);
            reinterpret_cast<Pair<T>*>(out)[1] = Pair<T>(f[2], f[3]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < left) out[k] = from_f32<T>(bad ? NAN : f[k]);
          }
        }
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

template <int BN, bool COL, typename T>
cudaError_t launch(const Gemm8& g, cudaStream_t st) {
  using C = GCfg<BN, COL>;
  // rows of B that lie across the summed dim come 128 columns at a time
  if (BN < 128 && g.b_mn) return cudaErrorInvalidValue;
  // many columns with a scale each lie side by side
  if (COL && BN >= 128 && g.sb_i != 1) return cudaErrorInvalidValue;
  CUtensorMap ta, tb;
  const int box_b = g.b_mn || BN > 128 ? 128 : BN;
  if (!make_codes_map(&ta, g.a, g.a_mn ? g.m : g.k, g.a_mn ? g.k : g.m, g.a_pitch, 128) ||
      !make_codes_map(&tb, g.b, g.b_mn ? g.n : g.k, g.b_mn ? g.k : g.n, g.b_pitch, box_b))
    return cudaErrorInvalidValue;
  constexpr auto* k = gemm8_kernel<BN, COL, T>;
  cudaError_t e = allow_smem<k>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)((g.m + 127) / 128) * ((g.n + BN - 1) / BN);
  const int64_t most = kSMs * C::CTAS;
  const int share = g.splits;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (share > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = share;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  cfg.gridDim = dim3((unsigned)((g.splits > 1 || tiles < most ? tiles : most) * share));
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

// Which tile, by an estimate of the time.  A block of 128 of the summed dim takes 0.46 us in
// a tile of 128 x 256 (0.64 with a scale a column), 0.33 (0.45) in one of 128 x 128, 0.3 in
// one of 128 x 64, 0.25 in a narrow one, whose products are too short to fill the time
// between one wait and the next; a tile's end takes 1 to 1.5, a sum over a cluster 1.5 and
// more with the columns.  Measured: 512 x 5120 x 5120 in 23, 33 and 41 us in tiles of 256, 128
// and 64 columns, 128 x 5120 x 5120 in 23, 18.5 and 17 us, 14.8 with two CTAs a tile.
struct Choice {
  int bn, splits;
  float us;
};
void consider(Choice& best, const Gemm8& g, int bn, int ctas, float block_us, float tile_us) {
  const int nkb = (g.k + 127) / 128;
  const int64_t tiles = (int64_t)((g.m + 127) / 128) * ((g.n + bn - 1) / bn);
  const int64_t at_once = (int64_t)kSMs * ctas;
  for (int splits = 1; splits <= (bn == 256 ? 1 : kMostSplits); splits *= 2) {
    if (splits > 1 && (splits > nkb || tiles * splits > at_once)) break;
    const int64_t rounds = (tiles * splits + at_once - 1) / at_once;
    const int blocks = (nkb + splits - 1) / splits;
    const float us = rounds * (blocks * block_us + tile_us) + (splits > 1 ? 1.5f + bn / 64.f : 0.f);
    if (us < best.us) best = Choice{bn, splits, us};
  }
}

template <typename T>
cudaError_t run(const Gemm8& in, cudaStream_t st) {
  Gemm8 g = in;
  // few rows become the columns of narrow tiles
  const bool few = g.m <= 64 && !g.a_mn;
  if (few) g = swapped(g);
  const bool col = g.sb_shift != 7;
  Choice c{128, 1, 1e30f};
  if (few) {
    const int bn = g.n <= 16 ? 16 : g.n <= 32 ? 32 : 64;
    consider(c, g, bn, bn == 64 ? 1 : 2, bn == 64 ? 0.3f : 0.25f, 1.f);
  } else {
    consider(c, g, 256, 1, col ? 0.64f : 0.46f, 1.5f);
    consider(c, g, 128, 1, col ? 0.45f : 0.33f, 1.f);
    if (!g.b_mn) consider(c, g, 64, 1, 0.3f, 1.f);
  }
  g.splits = c.splits;
  const size_t z = sizeof(T);
  g.wide = g.out_j == 1 && aligned_to(g.out, 32) && g.out_i * z % 32 == 0;
  g.pairs = g.out_j == 1 && aligned_to(g.out, 2 * z) && g.out_i % 2 == 0;
  g.quads = aligned_to(g.out, 2 * z) && (g.out_j == 1 ? g.out_i : g.out_j) % 2 == 0;
  if (c.bn == 256) return col ? launch<256, true, T>(g, st) : launch<256, false, T>(g, st);
  if (c.bn == 128) return col ? launch<128, true, T>(g, st) : launch<128, false, T>(g, st);
  if (c.bn == 64) return col ? launch<64, true, T>(g, st) : launch<64, false, T>(g, st);
  if (c.bn == 32) return launch<32, true, T>(g, st);
  return launch<16, true, T>(g, st);
}

}  // namespace

cudaError_t launch_gemm8(int dtype, const Gemm8& g, cudaStream_t st) {
  return with_type(dtype, [&](auto* z) { return run<std::remove_pointer_t<decltype(z)>>(g, st); });
}

}  // namespace bl
