// Dense bf16 products of a calibration pass with their epilogues:
//   kronq_linear    Y = act(X W^T + bias) + R
//   kronq_gated     H = act(X Wg^T) * (X Wu^T)
// and the products of their backward passes (dX = dZ W, dW = dZ^T X).
//
// One template: D = A B^T (A: M x K, B: N x K, either stored K-major or
// MN-major) on tcgen05.mma kind::f16, bf16 operands, fp32 accumulator in
// TMEM. A CTA owns 128 rows of D and 128 columns (gated: the same 128
// columns of both products, side by side in TMEM, so that one thread holds
// both factors of an output):
//   warp 0      TMA producer (one elected lane), 4-stage ring of 64-wide slabs
//   warp 1      TMEM owner and MMA issuer (one elected lane)
//   warps 2..5  epilogue: TMEM -> registers -> bias, activation, residual ->
//               bf16 -> global
// dX of the gated pair is one product over K = 2 f: the k-slabs of (Gg, Wg)
// and then those of (Gu, Wu) go into one accumulator.
#include <string.h>

#include "act.cuh"
#include "kernels.cuh"

namespace kronq {
namespace {

constexpr int DT = 128;                  // tile rows and columns
constexpr int DBK = 64;                  // k per stage
constexpr int DSTAGES = 4;
constexpr int DTHREADS = 192;
constexpr int DPANEL = DT * DBK * 2;     // one operand panel of a stage (bytes)
constexpr int DBOX = 64 * DBK * 2;       // one MN-major box: 64 x 64

struct DenseP {
  int64_t M, N;
  int nk1, nseg;               // k-stages per segment, segments
  int tiles_m;
  const float *bias;           // linear
  __nv_bfloat16 *Z, *Z2;       // kept pre-activations (gated: A and U)
  int64_t ldz;
  const __nv_bfloat16 *R;
  int64_t ldr;
  __nv_bfloat16 *Y;
  int64_t ldy;
  int32_t *info;
};

struct DenseCtl {
  uint64_t full[DSTAGES], empty[DSTAGES], done, drain;
  uint32_t tmem_base;
  int abort;
};

template <bool GATED>
constexpr int dense_smem() {
  return DSTAGES * DPANEL * (GATED ? 3 : 2) + 1024 + int(sizeof(DenseCtl)) + 64;
}

__device__ __forceinline__ void load_panel(uint8_t *dst, const CUtensorMap *map, uint64_t *bar,
                                           bool mn, int32_t r0, int32_t k0) {
  if (!mn) {
    tma_load_2d(dst, map, bar, k0, r0);
  } else {
    tma_load_2d(dst, map, bar, r0, k0);
    tma_load_2d(dst + DBOX, map, bar, r0 + 64, k0);
  }
}

// 32 consecutive outputs of a row to (or from) global memory; `n` of them
// exist. Rows are 16-byte aligned at multiples of 8 elements.
__device__ __forceinline__ void store32(__nv_bfloat16 *p, const float *v, int n) {
  if (n >= 32) {
    uint4 o[4];
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(o);
#pragma unroll
    for (int t = 0; t < 16; ++t) h[t] = __floats2bfloat162_rn(v[2 * t], v[2 * t + 1]);
#pragma unroll
    for (int t = 0; t < 4; ++t) reinterpret_cast<uint4 *>(p)[t] = o[t];
  } else {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (t < n) p[t] = __float2bfloat16_rn(v[t]);
  }
}
__device__ __forceinline__ void add32(const __nv_bfloat16 *p, float *v, int n) {
  if (n >= 32) {
    uint4 o[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = reinterpret_cast<const uint4 *>(p)[t];
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(o);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const float2 f = __bfloat1622float2(h[t]);
      v[2 * t] += f.x;
      v[2 * t + 1] += f.y;
    }
  } else {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (t < n) v[t] += __bfloat162float(p[t]);
  }
}

// The epilogue of 32 consecutive columns of a row: v the accumulator (gated: v
// of the gate, u of the up projection), n of them in range.
template <bool GATED, int ACT>
__device__ __forceinline__ void finish32(const DenseP &p, int64_t row, int64_t col, int n,
                                         float *v, float *u) {
  if (!GATED && p.bias) {
#pragma unroll
    for (int t = 0; t < 32; ++t) v[t] += t < n ? __ldg(p.bias + col + t) : 0.f;
  }
  if (p.Z) store32(p.Z + row * p.ldz + col, v, n);
  if constexpr (GATED) {
    if (p.Z) store32(p.Z2 + row * p.ldz + col, u, n);
#pragma unroll
    for (int t = 0; t < 32; ++t) v[t] = act_f<ACT>(v[t]) * u[t];
  } else {
#pragma unroll
    for (int t = 0; t < 32; ++t) v[t] = act_f<ACT>(v[t]);
    if (p.R) add32(p.R + row * p.ldr + col, v, n);
  }
  store32(p.Y + row * p.ldy + col, v, n);
}

template <bool GATED, int ACT, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(DTHREADS, 1)
    dense_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmA2,
                 const __grid_constant__ CUtensorMap tmB2, const DenseP p) {
  constexpr int STAGE = DPANEL * (GATED ? 3 : 2);
  constexpr int COLS = GATED ? 256 : 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  DenseCtl *ctl = reinterpret_cast<DenseCtl *>(smem + DSTAGES * STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t m0 = int64_t(blockIdx.x % p.tiles_m) * DT;
  const int64_t n0 = int64_t(blockIdx.x / p.tiles_m) * DT;
  const int nk = p.nk1 * p.nseg;

  if (threadIdx.x == 0) {
    for (int s = 0; s < DSTAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    mbar_init(&ctl->done, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ctl->tmem_base;
  volatile int *abort = &ctl->abort;

  int issued = 0;
  if (warp == 0) {
    if (lane == 0) {
      for (int it = 0; it < nk; ++it) {
        const int s = it % DSTAGES;
        if (it >= DSTAGES && !mbar_wait(&ctl->empty[s], ((it / DSTAGES) - 1) & 1, abort)) break;
        uint8_t *st = smem + s * STAGE;
        const bool second = it >= p.nk1;
        const int32_t k0 = (second ? it - p.nk1 : it) * DBK;
        mbar_expect_tx(&ctl->full[s], STAGE);
        load_panel(st, second ? &tmA2 : &tmA, &ctl->full[s], A_MN, static_cast<int32_t>(m0), k0);
        load_panel(st + DPANEL, !GATED && second ? &tmB2 : &tmB, &ctl->full[s], B_MN,
                   static_cast<int32_t>(n0), k0);
        if (GATED)
          load_panel(st + 2 * DPANEL, &tmB2, &ctl->full[s], B_MN, static_cast<int32_t>(n0), k0);
        issued = it + 1;
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_make(1, A_MN, B_MN, DT, DT);
      bool ok = true;
      for (int it = 0; it < nk; ++it) {
        const int s = it % DSTAGES;
        if (!mbar_wait(&ctl->full[s], (it / DSTAGES) & 1, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem + s * STAGE), b0 = a0 + DPANEL;
#pragma unroll
        for (int kk = 0; kk < DBK / 16; ++kk) {
          const uint64_t da = A_MN ? sdesc_sw128(a0 + kk * 2048, DBOX, 1024)
                                   : sdesc_sw128(a0 + kk * 32, 16, 1024);
#pragma unroll
          for (int h = 0; h < (GATED ? 2 : 1); ++h) {
            const uint32_t b = b0 + h * DPANEL;
            const uint64_t db = B_MN ? sdesc_sw128(b + kk * 2048, DBOX, 1024)
                                     : sdesc_sw128(b + kk * 32, 16, 1024);
            umma_bf16(tbase + DT * h, da, db, idesc, (it | kk) != 0);
          }
        }
        umma_commit(&ctl->empty[s]);
      }
      if (ok) umma_commit(&ctl->done);
    }
  } else {
    const int q = warp & 3;
    const int64_t row = m0 + 32 * q + lane;
    const bool ok = mbar_wait(&ctl->done, 0, abort);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      for (int c = 0; c < DT / 32; ++c) {
        const int64_t col = n0 + 32 * c;
        if (col >= p.N) break;
        const int n = static_cast<int>(kq_min<int64_t>(32, p.N - col));
        const uint32_t ta = tbase + (static_cast<uint32_t>(32 * q) << 16) + 32 * c;
        float v[32], u[GATED ? 32 : 1];
        tmem_ld32(ta, v);
        if constexpr (GATED) tmem_ld32(ta + DT, u);
        if (row < p.M) finish32<GATED, ACT>(p, row, col, n, v, u);
      }
    }
  }

  // ---- teardown: after an abort make sure no copy or MMA is still in flight
  tc_fence_before();
  __syncthreads();
  if (ctl->abort) {
    if (threadIdx.x == 0) report(p.info, KRONQ_ERR_TIMEOUT);
    if (warp == 0 && lane == 0) {
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < DSTAGES && s < issued; ++s) {
        const int last = ((issued - 1 - s) / DSTAGES) * DSTAGES + s;
        while (!mbar_try_wait(&ctl->full[s], (last / DSTAGES) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    if (warp == 1 && lane == 0) {
      umma_commit(&ctl->drain);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&ctl->drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, COLS);
  }
}

// ---------------------------------------------------------------- CTA pairs
// The same products on CTA pairs, for many rows: a cluster of two CTAs owns a
// 256 x 256 tile of D (gated: 256 rows x 128 columns of both products). Each
// CTA holds 128 rows of A and 128 of the 256 columns' rows of B (gated: the
// even CTA Wg's, the odd one Wu's), so a k-slab of 64 costs a CTA 32 KB of
// shared-memory traffic for 128 x 256 x 64 products: half of what one CTA
// alone would load. The kernel is persistent: TMEM holds two accumulators,
// and the epilogue of one tile runs while the next one accumulates.
//   warps 0..7  epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and half
//               w / 4 of the tile's columns
//   warp 8      TMA producer (each CTA loads its own panels; the bytes of both
//               are counted on the even CTA's barrier)
//   warp 9      TMEM owner; in the even CTA the MMA issuer
constexpr int PSTAGES = 6;
constexpr int PSTAGE = 2 * DPANEL;
constexpr int PTHREADS = 320;
constexpr int PGROUP = 8;                // tile raster: row tiles per band

struct PairCtl {
  uint64_t full[PSTAGES];    // both CTAs' panels landed (even CTA's is used)
  uint64_t empty[PSTAGES];   // MMAs that read the stage finished (both CTAs)
  uint64_t tfull[2];         // accumulator complete (both CTAs)
  uint64_t tempty[2];        // read out by both CTAs' epilogues (even CTA's)
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int PSMEM = PSTAGES * PSTAGE + 1024 + int(sizeof(PairCtl)) + 64;

__device__ __forceinline__ void load_panel_pair(uint8_t *dst, const CUtensorMap *map,
                                                uint32_t bar, bool mn, int32_t r0, int32_t k0) {
  if (!mn) {
    tma_load_2d_pair(dst, map, bar, k0, r0);
  } else {
    tma_load_2d_pair(dst, map, bar, r0, k0);
    tma_load_2d_pair(dst + DBOX, map, bar, r0 + 64, k0);
  }
}

// Row and column tile of tile t: bands of PGROUP row tiles, column by column,
// so that the tiles in flight share their panels through L2.
__device__ __forceinline__ void pair_tile(int64_t t, int tiles_m, int tiles_n, int64_t &bi,
                                          int64_t &bj) {
  const int64_t band = t / (int64_t(PGROUP) * tiles_n);
  const int64_t rows = kq_min<int64_t>(PGROUP, tiles_m - band * PGROUP);
  const int64_t r = t - band * PGROUP * tiles_n;
  bi = band * PGROUP + r % rows;
  bj = r / rows;
}

template <bool GATED, int ACT, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PTHREADS, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmA2,
                      const __grid_constant__ CUtensorMap tmB2, const DenseP p) {
  constexpr int NT = GATED ? 128 : 256;   // columns of the output per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  PairCtl *ctl = reinterpret_cast<PairCtl *>(smem + PSTAGES * PSTAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int64_t cluster = cluster_id_x(), clusters = gridDim.x / 2;
  const int tiles_n = static_cast<int>((p.N + NT - 1) / NT);
  const int64_t tiles = int64_t(p.tiles_m) * tiles_n;
  const int nk = p.nk1 * p.nseg;

  if (threadIdx.x == 0) {
    for (int s = 0; s < PSTAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&ctl->tfull[a], 1);
      mbar_init(&ctl->tempty[a], 16);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  __syncthreads();
  if (warp == 9) tmem_alloc_pair(&ctl->tmem_base, 512);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = ctl->tmem_base;
  volatile int *abort = &ctl->abort;

  int64_t issued = 0;
  if (warp == 8) {
    if (lane == 0) {
      int64_t g = 0;
      bool ok = true;
      for (int64_t t = cluster; t < tiles && ok; t += clusters) {
        int64_t bi, bj;
        pair_tile(t, p.tiles_m, tiles_n, bi, bj);
        const int32_t m0 = static_cast<int32_t>(bi * 256 + 128 * rank);
        const int32_t n0 = static_cast<int32_t>(bj * NT + (GATED ? 0 : 128 * rank));
        for (int it = 0; it < nk; ++it, ++g) {
          const int s = static_cast<int>(g % PSTAGES);
          if (g >= PSTAGES && !mbar_wait(&ctl->empty[s], ((g / PSTAGES) - 1) & 1, abort)) {
            ok = false;
            break;
          }
          uint8_t *st = smem + s * PSTAGE;
          const bool second = it >= p.nk1;
          const int32_t k0 = (second ? it - p.nk1 : it) * DBK;
          const uint32_t bar = mapa_shared(smem_u32(&ctl->full[s]), 0);
          if (rank == 0) mbar_expect_tx(&ctl->full[s], 2 * PSTAGE);
          load_panel_pair(st, second ? &tmA2 : &tmA, bar, A_MN, m0, k0);
          load_panel_pair(st + DPANEL, (GATED ? rank != 0 : second) ? &tmB2 : &tmB, bar, B_MN, n0,
                          k0);
          issued = g + 1;
        }
      }
      // every arrival on this CTA's barriers has landed before the CTA ends
      for (int64_t e = kq_max<int64_t>(g - PSTAGES, 0); e < g && ok; ++e)
        ok = mbar_wait(&ctl->empty[e % PSTAGES], (e / PSTAGES) & 1, abort);
    }
  } else if (warp == 9) {
    if (rank == 0 && lane == 0) {
      const uint32_t idesc = idesc_make(1, A_MN, B_MN, 256, 256);
      int64_t g = 0;
      int i = 0;
      bool ok = true;
      for (int64_t t = cluster; t < tiles && ok; t += clusters, ++i) {
        const int a = i & 1;
        if (i >= 2 && !mbar_wait(&ctl->tempty[a], ((i >> 1) - 1) & 1, abort)) break;
        tc_fence_after();
        for (int it = 0; it < nk; ++it, ++g) {
          const int s = static_cast<int>(g % PSTAGES);
          if (!mbar_wait(&ctl->full[s], (g / PSTAGES) & 1, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * PSTAGE), b0 = a0 + DPANEL;
#pragma unroll
          for (int kk = 0; kk < DBK / 16; ++kk) {
            const uint64_t da = A_MN ? sdesc_sw128(a0 + kk * 2048, DBOX, 1024)
                                     : sdesc_sw128(a0 + kk * 32, 16, 1024);
            const uint64_t db = B_MN ? sdesc_sw128(b0 + kk * 2048, DBOX, 1024)
                                     : sdesc_sw128(b0 + kk * 32, 16, 1024);
            umma_bf16_pair(tbase + 256 * a, da, db, idesc, (it | kk) != 0);
          }
          umma_commit_pair(&ctl->empty[s]);
        }
        if (ok) umma_commit_pair(&ctl->tfull[a]);
      }
    }
  } else {
    const int q = warp & 3, half = warp >> 2;
    int i = 0;
    for (int64_t t = cluster; t < tiles; t += clusters, ++i) {
      const int a = i & 1;
      const bool ok = mbar_wait(&ctl->tfull[a], (i >> 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      int64_t bi, bj;
      pair_tile(t, p.tiles_m, tiles_n, bi, bj);
      const int64_t row = bi * 256 + 128 * rank + 32 * q + lane;
      for (int c = 0; c < NT / 64; ++c) {
        const int cc = half * (NT / 2) + 32 * c;
        const int64_t col = bj * NT + cc;
        if (col >= p.N) break;
        const int n = static_cast<int>(kq_min<int64_t>(32, p.N - col));
        const uint32_t ta = tbase + (static_cast<uint32_t>(32 * q) << 16) + 256 * a + cc;
        float v[32], u[GATED ? 32 : 1];
        tmem_ld32(ta, v);
        if constexpr (GATED) tmem_ld32(ta + 128, u);
        if (row < p.M) finish32<GATED, ACT>(p, row, col, n, v, u);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->tempty[a]), 0));
    }
  }

  // ---- teardown: after an abort make sure no copy or MMA is still in flight
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (ctl->abort) {
    if (threadIdx.x == 0) report(p.info, KRONQ_ERR_TIMEOUT);
    if (rank == 0 && warp == 8 && lane == 0) {
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < PSTAGES && s < issued; ++s) {
        const int64_t last = ((issued - 1 - s) / PSTAGES) * PSTAGES + s;
        while (!mbar_try_wait(&ctl->full[s], (last / PSTAGES) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    if (rank == 0 && warp == 9 && lane == 0) {
      umma_commit_pair(&ctl->drain);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&ctl->drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
  }
  __syncwarp();
  cluster_sync_all();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

// dZ = dY * act'(Z), or the gated pair's Gg and Gu, eight columns a thread.
// Every element is read before it is written by the same thread, so an output
// may be one of the inputs.
struct ActBwdP {
  int64_t n, w;
  const __nv_bfloat16 *dY, *Z, *U;
  int64_t lddy, ldz;
  __nv_bfloat16 *G, *G2;
  int64_t ldg;
};

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *v, int n) {
  if (n >= 8) {
    const uint4 o = *reinterpret_cast<const uint4 *>(p);
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&o);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 f = __bfloat1622float2(h[t]);
      v[2 * t] = f.x;
      v[2 * t + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = t < n ? __bfloat162float(p[t]) : 0.f;
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *v, int n) {
  if (n >= 8) {
    uint4 o;
    __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int t = 0; t < 4; ++t) h[t] = __floats2bfloat162_rn(v[2 * t], v[2 * t + 1]);
    *reinterpret_cast<uint4 *>(p) = o;
  } else {
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t < n) p[t] = __float2bfloat16_rn(v[t]);
  }
}

template <int ACT, bool GATED>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdP p) {
  const int64_t w8 = (p.w + 7) / 8, total = p.n * w8;
  for (int64_t e = blockIdx.x * int64_t(blockDim.x) + threadIdx.x; e < total;
       e += int64_t(gridDim.x) * blockDim.x) {
    const int64_t r = e / w8, c = (e - r * w8) * 8;
    const int n = static_cast<int>(kq_min<int64_t>(8, p.w - c));
    float g[8], z[8], u[8];
    load8(p.dY + r * p.lddy + c, g, n);
    if (GATED || ACT != KRONQ_ACT_NONE) load8(p.Z + r * p.ldz + c, z, n);
    if (GATED) load8(p.U + r * p.ldz + c, u, n);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      float h, dh;
      act_df<ACT>(GATED || ACT != KRONQ_ACT_NONE ? z[t] : 0.f, h, dh);
      if (GATED) {
        u[t] = g[t] * u[t] * dh;
        z[t] = g[t] * h;
      } else if (ACT != KRONQ_ACT_NONE) {
        g[t] *= dh;
      }
    }
    if (GATED) {
      store8(p.G + r * p.ldg + c, u, n);
      store8(p.G2 + r * p.ldg + c, z, n);
    } else {
      store8(p.G + r * p.ldg + c, g, n);
    }
  }
}

// db = column sums of dY * act'(Z): a CTA owns 32 columns and walks all rows,
// 8 rows at a time (one warp a row); the warps meet in a fixed order.
template <int ACT>
__global__ void __launch_bounds__(256)
    bias_grad_kernel(const __nv_bfloat16 *dY, int64_t lddy, const __nv_bfloat16 *Z, int64_t ldz,
                     int64_t n, int64_t w, float *db) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * int64_t(32) + lane;
  float s = 0.f;
  if (c < w) {
    for (int64_t r = warp; r < n; r += 8) {
      float h, dh = 1.f;
      if (ACT != KRONQ_ACT_NONE) act_df<ACT>(__bfloat162float(Z[r * ldz + c]), h, dh);
      s = fmaf(__bfloat162float(dY[r * lddy + c]), dh, s);
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < w) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += part[k][lane];
    db[c] = t;
  }
}

// Calls f with the activation as a compile-time constant.
template <class F>
kronq_status with_act(int act, F f) {
  switch (act) {
    case KRONQ_ACT_RELU: return f(std::integral_constant<int, KRONQ_ACT_RELU>());
    case KRONQ_ACT_SILU: return f(std::integral_constant<int, KRONQ_ACT_SILU>());
    case KRONQ_ACT_GELU: return f(std::integral_constant<int, KRONQ_ACT_GELU>());
    case KRONQ_ACT_GELU_TANH: return f(std::integral_constant<int, KRONQ_ACT_GELU_TANH>());
    default: return f(std::integral_constant<int, KRONQ_ACT_NONE>());
  }
}

// rows x K operand: K-major maps are {K, rows}, MN-major ones {rows, K}
kronq_status operand_map(CUtensorMap *m, const void *p, int64_t ld, bool mn, int64_t rows,
                         int64_t K) {
  return mn ? make_tmap_2d(m, p, true, rows, K, ld, 64, DBK)
            : make_tmap_2d(m, p, true, K, rows, ld, DBK, DT);
}

template <bool GATED, int ACT, bool A_MN, bool B_MN>
kronq_status launch_dense(cudaStream_t st, const CUtensorMap *tm, DenseP p) {
  if (p.M > 128) {
    auto *kern = dense_pair_kernel<GATED, ACT, A_MN, B_MN>;
    KQ_TRY(smem_attr(kern, PSMEM));
    p.tiles_m = static_cast<int>(ceil_div(p.M, 256));
    const int64_t tiles = p.tiles_m * ceil_div(p.N, GATED ? 128 : 256);
    const int64_t clusters = kq_min<int64_t>(tiles, 74);
    kern<<<static_cast<unsigned>(2 * clusters), PTHREADS, PSMEM, st>>>(tm[0], tm[1], tm[2], tm[3],
                                                                       p);
    KQ_CHECK_LAUNCH();
    return KRONQ_OK;
  }
  auto *kern = dense_kernel<GATED, ACT, A_MN, B_MN>;
  KQ_TRY(smem_attr(kern, dense_smem<GATED>()));
  p.tiles_m = static_cast<int>(ceil_div(p.M, DT));
  const int64_t tiles = p.tiles_m * ceil_div(p.N, DT);
  if (tiles > 0x7fffffff) return KRONQ_ERR_UNSUPPORTED;
  kern<<<static_cast<unsigned>(tiles), DTHREADS, dense_smem<GATED>(), st>>>(tm[0], tm[1], tm[2],
                                                                            tm[3], p);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

// C = sum over segments of A_s B_s^T (+ R), stored as bf16
kronq_status product(cudaStream_t st, int64_t M, int64_t N, int64_t K, const Mat &A, bool a_mn,
                     const Mat &B, const Mat *A2, const Mat *B2, const Mat &R, const Mat &C,
                     int32_t *info) {
  CUtensorMap tm[4];
  memset(tm, 0, sizeof(tm));
  KQ_TRY(operand_map(&tm[0], A.p, A.ld, a_mn, M, K));
  KQ_TRY(operand_map(&tm[1], B.p, B.ld, true, N, K));
  if (A2) {
    KQ_TRY(operand_map(&tm[2], A2->p, A2->ld, a_mn, M, K));
    KQ_TRY(operand_map(&tm[3], B2->p, B2->ld, true, N, K));
  }
  DenseP p = {};
  p.M = M;
  p.N = N;
  p.nk1 = static_cast<int>(ceil_div(K, DBK));
  p.nseg = A2 ? 2 : 1;
  p.R = static_cast<const __nv_bfloat16 *>(R.p);
  p.ldr = R.ld;
  p.Y = static_cast<__nv_bfloat16 *>(C.p);
  p.ldy = C.ld;
  p.info = info;
  return a_mn ? launch_dense<false, KRONQ_ACT_NONE, true, true>(st, tm, p)
              : launch_dense<false, KRONQ_ACT_NONE, false, true>(st, tm, p);
}

kronq_status zero_rows(cudaStream_t st, const Mat &m, int64_t rows, int64_t cols) {
  KQ_CUDA(cudaMemset2DAsync(m.p, m.ld * 2, 0, cols * 2, rows, st));
  return KRONQ_OK;
}

template <int ACT, bool GATED>
kronq_status launch_act_bwd(cudaStream_t st, const ActBwdP &p) {
  const int64_t total = p.n * ceil_div(p.w, 8);
  act_bwd_kernel<ACT, GATED>
      <<<static_cast<unsigned>(kq_min<int64_t>(ceil_div(total, 256), 148 * 16)), 256, 0, st>>>(p);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

__nv_bfloat16 *bf(void *p) { return static_cast<__nv_bfloat16 *>(p); }

}  // namespace

kronq_status linear_fwd(cudaStream_t st, int64_t n, int64_t d_in, int64_t d_out, const Mat &X,
                        const Mat &W, const float *bias, int act, const Mat &Z, const Mat &R,
                        const Mat &Y, int32_t *info) {
  CUtensorMap tm[4];
  memset(tm, 0, sizeof(tm));
  KQ_TRY(operand_map(&tm[0], X.p, X.ld, false, n, d_in));
  KQ_TRY(operand_map(&tm[1], W.p, W.ld, false, d_out, d_in));
  DenseP p = {};
  p.M = n;
  p.N = d_out;
  p.nk1 = static_cast<int>(ceil_div(d_in, DBK));
  p.nseg = 1;
  p.bias = bias;
  p.Z = bf(Z.p);
  p.ldz = Z.ld;
  p.R = bf(R.p);
  p.ldr = R.ld;
  p.Y = bf(Y.p);
  p.ldy = Y.ld;
  p.info = info;
  return with_act(act, [&](auto a) {
    return launch_dense<false, decltype(a)::value, false, false>(st, tm, p);
  });
}

kronq_status gated_fwd(cudaStream_t st, int64_t n, int64_t d, int64_t f, const Mat &X,
                       const Mat &Wg, const Mat &Wu, int act, const Mat &A, const Mat &U,
                       const Mat &H, int32_t *info) {
  CUtensorMap tm[4];
  memset(tm, 0, sizeof(tm));
  KQ_TRY(operand_map(&tm[0], X.p, X.ld, false, n, d));
  KQ_TRY(operand_map(&tm[1], Wg.p, Wg.ld, false, f, d));
  KQ_TRY(operand_map(&tm[3], Wu.p, Wu.ld, false, f, d));
  DenseP p = {};
  p.M = n;
  p.N = f;
  p.nk1 = static_cast<int>(ceil_div(d, DBK));
  p.nseg = 1;
  p.Z = bf(A.p);
  p.Z2 = bf(U.p);
  p.ldz = A.ld;
  p.Y = bf(H.p);
  p.ldy = H.ld;
  p.info = info;
  return with_act(act, [&](auto a) {
    return launch_dense<true, decltype(a)::value, false, false>(st, tm, p);
  });
}

kronq_status linear_bwd(cudaStream_t st, int64_t n, int64_t d_in, int64_t d_out, const Mat &dY,
                        const Mat &Z, int act, const Mat &X, const Mat &W, const Mat &dZ,
                        float *db, const Mat &dXr, const Mat &dX, const Mat &dW, int32_t *info) {
  if (n == 0) {
    if (db) KQ_CUDA(cudaMemsetAsync(db, 0, d_out * 4, st));
    return dW.p ? zero_rows(st, dW, d_out, d_in) : KRONQ_OK;
  }
  if (db) {  // before dZ is written: it may be dY or Z
    KQ_TRY(with_act(act, [&](auto a) {
      bias_grad_kernel<decltype(a)::value>
          <<<static_cast<unsigned>(ceil_div(d_out, 32)), 256, 0, st>>>(bf(dY.p), dY.ld, bf(Z.p),
                                                                       Z.ld, n, d_out, db);
      KQ_CHECK_LAUNCH();
      return KRONQ_OK;
    }));
  }
  Mat G = dY;
  if (act != KRONQ_ACT_NONE || (dZ.p && dZ.p != dY.p)) {
    ActBwdP p = {};
    p.n = n;
    p.w = d_out;
    p.dY = bf(dY.p);
    p.lddy = dY.ld;
    p.Z = bf(Z.p);
    p.ldz = Z.ld;
    p.G = bf(dZ.p);
    p.ldg = dZ.ld;
    KQ_TRY(with_act(act, [&](auto a) {
      return launch_act_bwd<decltype(a)::value, false>(st, p);
    }));
    G = dZ;
  }
  if (dX.p)
    KQ_TRY(product(st, n, d_in, d_out, G, false, W, nullptr, nullptr, dXr, dX, info));
  if (dW.p)
    KQ_TRY(product(st, d_out, d_in, n, G, true, X, nullptr, nullptr, Mat{}, dW, info));
  return KRONQ_OK;
}

kronq_status gated_bwd(cudaStream_t st, int64_t n, int64_t d, int64_t f, const Mat &dH,
                       const Mat &A, const Mat &U, int act, const Mat &X, const Mat &Wg,
                       const Mat &Wu, const Mat &Gg, const Mat &Gu, const Mat &dXr,
                       const Mat &dX, const Mat &dWg, const Mat &dWu, int32_t *info) {
  if (n == 0) {
    if (!dWg.p) return KRONQ_OK;
    KQ_TRY(zero_rows(st, dWg, f, d));
    return zero_rows(st, dWu, f, d);
  }
  ActBwdP p = {};
  p.n = n;
  p.w = f;
  p.dY = bf(dH.p);
  p.lddy = dH.ld;
  p.Z = bf(A.p);
  p.U = bf(U.p);
  p.ldz = A.ld;
  p.G = bf(Gg.p);
  p.G2 = bf(Gu.p);
  p.ldg = Gg.ld;
  KQ_TRY(with_act(act, [&](auto a) { return launch_act_bwd<decltype(a)::value, true>(st, p); }));
  if (dX.p) KQ_TRY(product(st, n, d, f, Gg, false, Wg, &Gu, &Wu, dXr, dX, info));
  if (dWg.p) {
    KQ_TRY(product(st, f, d, n, Gg, true, X, nullptr, nullptr, Mat{}, dWg, info));
    KQ_TRY(product(st, f, d, n, Gu, true, X, nullptr, nullptr, Mat{}, dWu, info));
  }
  return KRONQ_OK;
}

}  // namespace kronq
