// Dense bf16 products of a calibration pass with their epilogues:
//   kronq_linear    Y = act(X W^T + bias) + R
//   kronq_gated     H = act(X Wg^T) * (X Wu^T)
// and the products of their backward passes (dX = dZ W, dW = dZ^T X).
//
// All of them are D = A B^T (A: M x K, B: N x K, either stored K-major or
// MN-major) on tcgen05.mma kind::f16, bf16 operands brought in by TMA, fp32
// accumulators in TMEM, and an epilogue on the way out (bias, activation,
// product of the pair, residual, one rounding to bf16). Two kernels: CTA pairs
// on tiles of 256 rows for many tokens, and a kernel for few tokens that is
// bound by reading the weights and splits k over the CTAs of a cluster. In
// both, the gated pair's two products share one pass over X and meet in the
// epilogue of the thread that holds both factors of an output.
// dX of the gated pair is one product over K = 2 f: the k-slabs of (Gg, Wg)
// and then those of (Gu, Wu) go into one accumulator.
#include <string.h>

#include "act.cuh"
#include "kernels.cuh"

namespace kronq {
namespace {

constexpr int DT = 128;                  // tile rows and columns
constexpr int DBK = 64;                  // k per stage
constexpr int DPANEL = DT * DBK * 2;     // one operand panel of a stage (bytes)
constexpr int DBOX = 64 * DBK * 2;       // one MN-major box: 64 x 64

struct DenseP {
  int64_t M, N, K;
  int nk1, nseg;               // k-stages per segment, segments
  int tiles_m, act;
  const float *bias;           // linear
  __nv_bfloat16 *Z, *Z2;       // kept pre-activations (gated: A and U)
  int64_t ldz;
  const __nv_bfloat16 *R;
  int64_t ldr;
  __nv_bfloat16 *Y;
  int64_t ldy;
  int32_t *info;
};

__device__ __forceinline__ void load_panel(uint8_t *dst, const CUtensorMap *map, uint64_t *bar,
                                           bool mn, int32_t r0, int32_t k0) {
  if (!mn) {
    tma_load_2d(dst, map, bar, k0, r0);
  } else {
    tma_load_2d(dst, map, bar, r0, k0);
    tma_load_2d(dst + DBOX, map, bar, r0 + 64, k0);
  }
}

// ---------------------------------------------------------------- few tokens
// For few tokens the sides change places: 128 weight rows are the MMA's M and
// up to NT tokens its N, so that a tile wastes no tensor work on absent rows
// and the weights, which bound the call, stream through one 64-wide slab ring.
// The k range is split over a cluster of S CTAs (as many as fill the SMs):
// each accumulates its part in TMEM, writes it to its shared memory as
// [token][feature], and after a cluster barrier every CTA sums a share of the
// tile over the S parts, always in the order of their ranks, through
// distributed shared memory. Warp 0 loads (one lane), warp 1 issues the MMAs
// (one lane), then all four warps read TMEM and finish the tile.
//   Bound by reading the weights. Back to back: one token 4096 -> 11008 16.5 us
// (5.5 TB/s), the gated pair 30.5 us (5.9 TB/s), 48 tokens 11008 -> 4096 20.3 us;
// 4096 -> 4096 7.3 us (4.6 TB/s: start, the clusters' meeting and the end cost 3 us).
constexpr int FTHREADS = 128;

template <bool GATED, int NT, bool TWO>
struct Few {
  static constexpr int STAGE = DPANEL * (GATED ? 2 : 1) + NT * 128;
  // two CTAs an SM where four stages fit in half of it (TWO: three), else one
  static constexpr int PER_SM = TWO || STAGE * 4 <= 108 * 1024 ? 2 : 1;
  static constexpr int STAGES = (PER_SM == 2 ? 108 : 216) * 1024 / STAGE;
  static constexpr int SMEM = STAGES * STAGE + 1024 + 256;
  static constexpr int COLS = (GATED ? 2 : 1) * NT < 32 ? 32 : (GATED ? 2 : 1) * NT;
  static_assert(STAGES * STAGE >= (GATED ? 2 : 1) * NT * 128 * 4, "parts fit in the ring");
};

struct FewP {
  DenseP d;
  int split, tiles_t;   // CTAs per tile, token tiles
};

template <int STAGES>
struct FewCtl {
  uint64_t full[STAGES], empty[STAGES], done, drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void store4(__nv_bfloat16 *p, float4 v, int n) {
  const __nv_bfloat162 o[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
  if (n >= 4) {
    *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(o);
  } else {
    p[0] = o[0].x;
    if (n > 1) p[1] = o[0].y;
    if (n > 2) p[2] = o[1].x;
  }
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
// The epilogue of four consecutive columns (n of them in range) of a row, bias
// added: v the accumulator (gated: v of the gate, u of the up projection).
template <bool GATED>
__device__ __forceinline__ void finish4(const DenseP &p, int64_t row, int64_t col, int n, float4 v,
                                        float4 u) {
  if (p.Z) store4(p.Z + row * p.ldz + col, v, n);
  if (GATED && p.Z) store4(p.Z2 + row * p.ldz + col, u, n);
  if (p.act != KRONQ_ACT_NONE) v = act4(p.act, v);
  if (GATED) {
    v = make_float4(v.x * u.x, v.y * u.y, v.z * u.z, v.w * u.w);
  } else if (p.R) {
    const __nv_bfloat16 *r = p.R + row * p.ldr + col;
    v.x += __bfloat162float(r[0]);
    if (n > 1) v.y += __bfloat162float(r[1]);
    if (n > 2) v.z += __bfloat162float(r[2]);
    if (n > 3) v.w += __bfloat162float(r[3]);
  }
  store4(p.Y + row * p.ldy + col, v, n);
}

template <bool GATED, bool W_MN, int NT, bool TWO>
__global__ void __launch_bounds__(FTHREADS, Few<GATED, NT, TWO>::PER_SM)
    dense_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                     const __grid_constant__ CUtensorMap tmX2,
                     const __grid_constant__ CUtensorMap tmW2, const FewP fp) {
  using C = Few<GATED, NT, TWO>;
  const DenseP &p = fp.d;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto *ctl = reinterpret_cast<FewCtl<C::STAGES> *>(smem + C::STAGES * C::STAGE);
  static_assert(sizeof(*ctl) <= 256, "control block");
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int split = fp.split, rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t tile = blockIdx.x / split;
  const int64_t t0 = tile % fp.tiles_t * NT, f0 = tile / fp.tiles_t * DT;
  // this CTA's k-slabs
  const int nk = p.nk1 * p.nseg, base = nk / split, extra = nk % split;
  const int kb = rank * base + (rank < extra ? rank : extra), cnt = base + (rank < extra ? 1 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    mbar_init(&ctl->done, 1);
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, C::COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ctl->tmem_base;
  volatile int *abort = &ctl->abort;
  pdl_launch();
  pdl_wait();

  int issued = 0;
  if (warp == 0 && elect_one()) {
    for (int it = 0; it < cnt; ++it) {
      const int s = it % C::STAGES;
      if (it >= C::STAGES && !mbar_wait(&ctl->empty[s], ((it / C::STAGES) - 1) & 1, abort)) break;
      uint8_t *st = smem + s * C::STAGE;
      const int kt = kb + it;
      const bool second = kt >= p.nk1;
      const int32_t k0 = (second ? kt - p.nk1 : kt) * DBK;
      mbar_expect_tx(&ctl->full[s], C::STAGE);
      load_panel(st, !GATED && second ? &tmW2 : &tmW, &ctl->full[s], W_MN,
                 static_cast<int32_t>(f0), k0);
      if (GATED) load_panel(st + DPANEL, &tmW2, &ctl->full[s], W_MN, static_cast<int32_t>(f0), k0);
      tma_load_2d(st + DPANEL * (GATED ? 2 : 1), second ? &tmX2 : &tmX, &ctl->full[s], k0,
                  static_cast<int32_t>(t0));
      issued = it + 1;
    }
  } else if (warp == 1 && elect_one()) {
    const uint32_t idesc = idesc_make(1, W_MN, 0, DT, NT);
    const uint32_t w0 = smem_u32(smem), x0 = w0 + DPANEL * (GATED ? 2 : 1);
    const uint64_t dw0 = W_MN ? sdesc_sw128(w0, DBOX, 1024) : sdesc_sw128(w0, 16, 1024);
    const uint64_t dx0 = sdesc_sw128(x0, 16, 1024);
    // (the next slab's barrier is tested before this one's MMAs: see the pair
    // kernel)
    bool ok = true, landed = false;
    int s = 0;
    uint32_t parity = 0;
    for (int it = 0; it < cnt; ++it) {
      if (!landed && !mbar_wait(&ctl->full[s], parity, abort)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t at = s * (C::STAGE >> 4);
      uint64_t *used = &ctl->empty[s];
      if (++s == C::STAGES) s = 0, parity ^= 1;
      landed = mbar_try_wait(&ctl->full[s], parity);
#pragma unroll
      for (int kk = 0; kk < DBK / 16; ++kk) {
#pragma unroll
        for (int h = 0; h < (GATED ? 2 : 1); ++h)
          umma_bf16(tbase + NT * h, dw0 + at + h * (DPANEL >> 4) + kk * (W_MN ? 128 : 2),
                    dx0 + at + kk * 2, idesc, (it | kk) != 0);
      }
      umma_commit(used);
    }
    if (ok) umma_commit(&ctl->done);
  }
  __syncwarp();

  // ---- this CTA's part of the tile -> shared memory (the ring is free: every
  // slab has landed and been multiplied)
  float *part = reinterpret_cast<float *>(smem);
  {
    const bool ok = mbar_wait(&ctl->done, 0, abort);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const int feat = 32 * warp + lane;
#pragma unroll
      for (int h = 0; h < (GATED ? 2 : 1); ++h) {
        for (int c = 0; c < NT; c += NT < 32 ? 16 : 32) {
          constexpr int W = NT < 32 ? 16 : 32;
          if (t0 + c >= p.M) break;
          float v[W];
          const uint32_t ta = tbase + (static_cast<uint32_t>(32 * warp) << 16) + NT * h + c;
          if constexpr (W == 16) tmem_ld16(ta, v);
          else tmem_ld32(ta, v);
#pragma unroll
          for (int t = 0; t < W; ++t) part[(NT * h + c + t) * DT + feat] = v[t];
        }
      }
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync_all();
  else __syncthreads();

  // ---- sum over the parts, epilogue: four features of a token per step, every
  // part's loads of U steps in flight together
  const int tokens = static_cast<int>(kq_min<int64_t>(NT, p.M - t0));
  const int items = tokens * (DT / 4), stride = split * FTHREADS;
  constexpr int U = NT <= 32 ? 1 : 2;
  if (!*abort) {
#pragma unroll 1
    for (int e0 = rank * FTHREADS + threadIdx.x; e0 < items; e0 += U * stride) {
      float4 v[U], u[U];
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int r0 = 0; r0 < split; r0 += 4) {   // four parts at a time
        float4 x[4][U], y[4][GATED ? U : 1];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int o = kq_min(r0 + r, split - 1);
          const uint32_t base = split > 1 ? mapa_shared(smem_u32(part), o) : smem_u32(part);
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int e = kq_min(e0 + k * stride, items - 1);   // (token, features) e
            x[r][k] = ld_dsmem_f4(base + static_cast<uint32_t>(e) * 16);
            if constexpr (GATED)
              y[r][k] = ld_dsmem_f4(base + static_cast<uint32_t>(e) * 16 + NT * DT * 4);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < U; ++k) {
            v[k] = add4(v[k], r0 + r < split ? x[r][k] : zero);
            if constexpr (GATED) u[k] = add4(u[k], r0 + r < split ? y[r][k] : zero);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int e = e0 + k * stride, t = e / (DT / 4);
        const int64_t col = f0 + e % (DT / 4) * 4;
        if (e >= items || col >= p.N) continue;
        const int n = static_cast<int>(kq_min<int64_t>(4, p.N - col));
        if (!GATED && p.bias) {
          v[k].x += p.bias[col];
          if (n > 1) v[k].y += p.bias[col + 1];
          if (n > 2) v[k].z += p.bias[col + 2];
          if (n > 3) v[k].w += p.bias[col + 3];
        }
        finish4<GATED>(p, t0 + t, col, n, v[k], u[k]);
      }
    }
  }
  // no CTA leaves while another may still read its part
  __syncwarp();
  if (split > 1) cluster_sync_all();
  else __syncthreads();

  // ---- teardown: after an abort make sure no copy or MMA is still in flight
  if (ctl->abort) {
    if (threadIdx.x == 0) report(p.info, KRONQ_ERR_TIMEOUT);
    // (the same lanes are elected again)
    if (warp == 0 && elect_one()) {
      const uint64_t c0 = globaltimer();
      for (int s = 0; s < C::STAGES && s < issued; ++s) {
        const int last = ((issued - 1 - s) / C::STAGES) * C::STAGES + s;
        while (!mbar_try_wait(&ctl->full[s], (last / C::STAGES) & 1) &&
               globaltimer() - c0 < kWaitLimitNs) {
        }
      }
    }
    if (warp == 1 && elect_one()) {
      umma_commit(&ctl->drain);
      const uint64_t c0 = globaltimer();
      while (!mbar_try_wait(&ctl->drain, 0) && globaltimer() - c0 < kWaitLimitNs) {
      }
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, C::COLS);
  }
}

// ---------------------------------------------------------------- CTA pairs
// The same products on CTA pairs, for many rows: a cluster of two CTAs owns a
// tile of D of 256 rows and NB = 256, 192 or 128 columns (gated: NB / 2 columns of
// both products). Each CTA holds 128 rows of A and NB / 2 of B's (gated: the
// even CTA Wg's, the odd one Wu's), so at 256 columns a k-slab of 64 costs a CTA
// 32 KB of shared memory for 128 x 256 x 64 products: half of what one CTA
// alone would load. The kernel is persistent: TMEM holds two accumulators,
// and the epilogue of one tile runs while the next one accumulates.
//   Bound by the tensor cores: 4096 tokens 4096 -> 11008 with its gated pair takes
// 570 us (1.30 PFLOP/s, at the power cap, 1.23 GHz), and in the input gradient of
// 2048 tokens of that pair the tensor pipe is active for 96 % of an SM's cycles.
//   warps 0..7  epilogue: warp w takes TMEM lanes 32 (w % 4) .. + 31 (rows) and
//               half w / 4 of the tile's columns, 64 at a time: two slots of 4 KB
//               collect 32 rows x 64 columns of an output, which one TMA store
//               takes out (stores straight from the row-per-lane registers
//               touch 32 rows an instruction and took 5000 cycles a tile).
//               Residual values come into the same slot by asynchronous
//               copies, the first before the accumulator is ready.
//   warp 8      TMA producer (each CTA loads its own panels; the bytes of both
//               are counted on the even CTA's barrier)
//   warp 9      TMEM owner; in the even CTA the MMA issuer
constexpr int PTHREADS = 320;
constexpr int PGROUP = 8;                // tile raster: row tiles per band
constexpr int PSLOT = 32 * 128;          // staging slot: 32 rows of 64 bf16

template <int STAGES>
struct PairCtl {
  uint64_t full[STAGES];     // both CTAs' panels landed (even CTA's is used)
  uint64_t empty[STAGES];    // MMAs that read the stage finished (both CTAs)
  uint64_t tfull[2];         // accumulator complete (both CTAs)
  uint64_t tempty[2];        // read out by both CTAs' epilogues (even CTA's)
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// NB: columns of the accumulator. A CTA's stage: 128 rows of A, NB / 2 of B.
template <int NB>
struct Pair {
  static constexpr int STAGE = DPANEL + (NB > 128 ? DPANEL : DPANEL / 2);
  static constexpr int STAGES = NB > 128 ? 5 : 6;
  // bytes of B that land in a CTA's stage: MN-major panels come in 64-wide boxes
  static constexpr int BYTES_K = NB / 2 * 128, BYTES_MN = (NB / 2 + 63) / 64 * 64 * 128;
  static constexpr int TMEM = NB > 128 ? 512 : 256;
  static constexpr int SMEM = STAGES * STAGE + 16 * PSLOT + 1024 + int(sizeof(PairCtl<STAGES>)) + 64;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(STAGES * STAGE >= 128 * NB * 4, "the partial sums fit in the ring");
};

// Output maps of the pair kernel: Y, and the kept pre-activations.
struct OutMaps {
  CUtensorMap y, z, z2;
};

// Columns [32 h, 32 h + 32) of lane's row in a staging slot (128-byte rows,
// 16-byte granules swizzled by the row's low bits, as the TMA maps have it).
__device__ __forceinline__ void stage32(uint8_t *slot, int lane, int h, const float *v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 o;
    __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
    for (int t = 0; t < 4; ++t) b[t] = __floats2bfloat162_rn(v[8 * j + 2 * t], v[8 * j + 2 * t + 1]);
    *reinterpret_cast<uint4 *>(slot + lane * 128 + ((4 * h + j) ^ (lane & 7)) * 16) = o;
  }
}
__device__ __forceinline__ void add_staged32(const uint8_t *slot, int lane, int h, float *v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 o =
        *reinterpret_cast<const uint4 *>(slot + lane * 128 + ((4 * h + j) ^ (lane & 7)) * 16);
    const __nv_bfloat162 *b = reinterpret_cast<const __nv_bfloat162 *>(&o);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float2 f = __bfloat1622float2(b[t]);
      v[8 * j + 2 * t] += f.x;
      v[8 * j + 2 * t + 1] += f.y;
    }
  }
}
// Takes a staged slot out to (col, row) of an M x N matrix; the slot is free
// again after slot_free. A TMA store leaves out what lies outside its map in
// whole 16-byte granules only, so the maps end at the last multiple of 8
// columns, and the lanes write their rows' last N % 8 columns themselves.
__device__ __forceinline__ void slot_out(const CUtensorMap *map, __nv_bfloat16 *y, int64_t ld,
                                         int64_t M, int64_t N, const uint8_t *slot, int lane,
                                         int64_t col, int64_t row) {
  fence_proxy_async_smem();
  __syncwarp();
  const int64_t n8 = N & ~int64_t(7);
  if (lane == 0) {   // (a group for every slot, empty or not: slot_free counts them)
    if (col < n8) tma_store_2d(map, slot, static_cast<int32_t>(col), static_cast<int32_t>(row));
    bulk_commit();
  }
  if (n8 < N && n8 - col < 64 && n8 >= col && row + lane < M) {
    const int j = static_cast<int>(n8 - col) / 8;
    const __nv_bfloat16 *v =
        reinterpret_cast<const __nv_bfloat16 *>(slot + lane * 128 + (j ^ (lane & 7)) * 16);
    for (int t = 0; t < N - n8; ++t) y[(row + lane) * ld + n8 + t] = v[t];
  }
}
// Waits until all but the warp's last store (ALL: every store) have read their
// slots.
template <bool ALL>
__device__ __forceinline__ void slot_free(int lane) {
  if (lane == 0) {
    if constexpr (ALL) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
  }
  __syncwarp();
}

template <int ROWS>
__device__ __forceinline__ void load_panel_pair(uint8_t *dst, const CUtensorMap *map,
                                                uint32_t bar, bool mn, int32_t r0, int32_t k0) {
  if (!mn) {
    tma_load_2d_pair(dst, map, bar, k0, r0);
  } else {
#pragma unroll
    for (int r = 0; r < ROWS; r += 64)
      tma_load_2d_pair(dst + r / 64 * DBOX, map, bar, r0 + r, k0);
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

// With few tiles (S > 1) the k range of a tile is divided over the S pairs of a
// larger cluster: every CTA writes its 128 x NB partial sums to the ring's shared
// memory (NB = 128: 64 KB of fp32, 16-byte granules swizzled by the row), and
// after a cluster barrier each pair sums and finishes its share of the columns
// over all parts, in the order of their ranks, through distributed shared
// memory. One tile a cluster.
template <bool GATED, int ACT, bool A_MN, bool B_MN, int S, int NB>
__global__ void __launch_bounds__(PTHREADS, 1)
    dense_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmA2,
                      const __grid_constant__ CUtensorMap tmB2,
                      const __grid_constant__ OutMaps out, const DenseP p) {
  using C = Pair<NB>;
  constexpr int NT = GATED ? NB / 2 : NB;   // columns of the output per tile
  constexpr int PSTAGES = C::STAGES, PSTAGE = C::STAGE;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto *ctl = reinterpret_cast<PairCtl<PSTAGES> *>(smem + PSTAGES * PSTAGE + 16 * PSLOT);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr bool SPLIT = S > 1;           // S pairs in the cluster
  // (broadcasts tell the compiler that the values are the same in a warp)
  const int crank = __shfl_sync(0xffffffffu, static_cast<int>(cluster_ctarank()), 0);
  const int rank = crank & 1, part = SPLIT ? crank >> 1 : 0, leader = crank & ~1;
  const int64_t cluster = __shfl_sync(0xffffffffu, static_cast<int>(cluster_id_x()), 0);
  const int64_t clusters = gridDim.x / (2 * S);
  const int tiles_n = static_cast<int>((p.N + NT - 1) / NT);
  const int64_t tiles = int64_t(p.tiles_m) * tiles_n;
  const int nk_all = p.nk1 * p.nseg, kb = SPLIT ? nk_all * part / S : 0;
  const int nk = SPLIT ? nk_all * (part + 1) / S - kb : nk_all;   // this pair's k-slabs

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
  if (warp == 9) tmem_alloc_pair(&ctl->tmem_base, C::TMEM);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tbase = ctl->tmem_base;
  volatile int *abort = &ctl->abort;
  pdl_launch();
  pdl_wait();

  // ring position: slot s, and the parity of its current round
  uint32_t issued = 0;
  if (warp == 8) {
    if (elect_one()) {
      int s = 0;
      uint32_t round = 0;
      bool ok = true;
      const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), leader);
      for (int64_t t = cluster; t < tiles && ok; t += clusters) {
        int64_t bi, bj;
        pair_tile(t, p.tiles_m, tiles_n, bi, bj);
        const int32_t m0 = static_cast<int32_t>(bi * 256 + 128 * rank);
        const int32_t n0 = static_cast<int32_t>(bj * NT + (GATED ? 0 : NB / 2 * rank));
        for (int it = 0; it < nk; ++it) {
          if (round > 0 && !mbar_wait(&ctl->empty[s], (round - 1) & 1, abort)) {
            ok = false;
            break;
          }
          uint8_t *st = smem + s * PSTAGE;
          const bool second = kb + it >= p.nk1;
          const int32_t k0 = (second ? kb + it - p.nk1 : kb + it) * DBK;
          const uint32_t bar = full0 + s * 8;
          if (rank == 0) mbar_expect_tx(&ctl->full[s], 2 * (DPANEL + (B_MN ? C::BYTES_MN : C::BYTES_K)));
          load_panel_pair<128>(st, second ? &tmA2 : &tmA, bar, A_MN, m0, k0);
          load_panel_pair<NB / 2>(st + DPANEL, (GATED ? rank != 0 : second) ? &tmB2 : &tmB, bar,
                                  B_MN, n0, k0);
          ++issued;
          if (++s == PSTAGES) s = 0, ++round;
        }
      }
      // every arrival on this CTA's barriers has landed before the CTA ends
      for (uint32_t e = issued > PSTAGES ? issued - PSTAGES : 0; e < issued && ok; ++e)
        ok = mbar_wait(&ctl->empty[e % PSTAGES], (e / PSTAGES) & 1, abort);
    }
  } else if (warp == 9) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_make(1, A_MN, B_MN, 256, NB);
      // descriptors of slot 0's first step; others differ in the address field
      const uint32_t a0 = smem_u32(smem), b0 = a0 + DPANEL;
      const uint64_t da0 = A_MN ? sdesc_sw128(a0, DBOX, 1024) : sdesc_sw128(a0, 16, 1024);
      const uint64_t db0 = B_MN ? sdesc_sw128(b0, DBOX, 1024) : sdesc_sw128(b0, 16, 1024);
      // Measured per slab of four 256 x 128 MMAs (260 cycles of tensor work): 335
      // cycles with the barrier wait between the slabs, 264 with the next slab's
      // barrier tested before this one's MMAs, so that only a slab that is late is
      // waited for.
      int s = 0, i = 0;
      uint32_t parity = 0;
      bool ok = true, landed = false;
      for (int64_t t = cluster; t < tiles && ok; t += clusters, ++i) {
        const int a = i & 1;
        if (i >= 2 && !mbar_wait(&ctl->tempty[a], ((i >> 1) - 1) & 1, abort)) break;
        for (int it = 0; it < nk; ++it) {
          if (!landed && !mbar_wait(&ctl->full[s], parity, abort)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = s * (PSTAGE >> 4);
          uint64_t *used = &ctl->empty[s];
          if (++s == PSTAGES) s = 0, parity ^= 1;
          landed = mbar_try_wait(&ctl->full[s], parity);
#pragma unroll
          for (int kk = 0; kk < DBK / 16; ++kk)
            umma_bf16_pair(tbase + NB * a, da0 + at + kk * (A_MN ? 128 : 2),
                           db0 + at + kk * (B_MN ? 128 : 2), idesc, (it | kk) != 0);
          umma_commit_pair(used, leader);
        }
        if (ok) umma_commit_pair(&ctl->tfull[a], leader);
      }
    }
  } else {
    const int q = warp & 3, half = warp >> 2;
    uint8_t *slots = smem + PSTAGES * PSTAGE + 2 * warp * PSLOT;
    if constexpr (SPLIT) {
      const bool ok = mbar_wait(&ctl->tfull[0], 0, abort);
      const bool alive = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t tq = tbase + (static_cast<uint32_t>(32 * q) << 16);
      if (alive) {   // this CTA's part -> shared memory
        const int r = 32 * q + lane;
        for (int c = NB / 2 * half; c < NB / 2 * (half + 1); c += 32) {
          float v[32];
          tmem_ld32(tq + c, v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4 *>(smem + r * (NB * 4) + ((c / 4 + j) ^ (r & 7)) * 16) =
                make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      cluster_sync_all();
      // four columns a lane, whole row segments a warp (remote reads and
      // global stores of 256 bytes and more), 16 rows a warp in two batches
      int64_t bi, bj;
      pair_tile(cluster, p.tiles_m, tiles_n, bi, bj);
      constexpr int WIDTH = NT / S, PER_ROW = WIDTH / 4, STEP = 32 / PER_ROW;
      // rows in flight: up to 8 loads a lane
      constexpr int U = 8 / (S * (GATED ? 2 : 1)) < 16 / STEP ? 8 / (S * (GATED ? 2 : 1)) : 16 / STEP;
      const int cc = WIDTH * part + lane % PER_ROW * 4;
      const int64_t col = bj * NT + cc, row0 = bi * 256 + 128 * rank;
      const int n = static_cast<int>(kq_max<int64_t>(kq_min<int64_t>(4, p.N - col), 0));
      float4 bias = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!GATED && p.bias && n > 0) {
        bias.x = p.bias[col];
        if (n > 1) bias.y = p.bias[col + 1];
        if (n > 2) bias.z = p.bias[col + 2];
        if (n > 3) bias.w = p.bias[col + 3];
      }
#pragma unroll 1
      for (int r0 = warp * 16 + lane / PER_ROW; r0 < warp * 16 + 16 && alive && n > 0;
           r0 += U * STEP) {
        float4 x[S][U], y[S][GATED ? U : 1];
#pragma unroll
        for (int o = 0; o < S; ++o) {
          const uint32_t base = mapa_shared(smem_u32(smem), 2 * o + rank);
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int r = kq_min(r0 + k * STEP, 127);
            x[o][k] = ld_dsmem_f4(base + r * (NB * 4) + ((cc / 4) ^ (r & 7)) * 16);
            if constexpr (GATED)
              y[o][k] = ld_dsmem_f4(base + r * (NB * 4) + ((cc / 4 + NB / 8) ^ (r & 7)) * 16);
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int r = r0 + k * STEP;
          const int64_t row = row0 + r;
          if (r >= warp * 16 + 16 || row >= p.M) continue;
          float4 v = x[0][k], u = y[0][GATED ? k : 0];
#pragma unroll
          for (int o = 1; o < S; ++o) {
            v = add4(v, x[o][k]);
            if constexpr (GATED) u = add4(u, y[o][k]);
          }
          finish4<GATED>(p, row, col, n, add4(v, bias), u);
        }
      }
    }
    uint32_t used = 0;   // outputs taken out so far: they use the two slots in turn
    int i = 0;
    for (int64_t t = cluster; t < tiles && !SPLIT; t += clusters, ++i) {
      const int a = i & 1;
      int64_t bi, bj;
      pair_tile(t, p.tiles_m, tiles_n, bi, bj);
      const int64_t row0 = bi * 256 + 128 * rank + 32 * q;   // this warp's rows
      const uint32_t tq = tbase + (static_cast<uint32_t>(32 * q) << 16) + NB * a;
      // residual values of columns [col, col + 64) into a slot
      auto residual = [&](uint8_t *slot, int64_t col) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + (lane >> 3), j = lane & 7;
          const int64_t row = row0 + r, c = col + 8 * j;
          const int bytes =
              row < p.M ? static_cast<int>(kq_max<int64_t>(kq_min<int64_t>(p.N - c, 8), 0)) * 2 : 0;
          cp_async16(smem_u32(slot + r * 128 + (j ^ (r & 7)) * 16),
                     bytes > 0 ? p.R + row * p.ldr + c : p.R, bytes);
        }
      };
      // slots of 64 columns of this half: the first half takes the odd one
      constexpr int SLOTS = NT / 64, FIRST = (SLOTS + 1) / 2;
      const int mine = half == 0 ? FIRST : SLOTS - FIRST, first = half * FIRST * 64;
      const bool busy = mine > 0;
      // The first output takes R. Only if there is one: what lies outside the
      // matrix is left without waiting for its copies, and those of the next tile
      // to the same slot are not ordered behind them.
      const bool early = !GATED && busy && p.R && !p.Z && bj * NT + first < p.N && row0 < p.M;
      if (early) {
        slot_free<false>(lane);
        residual(slots + (used & 1) * PSLOT, bj * NT + first);
      }
      // the bias of this half's columns, 32 a register, before it is needed
      constexpr int BREGS = GATED ? 1 : 2 * FIRST;
      float bias[BREGS];
      if constexpr (!GATED) {
#pragma unroll
        for (int k = 0; k < BREGS; ++k) {
          const int64_t col = bj * NT + first + 32 * k + lane;
          bias[k] = p.bias && k < 2 * mine && col < p.N ? p.bias[col] : 0.f;
        }
      }
      const bool ok = mbar_wait(&ctl->tfull[a], (i >> 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      for (int c = 0; c < mine; ++c) {
        const int cc = first + 64 * c;
        const int64_t col = bj * NT + cc;
        if (col >= p.N || row0 >= p.M) break;
        if (GATED && p.Z) {
#pragma unroll 1
          for (int o = 0; o < 2; ++o) {
            uint8_t *slot = slots + (used++ & 1) * PSLOT;
            slot_free<false>(lane);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float v[32];
              tmem_ld32(tq + cc + NB / 2 * o + 32 * h, v);
              stage32(slot, lane, h, v);
            }
            slot_out(o ? &out.z2 : &out.z, o ? p.Z2 : p.Z, p.ldz, p.M, p.N, slot, lane, col, row0);
          }
        }
        // (Z of a linear product goes out beside Y, through the other slot)
        const bool keep = !GATED && p.Z;
        uint8_t *zslot = slots + (used & 1) * PSLOT;
        if (keep) {
          ++used;
          slot_free<true>(lane);
        }
        uint8_t *slot = slots + (used++ & 1) * PSLOT;
        if (!early || c > 0) {
          if (!keep) slot_free<false>(lane);
          if (!GATED && p.R) residual(slot, col);
        }
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[32], u[GATED ? 32 : 1];
          tmem_ld32(tq + cc + 32 * h, v);
          if constexpr (GATED) tmem_ld32(tq + cc + NB / 2 + 32 * h, u);
          if constexpr (!GATED) {
            if (p.bias) {
              float bl = bias[0];
#pragma unroll
              for (int k = 1; k < BREGS; ++k) bl = 2 * c + h == k ? bias[k] : bl;
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] += __shfl_sync(0xffffffffu, bl, k);
            }
          }
          if (keep) stage32(zslot, lane, h, v);
#pragma unroll
          for (int k = 0; k < 32; ++k) v[k] = act_f<ACT>(v[k]);
          if constexpr (GATED) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= u[k];
          }
          if (!GATED && p.R) {
            if (h == 0) {
              cp_async_wait();
              __syncwarp();
            }
            add_staged32(slot, lane, h, v);
          }
          stage32(slot, lane, h, v);
        }
        if (keep) slot_out(&out.z, p.Z, p.ldz, p.M, p.N, zslot, lane, col, row0);
        slot_out(&out.y, p.Y, p.ldy, p.M, p.N, slot, lane, col, row0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->tempty[a]), leader));
    }
    // the slots are read before the CTA ends (the stores complete with the grid)
    cp_async_wait();
    slot_free<true>(lane);
  }

  __syncwarp();
  if (SPLIT && warp >= 8) cluster_sync_all();   // the parts are written

  // ---- teardown: after an abort make sure no copy or MMA is still in flight
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (ctl->abort) {
    if (threadIdx.x == 0) report(p.info, KRONQ_ERR_TIMEOUT);
    // (the same lanes are elected again)
    if (rank == 0 && warp == 8 && elect_one()) {
      const uint64_t t0 = globaltimer();
      for (uint32_t s = 0; s < PSTAGES && s < issued; ++s) {
        const uint32_t last = ((issued - 1 - s) / PSTAGES) * PSTAGES + s;
        while (!mbar_try_wait(&ctl->full[s], (last / PSTAGES) & 1) &&
               globaltimer() - t0 < kWaitLimitNs) {
        }
      }
    }
    if (rank == 0 && warp == 9 && elect_one()) {
      umma_commit_pair(&ctl->drain, leader);
      const uint64_t t0 = globaltimer();
      while (!mbar_try_wait(&ctl->drain, 0) && globaltimer() - t0 < kWaitLimitNs) {
      }
    }
  }
  __syncwarp();
  cluster_sync_all();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, C::TMEM);
  }
}

// dZ = dY * act'(Z), or the gated pair's Gg and Gu, eight columns a thread.
// Every element is read before it is written by the same thread, so an output
// may be one of the inputs. Bound by memory: the gated pair's 4096 x 11008 take
// 73 us (6.2 TB/s), 4096 x 4096 with relu 17.2 us.
struct ActBwdP {
  int64_t n, w;
  const __nv_bfloat16 *dY, *Z, *U;
  int64_t lddy, ldz;
  __nv_bfloat16 *G, *G2;
  int64_t ldg;
};

// eight bf16 numbers, those from the n-th on 0
__device__ __forceinline__ uint4 load8_raw(const __nv_bfloat16 *p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint4 *>(p);
  uint32_t o[4] = {0, 0, 0, 0};
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if (t < n) o[t / 2] |= uint32_t(__bfloat16_as_ushort(p[t])) << (16 * (t & 1));
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void unpack8(const uint4 &o, float *v) {
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&o);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float2 f = __bfloat1622float2(h[t]);
    v[2 * t] = f.x;
    v[2 * t + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *v, int n) {
  unpack8(load8_raw(p, n), v);
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

// The same with db = column sums of dZ before its rounding: a cluster of CTAs
// owns 64 columns, each of its CTAs every (cluster size)-th band of 32 rows;
// a thread sums 8 columns of its rows, and the threads and then the CTAs meet
// in a fixed order (the first CTA reads the others' sums through distributed
// shared memory). Bound by reading dY and Z and writing dZ once: 4096 x 4096 with
// relu take 19.5 us (5.2 TB/s), with gelu 31.1 us, bound by its instructions; a wave
// and a half of CTAs costs more than fewer parts (2048 x 11008 25.2 us in three parts,
// 31.5 in eight).
constexpr int BG_MAXC = 8;
template <int ACT>
__global__ void __launch_bounds__(256, 4) bias_grad_kernel(const ActBwdP p, float *db, int parts) {
  __shared__ __align__(16) float part[32][64];
  const int cg = threadIdx.x & 7, rl = threadIdx.x >> 3;
  const int rank = blockIdx.x % parts;
  const int64_t c = blockIdx.x / parts * int64_t(64) + 8 * cg;
  const int n = static_cast<int>(kq_max<int64_t>(kq_min<int64_t>(8, p.w - c), 0));
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (n > 0) {
    const int64_t step = 32 * parts;
    constexpr int U = 3;   // rows in flight (64 registers: four CTAs an SM)
    for (int64_t r0 = rank * 32 + rl; r0 < p.n; r0 += U * step) {
      uint4 gr[U], zr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * step;
        if (r >= p.n) continue;
        gr[u] = load8_raw(p.dY + r * p.lddy + c, n);
        if (ACT != KRONQ_ACT_NONE) zr[u] = load8_raw(p.Z + r * p.ldz + c, n);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * step;
        if (r >= p.n) continue;
        float g[8], z[8];
        unpack8(gr[u], g);
        if (ACT != KRONQ_ACT_NONE) unpack8(zr[u], z);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          if (ACT != KRONQ_ACT_NONE) {
            float h, dh;
            act_df<ACT>(z[t], h, dh);
            g[t] *= dh;
          }
          sum[t] += g[t];
        }
        if (p.G) store8(p.G + r * p.ldg + c, g, n);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) part[rl][8 * cg + t] = sum[t];
  __syncthreads();
  if (threadIdx.x < 64) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += part[k][threadIdx.x];
    part[0][threadIdx.x] = s;   // only this thread reads the column
  }
  if (parts > 1) {
    __syncwarp();
    cluster_sync_all();
  } else {
    __syncthreads();
  }
  const int64_t col = blockIdx.x / parts * int64_t(64) + 4 * threadIdx.x;
  if (rank == 0 && threadIdx.x < 16 && col < p.w) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < parts; ++k) {
      const uint32_t at = smem_u32(&part[0][4 * threadIdx.x]);
      const float4 v = ld_dsmem_f4(parts > 1 ? mapa_shared(at, k) : at);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int t = 0; t < 4; ++t)
      if (col + t < p.w) db[col + t] = v[t];
  }
  __syncwarp();
  if (parts > 1) cluster_sync_all();   // the others' sums stay until they are read
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
                         int64_t K, int box_rows) {
  return mn ? make_tmap_2d(m, p, true, rows, K, ld, 64, DBK)
            : make_tmap_2d(m, p, true, K, rows, ld, DBK, box_rows);
}

// How many clusters of n CTAs are on the chip at once: they do not reach over the
// groups of SMs it is made of, some of which have fewer SMs.
int resident_clusters(int per_sm, int n) {
  static constexpr int one[9] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
  static constexpr int two[9] = {0, 296, 148, 93, 71, 56, 45, 34, 33};
  return per_sm == 2 ? two[n] : one[n];
}

// The few-token kernel splits k over the CTAs of a cluster, as many as leave two
// slabs each and are all on the chip at once: one token 4096 -> 5120 (40 tiles) takes
// 9.7 us in six parts and 13.9 in seven, of which 34 clusters are on the chip. Five
// to seven parts pay for one tile of 16 tokens only: 64 tokens 4096 -> 6016 take 17.8
// in five, 14.7 in four (the sums of the parts are shared out evenly over four).
template <bool GATED, bool W_MN, int NT, bool TWO = false>
kronq_status launch_few(cudaStream_t st, const CUtensorMap *tm, const DenseP &d, int act) {
  using C = Few<GATED, NT, TWO>;
  auto *kern = dense_few_kernel<GATED, W_MN, NT, TWO>;
  KQ_TRY(smem_attr(kern, C::SMEM));
  FewP p;
  p.d = d;
  p.d.act = act;
  p.tiles_t = static_cast<int>(ceil_div(d.M, NT));
  const int64_t tiles = p.tiles_t * ceil_div(d.N, DT);
  p.split = static_cast<int>(
      kq_min<int64_t>(kq_min<int64_t>(8, 148 * C::PER_SM / tiles), d.nk1 * d.nseg / 2));
  while (p.split > 1 && (tiles > resident_clusters(C::PER_SM, p.split) ||
                         (NT > 16 && p.split > 4 && p.split < 8)))
    --p.split;
  p.split = kq_max(p.split, 1);
  return launch_kernel(st, kern, tiles * p.split, FTHREADS, C::SMEM, p.split, true, tm[0], tm[1],
                       tm[2], tm[3], p);
}

// How a product runs on pairs: columns of the accumulator and pairs a tile.
//   A round of 74 pairs takes about nk * 520 + 6000 cycles at 256 columns,
// nk * 440 + 5500 at 192 (480 with B MN-major, whose panels of 96 rows load as 128)
// and nk * 320 + 5000 at 128 (nk slabs of k): tiles are as wide as the number of
// rounds lets them. Measured (us, 256 | 192 columns): 2000 tokens 3000 -> 5000 66.9 |
// 63.8, its input gradient 80.2 | 73.3, 304 tokens 2504 -> 10000 40.0 | 33.1, but 4096
// tokens 4096 -> 4096 111.7 | 115.7.
//   Where a single round leaves pairs idle, k is split over two or four of them if
// the clusters that takes all fit on the chip (33 of four CTAs of this size, 15 of
// eight) and enough slabs remain each: 256 tokens 4096 -> 4096 take 15.2 us in two
// parts and 19.3 in one, 200 tokens 8192 -> 1024 11.7 in four and 26.0 in one, but
// 250 tokens 1024 -> 1024 7.0 in two and 6.5 in one.
struct PairPlan {
  int nb, split;
};
PairPlan pair_plan(int64_t rows, int64_t cols, int nk, bool gated, bool b_mn) {
  const int64_t tm = ceil_div(rows, 256);
  const int64_t wide = tm * ceil_div(cols, gated ? 128 : 256);
  const int64_t narrow = tm * ceil_div(cols, gated ? 64 : 128);
  if (narrow <= 15 && nk >= 32) return {128, 4};
  if (narrow <= 33 && nk >= 20) return {128, 2};
  const int64_t c256 = ceil_div(wide, 74) * (int64_t(nk) * 520 + 6000);
  const int64_t c192 = ceil_div(tm * ceil_div(cols, 192), 74) * (int64_t(nk) * (b_mn ? 480 : 440) + 5500);
  const int64_t c128 = ceil_div(narrow, 74) * (int64_t(nk) * 320 + 5000);
  if (!gated && c192 < c256 && c192 < c128) return {192, 1};   // (no gated tiles of 96)
  return {c128 < c256 ? 128 : 256, 1};
}

struct Operands {
  Mat X, W, X2, W2;
};

// D (M x N) = A B^T on pairs, A = (o.X, o.X2), B = (o.W, o.W2)
template <bool GATED, bool A_MN, bool B_MN>
kronq_status launch_pair(cudaStream_t st, const Operands &o, DenseP p, int act) {
  const PairPlan plan = pair_plan(p.M, p.N, p.nk1 * p.nseg, GATED, B_MN);
  CUtensorMap tm[4];
  memset(tm, 0, sizeof(tm));
  KQ_TRY(operand_map(&tm[0], o.X.p, o.X.ld, A_MN, p.M, p.K, 128));
  KQ_TRY(operand_map(&tm[1], o.W.p, o.W.ld, B_MN, p.N, p.K, plan.nb / 2));
  if (o.X2.p) KQ_TRY(operand_map(&tm[2], o.X2.p, o.X2.ld, A_MN, p.M, p.K, 128));
  if (o.W2.p) KQ_TRY(operand_map(&tm[3], o.W2.p, o.W2.ld, B_MN, p.N, p.K, plan.nb / 2));
  OutMaps out;
  memset(&out, 0, sizeof(out));
  const int64_t n8 = p.N & ~int64_t(7);
  if (n8 && plan.split == 1) {
    KQ_TRY(make_tmap_2d(&out.y, p.Y, true, n8, p.M, p.ldy, 64, 32));
    if (p.Z) KQ_TRY(make_tmap_2d(&out.z, p.Z, true, n8, p.M, p.ldz, 64, 32));
    if (p.Z2) KQ_TRY(make_tmap_2d(&out.z2, p.Z2, true, n8, p.M, p.ldz, 64, 32));
  }
  p.act = act;
  p.tiles_m = static_cast<int>(ceil_div(p.M, 256));
  auto go = [&](auto a, auto split, auto nb) {
    constexpr int S = decltype(split)::value, NB = decltype(nb)::value;
    auto *kern = dense_pair_kernel<GATED, decltype(a)::value, A_MN, B_MN, S, NB>;
    KQ_TRY(smem_attr(kern, Pair<NB>::SMEM));
    const int64_t tiles = p.tiles_m * ceil_div(p.N, GATED ? NB / 2 : NB);
    return launch_kernel(st, kern, 2 * S * (S > 1 ? tiles : kq_min<int64_t>(tiles, 74)), PTHREADS,
                         Pair<NB>::SMEM, 2 * S, true, tm[0], tm[1], tm[2], tm[3], out, p);
  };
  using I0 = std::integral_constant<int, KRONQ_ACT_NONE>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I4 = std::integral_constant<int, 4>;
  using N128 = std::integral_constant<int, 128>;
  using N192 = std::integral_constant<int, GATED ? 256 : 192>;
  using N256 = std::integral_constant<int, 256>;
  if (plan.split == 4) return go(I0(), I4(), N128());   // (split tiles: p.act)
  if (plan.split == 2) return go(I0(), I2(), N128());
  if constexpr (!A_MN && !B_MN) {
    return with_act(act, [&](auto a) {
      return plan.nb == 128   ? go(a, I1(), N128())
             : plan.nb == 192 ? go(a, I1(), N192())
                              : go(a, I1(), N256());
    });
  } else {
    return plan.nb == 128   ? go(I0(), I1(), N128())
           : plan.nb == 192 ? go(I0(), I1(), N192())
                            : go(I0(), I1(), N256());
  }
}

// Tokens per tile of the few-token kernel, 0 for the pair kernel. Above 64 tokens
// the few-token kernel's partial sums cost as much as the weights they save,
// unless K is long. Measured (us, few | pair), 128 tokens: 4096 -> 4096 13.0 | 14.6,
// 11008 -> 4096 22.7 | 27.6, 1024 -> 8192 10.9 | 7.7, 1352 -> 2008 15.6 | 9.1, and
// for the gated pair 4096 -> 2048 27.8 | 14.7, 1352 -> 1004 12.3 | 9.2; for the
// pair at 64 tokens 4096 -> 2048 21.2 | 14.2 (its 16 tiles fill too few SMs),
// 4096 -> 5504 22.1 | 27.1.
int few_width(int64_t tokens, int64_t N, int64_t K, bool gated) {
  if (tokens > 128 || (tokens > 64 && (gated || K < 4096))) return 0;
  if (gated && tokens > 32 && N < 4096) return 0;
  return tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
}

// D = X W^T by the kernel that takes it: few tokens, or pairs
template <bool GATED, bool W_MN>
kronq_status tokens_product(cudaStream_t st, const Operands &o, const DenseP &p, int act) {
  const int nt = few_width(p.M, p.N, p.K * p.nseg, GATED);
  if (nt == 0) return launch_pair<GATED, false, W_MN>(st, o, p, act);
  CUtensorMap tm[4];
  memset(tm, 0, sizeof(tm));
  KQ_TRY(operand_map(&tm[0], o.X.p, o.X.ld, false, p.M, p.K, nt));
  KQ_TRY(operand_map(&tm[1], o.W.p, o.W.ld, W_MN, p.N, p.K, DT));
  if (o.X2.p) KQ_TRY(operand_map(&tm[2], o.X2.p, o.X2.ld, false, p.M, p.K, nt));
  if (o.W2.p) KQ_TRY(operand_map(&tm[3], o.W2.p, o.W2.ld, W_MN, p.N, p.K, DT));
  switch (nt) {
    case 16: return launch_few<GATED, W_MN, 16>(st, tm, p, act);
    case 32: return launch_few<GATED, W_MN, 32>(st, tm, p, act);
    case 64: return launch_few<GATED, W_MN, 64>(st, tm, p, act);
  }
  // 128 tokens a tile: above 45 tiles one CTA an SM leaves too little to split. With
  // one | two an SM: 128 tokens 4096 -> 4096 12.9 | 14.8 us, 5120 15.4 | 17, 7424 19.9 |
  // 18.8, 11008 28.6 | 23.9.
  if constexpr (!GATED)
    return ceil_div(p.N, DT) > 45 ? launch_few<GATED, W_MN, 128, true>(st, tm, p, act)
                                  : launch_few<GATED, W_MN, 128>(st, tm, p, act);
  return KRONQ_ERR_UNSUPPORTED;   // (not reached)
}

// dX = G W (+ G2 W2) + R
kronq_status input_grad(cudaStream_t st, int64_t n, int64_t d_in, int64_t d_out,
                        const Operands &o, const Mat &R, const Mat &dX, int32_t *info) {
  DenseP p = {};
  p.M = n;
  p.N = d_in;
  p.K = d_out;
  p.nk1 = static_cast<int>(ceil_div(d_out, DBK));
  p.nseg = o.X2.p ? 2 : 1;
  p.R = static_cast<const __nv_bfloat16 *>(R.p);
  p.ldr = R.ld;
  p.Y = static_cast<__nv_bfloat16 *>(dX.p);
  p.ldy = dX.ld;
  p.info = info;
  return tokens_product<false, true>(st, o, p, KRONQ_ACT_NONE);
}

// dW = G^T X
kronq_status weight_grad(cudaStream_t st, int64_t n, int64_t d_in, int64_t d_out, const Mat &G,
                         const Mat &X, const Mat &dW, int32_t *info) {
  DenseP p = {};
  p.M = d_out;
  p.N = d_in;
  p.K = n;
  p.nk1 = static_cast<int>(ceil_div(n, DBK));
  p.nseg = 1;
  p.Y = static_cast<__nv_bfloat16 *>(dW.p);
  p.ldy = dW.ld;
  p.info = info;
  return launch_pair<false, true, true>(st, Operands{G, X, Mat{}, Mat{}}, p, KRONQ_ACT_NONE);
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
  DenseP p = {};
  p.M = n;
  p.N = d_out;
  p.K = d_in;
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
  return tokens_product<false, false>(st, Operands{X, W, Mat{}, Mat{}}, p, act);
}

kronq_status gated_fwd(cudaStream_t st, int64_t n, int64_t d, int64_t f, const Mat &X,
                       const Mat &Wg, const Mat &Wu, int act, const Mat &A, const Mat &U,
                       const Mat &H, int32_t *info) {
  DenseP p = {};
  p.M = n;
  p.N = f;
  p.K = d;
  p.nk1 = static_cast<int>(ceil_div(d, DBK));
  p.nseg = 1;
  p.Z = bf(A.p);
  p.Z2 = bf(U.p);
  p.ldz = A.ld;
  p.Y = bf(H.p);
  p.ldy = H.ld;
  p.info = info;
  return tokens_product<true, false>(st, Operands{X, Wg, Mat{}, Wu}, p, act);
}

// The products take dZ (below: Gg and Gu) as stored, rounded to bf16: that is the
// operand type of the tensor cores, and the sublayer's G that the caller gets. An fp32
// dZ would be a sum of two or three bf16 parts and as many products. It costs a second
// rounding: 4096 tokens of 4096 x 4096 are 2.3e-3 from the fp64 definition (norm of
// the error over the norm) where one rounding of the result alone is 1.7e-3.
kronq_status linear_bwd(cudaStream_t st, int64_t n, int64_t d_in, int64_t d_out, const Mat &dY,
                        const Mat &Z, int act, const Mat &X, const Mat &W, const Mat &dZ,
                        float *db, const Mat &dXr, const Mat &dX, const Mat &dW, int32_t *info) {
  if (n == 0) {
    if (db) KQ_CUDA(cudaMemsetAsync(db, 0, d_out * 4, st));
    return dW.p ? zero_rows(st, dW, d_out, d_in) : KRONQ_OK;
  }
  const bool write = act != KRONQ_ACT_NONE || (dZ.p && dZ.p != dY.p);
  if (db || write) {
    ActBwdP p = {};
    p.n = n;
    p.w = d_out;
    p.dY = bf(dY.p);
    p.lddy = dY.ld;
    p.Z = bf(Z.p);
    p.ldz = Z.ld;
    p.G = write ? bf(dZ.p) : nullptr;
    p.ldg = dZ.ld;
    KQ_TRY(with_act(act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
      if (!db) return launch_act_bwd<ACT, false>(st, p);
      // CTAs of a strip: three bands of rows each, and all strips on the chip at once
      const int64_t strips = ceil_div(d_out, 64);
      int parts = static_cast<int>(kq_min<int64_t>(BG_MAXC, ceil_div(n, 96)));
      while (parts > 1 && strips > 2 * resident_clusters(2, parts)) --parts;
      return launch_kernel(st, bias_grad_kernel<ACT>, strips * parts, 256, 0, parts,
                           false, p, db, parts);
    }));
  }
  const Mat G = write ? dZ : dY;
  if (dX.p)
    KQ_TRY(input_grad(st, n, d_in, d_out, Operands{G, W, Mat{}, Mat{}}, dXr, dX, info));
  if (dW.p) KQ_TRY(weight_grad(st, n, d_in, d_out, G, X, dW, info));
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
  if (dX.p) KQ_TRY(input_grad(st, n, d, f, Operands{Gg, Wg, Gu, Wu}, dXr, dX, info));
  if (dWg.p) {
    KQ_TRY(weight_grad(st, n, d, f, Gg, X, dWg, info));
    KQ_TRY(weight_grad(st, n, d, f, Gu, X, dWu, info));
  }
  return KRONQ_OK;
}

}  // namespace kronq
