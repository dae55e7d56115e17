// Distillation from a teacher's top logits, forward and backward. For a row
// of student logits z and the teacher's kept logits T at the places I:
//   p = softmax(T / tau),  q = softmax(z / tau),  lse = log sum exp(z / tau)
//   loss = tau^2 sum_j p_j (log p_j - z_{I_j} / tau + lse)
//   dz_v = w tau (q_v - sum_{j: I_j = v} p_j)
//
// One CTA a row: the row's maximum, the sum of exponentials, the loss over
// the k kept entries, then the dense part of the gradient, and last the k
// places that the teacher names, each written whole (a place named twice gets
// the same value twice). The exponent z/tau - lse is taken in base 2 as
// z c - L with c = log2(e) / tau and L = lse log2(e); for fp32 logits both
// constants are held in two parts, so that the exponent is off by half an ulp
// of itself, not of its larger terms.
#include "kernels.cuh"

namespace kronq {
namespace {

constexpr int DI_THREADS = 512;
constexpr int DI_WARPS = DI_THREADS / 32;
constexpr int DI_MAXK = 1024;

struct DistillP {
  const void *Z, *T;
  int64_t vocab, ldz, ldt, lddz;
  const int32_t *idx;
  int k, t_bf16;
  float c_hi, c_lo, tau;   // c = log2(e) / tau in two parts
  const float *weight;
  float *loss, *lse;
  void *dZ;
  int32_t *info;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// 2^(z c - b) with b in two parts
template <class T>
__device__ __forceinline__ float exp_term(float z, float c_hi, float c_lo, float b_hi, float b_lo) {
  float a;
  if constexpr (sizeof(T) == 4) {
    z = max_nan(z, -3.0e38f);   // -inf * c_lo has no place in a sum
    a = fmaf(z, c_hi, -b_hi) + fmaf(z, c_lo, -b_lo);
  } else {
    a = fmaf(z, c_hi, -b_hi);
  }
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
  return e;
}

// Block reductions in a fixed order; every thread gets the result.
template <class V, class F>
__device__ __forceinline__ V block_reduce(V v, V *red, V zero, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < DI_WARPS ? red[lane] : zero;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <class T, bool FWD, bool BWD>
__global__ void __launch_bounds__(DI_THREADS) distill_kernel(const DistillP a) {
  __shared__ float p_s[DI_MAXK], z_s[DI_MAXK];
  __shared__ int32_t i_s[DI_MAXK];
  __shared__ double red_d[DI_WARPS];
  __shared__ float red[DI_WARPS];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T *z = static_cast<const T *>(a.Z) + row * a.ldz;
  T *dz = static_cast<T *>(a.dZ) + row * a.lddz;
  const auto add = [](auto x, auto y) { return x + y; };
  const float w = a.weight ? a.weight[row] : 1.f;

  // ---- the teacher's kept entries
  bool any = false;
  float tmax = -INFINITY;
  if (w != 0.f) {
    for (int j = tid; j < a.k; j += DI_THREADS) {
      const int32_t i = a.idx[row * a.ldt + j];
      float t = a.t_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.T)[row * a.ldt + j])
                         : static_cast<const float *>(a.T)[row * a.ldt + j];
      const bool in = i >= 0 && i < a.vocab;
      if (i >= a.vocab) report(a.info, KRONQ_ERR_INVALID_ARG);
      if (!in) t = -INFINITY;
      i_s[j] = in && t != -INFINITY ? i : -1;
      p_s[j] = t;
      z_s[j] = in ? to_f(z[i]) : 0.f;
      any |= t != -INFINITY;
      tmax = fmaxf(tmax, t);
    }
  }
  any = __syncthreads_or(any);
  if (!any) {
    if (FWD && tid == 0) {
      a.loss[row] = 0.f;
      if (a.lse) a.lse[row] = 0.f;
    }
    if (BWD)
      for (int64_t v = tid; v < a.vocab; v += DI_THREADS) put(dz + v, 0.f);
    return;
  }
  tmax = block_reduce(tmax, red, -INFINITY, [](float x, float y) { return fmaxf(x, y); });
  float ts = 0.f;
  for (int j = tid; j < a.k; j += DI_THREADS)
    if (i_s[j] >= 0) ts += expf((p_s[j] - tmax) / a.tau);
  ts = block_reduce(ts, red, 0.f, add);

  // ---- log-sum-exp of the row
  double lse;
  if (FWD) {
    float m = -INFINITY;
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS) m = max_nan(m, to_f(z[v]));
    m = block_reduce(m, red, -INFINITY, [](float x, float y) { return max_nan(x, y); });
    const double mc = double(m) * (double(a.c_hi) + double(a.c_lo));
    const float b_hi = float(mc), b_lo = float(mc - double(b_hi));
    float s = 0.f;
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS)
      s += exp_term<T>(to_f(z[v]), a.c_hi, a.c_lo, b_hi, b_lo);
    s = block_reduce(s, red, 0.f, add);
    lse = double(m) / double(a.tau) + log(double(s));
    if (m == -INFINITY) lse = double(NAN);
  } else {
    lse = a.lse[row];
  }

  // ---- loss; p_s becomes p
  double loss = 0.0;
  const double lts = FWD ? log(double(ts)) : 0.0;
  for (int j = tid; j < a.k; j += DI_THREADS) {
    const float t = p_s[j];
    const float p = i_s[j] >= 0 ? expf((t - tmax) / a.tau) / ts : 0.f;
    p_s[j] = p;
    if (FWD && p != 0.f)
      loss += double(p) * ((double(t) - double(tmax) - double(z_s[j])) / double(a.tau) - lts + lse);
  }
  if (FWD) {
    loss = block_reduce(loss, red_d, 0.0, add);
    if (tid == 0) {
      const float l = float(double(a.tau) * double(a.tau) * loss);
      a.loss[row] = l;
      if (a.lse) a.lse[row] = float(lse);
      if (!isfinite(l)) report(a.info, KRONQ_ERR_NONFINITE);
    }
  }

  // ---- gradient
  if (BWD) {
    const double L = lse * 1.4426950408889634074;
    const float b_hi = float(L), b_lo = float(L - double(b_hi));
    const float wt = w * a.tau;
    __syncthreads();
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS)
      put(dz + v, wt * exp_term<T>(to_f(z[v]), a.c_hi, a.c_lo, b_hi, b_lo));
    __syncthreads();
    for (int j = tid; j < a.k; j += DI_THREADS) {
      const int32_t i = i_s[j];
      if (i < 0) continue;
      float p = 0.f;
      for (int l = 0; l < a.k; ++l) p += i_s[l] == i ? p_s[l] : 0.f;
      put(dz + i, wt * (exp_term<T>(z_s[j], a.c_hi, a.c_lo, b_hi, b_lo) - p));
    }
  }
}

template <class T>
kronq_status launch(cudaStream_t st, const DistillP &p, int64_t n, bool fwd, bool bwd) {
  const unsigned grid = static_cast<unsigned>(n);
  if (fwd && bwd)
    distill_kernel<T, true, true><<<grid, DI_THREADS, 0, st>>>(p);
  else if (fwd)
    distill_kernel<T, true, false><<<grid, DI_THREADS, 0, st>>>(p);
  else
    distill_kernel<T, false, true><<<grid, DI_THREADS, 0, st>>>(p);
  KQ_CHECK_LAUNCH();
  return KRONQ_OK;
}

}  // namespace

kronq_status distill(cudaStream_t st, const DistillArgs &a) {
  if (a.n == 0) return KRONQ_OK;
  DistillP p;
  p.Z = a.Z;
  p.T = a.T;
  p.vocab = a.vocab;
  p.ldz = a.ldz;
  p.ldt = a.ldt;
  p.lddz = a.lddz;
  p.idx = a.idx;
  p.k = a.k;
  p.t_bf16 = a.t_bf16;
  const double c = 1.4426950408889634074 / double(a.tau);
  p.c_hi = float(c);
  p.c_lo = float(c - double(p.c_hi));
  p.tau = a.tau;
  p.weight = a.weight;
  p.loss = a.loss;
  p.lse = a.lse;
  p.dZ = a.dZ;
  p.info = a.info;
  return a.z_bf16 ? launch<__nv_bfloat16>(st, p, a.n, a.loss != nullptr, a.dZ != nullptr)
                  : launch<float>(st, p, a.n, a.loss != nullptr, a.dZ != nullptr);
}

}  // namespace kronq
