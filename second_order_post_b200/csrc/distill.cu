// Distillation from a teacher's top logits, forward and backward. For a row
// of student logits z and the teacher's kept logits T at the places I:
//   p = softmax(T / tau),  q = softmax(z / tau),  lse = log sum exp(z / tau)
//   loss = tau^2 sum_j p_j (log p_j - z_{I_j} / tau + lse)
//   dz_v = w tau (q_v - sum_{j: I_j = v} p_j)
//
// A row's maximum and sum of exponentials, the loss over the k kept entries,
// the dense part of the gradient, and last the k places that the teacher
// names, each written whole (a place named twice gets the same value twice).
// With the gradient, distill_wide_kernel keeps a row in the shared memory of up to
// 8 CTAs, and rows too wide for that (over 281592 bf16 or 140796 fp32 logits) are
// read once per pass by distill_kernel. The loss alone needs a row once: streamed
// by distill_fwd_kernel. Exponentials are taken in base 2, with c = log2(e) / tau.
#include <map>
#include <mutex>
#include <tuple>

#include "kernels.cuh"

namespace kronq {
namespace {

constexpr int DI_THREADS = 512;
constexpr int DI_WARPS = DI_THREADS / 32;
constexpr int DI_MAXK = 1024;
constexpr float NO_LOGIT = -1.0e32f;   // what lies below counts as -inf

struct DistillP {
  const void *Z, *T;
  int64_t vocab, ldz, ldt, lddz;
  const int32_t *idx;
  int k, t_bf16;
  float c, tau;            // c = log2(e) / tau
  double inv_tau;
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
// a logit at a place that the teacher names: its distance to the maximum enters the
// loss (in the sums the exponentials of what lies below are 0 as they are)
__device__ __forceinline__ float named_logit(float z) { return z < NO_LOGIT ? -INFINITY : z; }
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float ex2(float a) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
  return e;
}

// exp((z - m) / tau) = 2^((z - m) c). The difference comes first, so that its
// rounding is relative to it: in z c - m c the rounding of m c alone is 2^-25 |m c|
// in the exponent, which has no bound over the logits and temperatures allowed (with
// |m| / tau = 1e8 the sum of a row came out negative). It costs an addition a pair.
//   shift: added to the exponent (0 with m from the row's own logits).
struct Exponent {
  F2 c, b, d;
  __device__ __forceinline__ Exponent(float m, float c1, float shift = 0.f)
      : c(f2(c1, c1)), b(f2(-m, -m)), d(f2(shift, shift)) {}
  __device__ __forceinline__ F2 operator()(F2 z) const {
    const float2 x = f2_get(f2_fma(f2_add(z, b), c, d));
    return f2(ex2(x.x), ex2(x.y));
  }
  __device__ __forceinline__ float one(float z) const { return f2_get((*this)(f2(z, z))).x; }
};

// exp(z / tau - lse) = 2^((z - m) c + shift) for a row's stored lse: m = tau lse in
// fp32, and shift what that drops of it, in the exponent (it is up to 2^-24 |lse|, and
// a factor 1 + shift ln 2 would do for small ones only).
__device__ __forceinline__ void lse_reference(float lse, const DistillP &a, float &m,
                                              float &shift) {
  const double r = double(lse) * double(a.tau);
  m = float(r);
  shift = float((double(m) - r) * double(a.c));
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

template <class T, bool FWD>
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
      z_s[j] = in ? named_logit(to_f(z[i])) : 0.f;
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
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS) put(dz + v, 0.f);
    return;
  }
  tmax = block_reduce(tmax, red, -INFINITY, [](float x, float y) { return fmaxf(x, y); });
  float ts = 0.f;
  for (int j = tid; j < a.k; j += DI_THREADS)
    if (i_s[j] >= 0) ts += expf((p_s[j] - tmax) / a.tau);
  ts = block_reduce(ts, red, 0.f, add);

  // ---- log-sum-exp of the row
  double lse, log_s = 0.0;
  float m = -INFINITY, s = 0.f, shift = 0.f;
  if (FWD) {
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS) m = max_nan(m, to_f(z[v]));
    m = block_reduce(m, red, -INFINITY, [](float x, float y) { return max_nan(x, y); });
    if (m < NO_LOGIT) m = NAN;   // no logit at all: q has no value
    const Exponent ex(m, a.c);
    for (int64_t v = tid; v < a.vocab; v += DI_THREADS) s += ex.one(to_f(z[v]));
    s = block_reduce(s, red, 0.f, add);
    log_s = log(double(s));
    lse = double(m) / double(a.tau) + log_s;
  } else {
    lse = a.lse[row];
    lse_reference(a.lse[row], a, m, shift);
  }

  // ---- loss; p_s becomes p
  double loss = 0.0;
  const double lts = FWD ? log(double(ts)) : 0.0;
  for (int j = tid; j < a.k; j += DI_THREADS) {
    const float t = p_s[j];
    const float p = i_s[j] >= 0 ? expf((t - tmax) / a.tau) / ts : 0.f;
    p_s[j] = p;
    if (FWD && p != 0.f)
      loss += double(p) * ((double(t) - double(tmax) + (double(m) - double(z_s[j]))) /
                               double(a.tau) + (log_s - lts));
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
  const Exponent ex(m, a.c, shift);
  const float wt = w * a.tau, scale = FWD ? __fdiv_rn(wt, s) : wt;
  __syncthreads();
  for (int64_t v = tid; v < a.vocab; v += DI_THREADS)
    put(dz + v, scale * ex.one(to_f(z[v])));
  __syncthreads();
  for (int j = tid; j < a.k; j += DI_THREADS) {
    const int32_t i = i_s[j];
    if (i < 0) continue;
    float p = 0.f;
    for (int l = 0; l < a.k; ++l) p += i_s[l] == i ? p_s[l] : 0.f;
    put(dz + i, scale * ex.one(z_s[j]) - wt * p);
  }
}

// ---------------------------------------------------------------- row on the chip
template <class T>
struct VecOf {
  static constexpr int E = 16 / sizeof(T);
};

// a vector's values in pairs
template <class T>
__device__ __forceinline__ void unpack2(const uint4 &r, F2 *x) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  if constexpr (sizeof(T) == 4) {
    x[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    x[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      x[t] = f2(__uint_as_float(w[t] << 16), __uint_as_float(w[t] & 0xffff0000u));
  }
}
__device__ __forceinline__ void store_vec2(float *p, const F2 *x) {
  const float2 a = f2_get(x[0]), b = f2_get(x[1]);
  *reinterpret_cast<float4 *>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_vec2(__nv_bfloat16 *p, const F2 *x) {
  uint4 o;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&o);
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const float2 a = f2_get(x[t]);
    h[t] = __floats2bfloat162_rn(a.x, a.y);
  }
  *reinterpret_cast<uint4 *>(p) = o;
}

// (m, s) pairs: m may be -inf (then s is 0)
__device__ __forceinline__ float rescale(float s, float from, float to, float c) {
  return from == -INFINITY ? 0.f : s * ex2((from - to) * c);
}

// largest value of a warp, NaN if one is
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// (m, s) over a warp, scaled to the common maximum
__device__ __forceinline__ void warp_pair(float &m, float &s, float c) {
  const float wm = warp_max_nan(m);
  s = warp_sum(rescale(s, m, wm, c));
  m = wm;
}

// With the gradient. A row lies in the shared memory of a CTA (or, over 70 KB, of a
// cluster of them, independent CTAs in the backward pass alone), where
// a bulk copy brings it. It is read there three times: maximum, sum of
// exponentials, gradient. The CTAs are persistent and independent, several an
// SM, so that the copies of some run under the arithmetic of others; while a
// CTA's own copy is on its way it writes the rest of the row before (the places
// that the teacher names, the loss) and has the teacher's entries of the next.
// Each thread makes a pair (maximum m, sum s of exponentials relative to it) of
// its part of the row and one of its teacher entries; the pairs meet by warp,
// CTA and cluster in a fixed order, scaled to the common maximum. q_v is then
// exp(z_v / tau - m) / s, without a logarithm; the loss needs one a row.
//   An entry needs the sum over all entries that name its place: they are found
// in a list of those whose places share a hash (about one entry long, made while
// the row is on its way) and added in the order of their numbers. (Comparing with
// all k entries cost 314 us for 1024 rows of 32000 bf16 logits and k = 1024, 63 us
// with the lists, backward alone; the same 27 us at k = 64.)
//   The copy takes whole 16-byte vectors inside the row; the threads that own
// the row's first and last vector put those together when they are cut.
//   Sizes: 384 threads and three CTAs an SM, or for rows of up to 22 KB 128
// threads and up to nine, of up to 6 KB 64 threads and up to sixteen.
// Measured (4096 rows of 32000 bf16 logits, k = 64, with the gradient; 110 us as it
// is): three CTAs of 384 threads 107 us, two of 512 threads 120 us, six of 192
// threads on half rows (clusters of two) 121 us; the row in registers, one CTA of
// 512 threads an SM, 135 us (its phases do not overlap).
constexpr int WIDE_VEC = 4400;   // vectors of a part at most: 70 KB
template <int ST>
constexpr int wide_per_sm() {
  return ST == 384 ? 3 : ST == 128 ? 9 : 16;
}

// ln(x) for a normal x > 0, off by less than 4e-8: exponent times ln 2 in
// fp64, plus the fp32 logarithm of a mantissa in [0.75, 1.5). NaN for what is no
// sum of a row that has a softmax: NaN, inf, 0 and less.
__device__ __forceinline__ double log_split(float x) {
  if (!(x > 0.f && x < INFINITY)) return double(NAN);
  const int ex = (__float_as_int(x) - 0x3f400000) >> 23;
  const float f = __int_as_float(__float_as_int(x) - (ex << 23));
  return double(ex) * 0.69314718055994530942 + double(logf(f));
}

// largest of 8 bf16 or 4 fp32
template <class T>
__device__ __forceinline__ float max_vec(const uint4 &r) {
  if constexpr (sizeof(T) == 4) {
    return max_nan(max_nan(__uint_as_float(r.x), __uint_as_float(r.y)),
                   max_nan(__uint_as_float(r.z), __uint_as_float(r.w)));
  } else {
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&r);
    const __nv_bfloat162 x = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
    return max_nan(__low2float(x), __high2float(x));
  }
}

template <class T>
__device__ __forceinline__ uint4 neg_inf_vec() {
  constexpr uint32_t b = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(b, b, b, b);
}

// The vector at element e of a row of `vocab`, places outside it -inf.
template <class T>
__device__ __forceinline__ uint4 cut_vec(const T *z, int64_t e, int64_t vocab) {
  constexpr int E = VecOf<T>::E;
  uint4 o = neg_inf_vec<T>();
  uint32_t *r = reinterpret_cast<uint32_t *>(&o);
#pragma unroll
  for (int t = 0; t < E; ++t) {
    if (e + t < 0 || e + t >= vocab) continue;
    if constexpr (sizeof(T) == 4) {
      r[t] = __float_as_uint(z[e + t]);
    } else {
      const uint32_t b = __bfloat16_as_ushort(z[e + t]);
      r[t / 2] = t % 2 ? (r[t / 2] & 0xffffu) | b << 16 : (r[t / 2] & 0xffff0000u) | b;
    }
  }
  return o;
}

// The loss and lse of a row from its (m, s), the teacher's sum and the warps' parts
// of sum p (T - max T + m - z) (one thread). The differences come first: m itself may
// be so large that even fp64 keeps nothing of them beside it.
__device__ __forceinline__ void finish_loss(const DistillP &a, int64_t r, bool counts, float m,
                                            float s, float ts, const double *parts_s, int np) {
  float l = 0.f, lse = 0.f;
  if (counts) {
    double x = 0.0;
    for (int q = 0; q < np; ++q) x += parts_s[q];
    const double ls = log_split(s);
    l = float(double(a.tau) * double(a.tau) * (x * a.inv_tau + (ls - log_split(ts))));
    lse = float(double(m) * a.inv_tau + ls);
    if (!isfinite(l)) report(a.info, KRONQ_ERR_NONFINITE);
  }
  a.loss[r] = l;
  if (a.lse) a.lse[r] = lse;
}

template <class T, bool FWD, int ST>
__global__ void __launch_bounds__(ST, wide_per_sm<ST>())
    distill_wide_kernel(const DistillP a, int parts, int per, int kp, int bits, int n) {
  constexpr int E = VecOf<T>::E, WARPS = ST / 32;
  extern __shared__ __align__(128) uint8_t dsm[];
  uint4 *buf = reinterpret_cast<uint4 *>(dsm);
  float *t_s = reinterpret_cast<float *>(buf + per);                  // [2][kp]: T, then w tau p
  int32_t *i_s = reinterpret_cast<int32_t *>(t_s + 2 * kp);           // [2][kp]: places
  float *z_s = reinterpret_cast<float *>(i_s + 2 * kp);               // [2][kp]: z, then w tau q
  int32_t *head_s = reinterpret_cast<int32_t *>(z_s + 2 * kp);        // [2][1 << bits]
  int16_t *next_s = reinterpret_cast<int16_t *>(head_s + (2 << bits));   // [2][kp]
  __shared__ __align__(16) float4 wpair[32];         // (m, s) of the row, of the teacher
  __shared__ __align__(16) float4 pair[2];           // the CTA's (m, s)
  __shared__ double loss_s[2][WARPS];
  __shared__ uint64_t bar;
  __shared__ int abort_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool clus = FWD && parts > 1;
  const int rank = blockIdx.x % parts, vocab = static_cast<int>(a.vocab), k = a.k;
  const int stride = gridDim.x / parts;
  const float c2e = a.c;
  const int lw = kq_min(WARPS, (k + 31) / 32);   // warps with teacher entries
  if (tid == 0) {
    mbar_init(&bar, 1);
    abort_s = 0;
    fence_mbar_init();
  }
  if (tid < 32) wpair[tid] = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  for (int j = tid; j < 2 * kp; j += ST) i_s[j] = -1, t_s[j] = 0.f;
  for (int j = tid; j < 2 << bits; j += ST) head_s[j] = -1;
  __syncthreads();
  pdl_launch();
  pdl_wait();

  // where this CTA's part of a row lies: `cnt` vectors from element e0 (which
  // may be negative: the row's first vector is an aligned address)
  auto row_ptr = [&](int r) { return static_cast<const T *>(a.Z) + int64_t(r) * a.ldz; };
  auto part_of = [&](const T *z, int &e0, int &cnt) {
    const int head = static_cast<int>(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
    const int nvec = (vocab + head + E - 1) / E, v0 = per * rank;
    e0 = v0 * E - head;
    cnt = kq_max(kq_min(nvec - v0, per), 0);
  };
  // Starts the copy of a row's part (all threads call it, the buffer is free):
  // whole vectors by bulk copy, cut ones by their owners. A part without a
  // whole vector completes the barrier's phase all the same.
  uint32_t copies = 0;
  auto fetch = [&](int r) {
    const T *z = row_ptr(r);
    int e0, cnt;
    part_of(z, e0, cnt);
    const int lo = e0 < 0 ? 1 : 0;
    const bool cut = cnt > 0 && e0 + cnt * E > vocab;
    const int hi = cut ? cnt - 1 : cnt;
    if (tid == 0) {
      const uint32_t bytes = hi > lo ? (hi - lo) * 16u : 0u;
      mbar_expect_tx(&bar, bytes);
      if (bytes) bulk_load(buf + lo, z + (e0 + lo * E), bytes, &bar);
      if (lo && cnt > 0) buf[0] = cut_vec(z, e0, vocab);
    }
    if (cut && tid == (cnt - 1) % ST) buf[cnt - 1] = cut_vec(z, e0 + (cnt - 1) * E, vocab);
    if (lo || cut) fence_proxy_async_smem();   // a later copy may write there
    ++copies;
  };
  auto weight_of = [&](int64_t r) { return r >= n ? 0.f : a.weight ? a.weight[r] : 1.f; };

  // the teacher's entry of this thread (entries past ST are read when needed)
  auto entry = [&](int r, int j, int &i, float &t) {
    const int64_t at = r * a.ldt + j;
    i = a.idx[at];
    t = a.t_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.T)[at])
                 : static_cast<const float *>(a.T)[at];
  };
  // which list of entries a place belongs to
  auto bucket = [&](int i) { return static_cast<int>((uint32_t(i) * 2654435769u) >> (32 - bits)); };
  // the student's logit there
  auto logit_at = [&](int r, int i) { return i >= 0 && i < vocab ? row_ptr(r)[i] : T(0.f); };
  int row = blockIdx.x / parts;
  float w = weight_of(row);
  if (w != 0.f) fetch(row);
  int ni = -1;
  float nt = 0.f;
  T nz = T(0.f);
  if (row < n && tid < k) {
    entry(row, tid, ni, nt);
    nz = logit_at(row, ni);
  }
  uint32_t phase = 0;
  int par = 0;
  bool abort = false;       // a wait ran out: no more copies, the barriers go on
  for (; row < n; par ^= 1) {
    const bool live = w != 0.f;
    const float w1 = weight_of(int64_t(row) + stride);
    const float lse_in = !FWD && live ? a.lse[row] : 0.f;
    const T *z = row_ptr(row);
    float *tr = t_s + par * kp, *zr = z_s + par * kp;
    int32_t *ir = i_s + par * kp, *head = head_s + (par << bits);
    int16_t *next = next_s + par * kp;
    int e0, cnt;
    part_of(z, e0, cnt);
    // ---- the teacher's entries, while the row is on its way
    float tm = -INFINITY, ts = 0.f;
    if (live) {
      for (int j = tid; j < k; j += ST) {
        int i = ni;
        float t = nt, zj = to_f(nz);
        if (j >= ST) {
          entry(row, j, i, t);
          zj = to_f(logit_at(row, i));
        }
        zj = named_logit(zj);
        if (i >= vocab) report(a.info, KRONQ_ERR_INVALID_ARG);
        if (i < 0 || i >= vocab) t = -INFINITY;
        if (t == -INFINITY) i = -1;
        zr[j] = zj;
        tr[j] = t;
        ir[j] = i;
        if (i >= 0 && i >= e0 && i < e0 + cnt * E)
          next[j] = static_cast<int16_t>(atomicExch(&head[bucket(i)], j));
        const float m2 = max_nan(tm, t);
        ts = rescale(ts, tm, m2, c2e) + (i < 0 ? 0.f : ex2((t - m2) * c2e));
        tm = m2;
      }
      if (warp * 32 < k) warp_pair(tm, ts, c2e);
    }
    // ---- (m, s) of this part
    float m = -INFINITY, s = 0.f;
    if (live) {
      if (!mbar_wait(&bar, phase, &abort_s)) abort = true;
      phase ^= 1;
      if (FWD) {
#pragma unroll 4
        for (int v = tid; v < cnt; v += ST) m = max_nan(m, max_vec<T>(buf[v]));
        m = m < NO_LOGIT ? NO_LOGIT : m;    // exponents of masked logits: -inf
        const Exponent ex(m, c2e);
        F2 acc0 = f2(0.f, 0.f), acc1 = acc0;
#pragma unroll 4
        for (int v = tid; v < cnt; v += ST) {
          F2 x[E / 2];
          unpack2<T>(buf[v], x);
#pragma unroll
          for (int t = 0; t < E / 2; t += 2) {
            acc0 = f2_add(acc0, ex(x[t]));
            acc1 = f2_add(acc1, ex(x[t + 1]));
          }
        }
        const float2 sum = f2_get(f2_add(acc0, acc1));
        s = sum.x + sum.y;
        warp_pair(m, s, c2e);
      }
    }
    if (lane == 0) wpair[warp] = make_float4(m, s, tm, ts);
    __syncthreads();
    if (stride < n - row && tid < k) entry(row + stride, tid, ni, nt);
    for (int j = tid; j < 1 << bits; j += ST) head_s[((par ^ 1) << bits) + j] = -1;
    {
      const float4 x = wpair[lane];
      m = FWD ? warp_max_nan(x.x) : 0.f;
      tm = warp_max_nan(x.z);
      s = FWD ? warp_sum(rescale(x.y, x.x, m, c2e)) : 0.f;
      ts = warp_sum(rescale(x.w, x.z, tm, c2e));
    }
    const bool counts = live && tm != -INFINITY;   // some entry is kept
    if (clus) {
      if (tid == 0) pair[par] = make_float4(m, s, 0.f, 0.f);
      __syncwarp();
      cluster_sync_all();
      const float4 x = lane < parts ? ld_dsmem_f4(mapa_shared(smem_u32(&pair[par]), lane))
                                    : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      m = warp_max_nan(x.x);
      s = warp_sum(rescale(x.y, x.x, m, c2e));
    }
    if (FWD && s == 0.f) m = NAN;   // no logit at all: q has no value
    // ---- the dense gradient
    const float wt = w * a.tau;
    // The exponentials of the gradient: those of the sums, relative to the row's
    // m, over s; in the backward pass alone relative to tau lse, of which the
    // part that fp32 drops goes into the exponent.
    float ref = m, shift = 0.f;
    if (!FWD) lse_reference(lse_in, a, ref, shift);
    const float scale = FWD ? __fdiv_rn(wt, s) : wt;
    const Exponent ex(ref, c2e, shift);
    T *dz = static_cast<T *>(a.dZ) + int64_t(row) * a.lddz;
    const bool vec =
        (reinterpret_cast<uintptr_t>(dz) & 15) == (reinterpret_cast<uintptr_t>(z) & 15);
    const F2 sc = f2(scale, scale);
    // the vectors that the row fills and that are aligned in dZ too
    const int lo = !vec ? cnt : e0 < 0 ? 1 : 0, hi = !vec ? cnt : e0 + cnt * E > vocab ? cnt - 1 : cnt;
    if (counts) {
#pragma unroll 4
      for (int v = tid; v < hi; v += ST) {
        if (v < lo) continue;
        F2 x[E / 2];
        unpack2<T>(buf[v], x);
#pragma unroll
        for (int t = 0; t < E / 2; ++t) x[t] = f2_mul(ex(x[t]), sc);
        store_vec2(dz + (e0 + v * E), x);
      }
    } else {
      F2 x[E / 2];
#pragma unroll
      for (int t = 0; t < E / 2; ++t) x[t] = f2(0.f, 0.f);
      for (int v = tid; v < hi; v += ST)
        if (v >= lo) store_vec2(dz + (e0 + v * E), x);
    }
    // the others (at most the first and the last, or all of them) by element
    for (int v = tid; v < cnt; v += ST) {
      if (v >= lo && v < hi) continue;
      F2 x[E / 2];
      unpack2<T>(buf[v], x);
      const int at = e0 + v * E;
#pragma unroll
      for (int t = 0; t < E / 2; ++t) {
        const float2 g = f2_get(f2_mul(ex(x[t]), sc));
        if (at + 2 * t >= 0 && at + 2 * t < vocab) put(dz + at + 2 * t, counts ? g.x : 0.f);
        if (at + 2 * t + 1 >= 0 && at + 2 * t + 1 < vocab)
          put(dz + at + 2 * t + 1, counts ? g.y : 0.f);
      }
    }
    // ---- the teacher's p (kept as w tau p) and its part of the loss
    if (counts && warp * 32 < k) {
      const float rts = __fdiv_rn(1.f, ts);
      double x = 0.0;
      for (int j = tid; j < k; j += ST) {
        const float t = tr[j], zj = zr[j];
        const float p = ir[j] >= 0 ? ex2((t - tm) * c2e) * rts : 0.f;
        if (FWD && rank == 0 && p != 0.f)
          x += double(p) * (double(t) - double(tm) + (double(m) - double(zj)));
        tr[j] = wt * p;
        zr[j] = scale * ex.one(zj);
      }
      if (FWD && rank == 0) {
        __syncwarp();
        x = warp_sum_d(x);
        if (lane == 0) loss_s[par][warp] = x;
      }
    }
    __syncthreads();
    if (w1 != 0.f && !abort) fetch(row + stride);   // the buffer is free
    if (stride < n - row && tid < k) nz = logit_at(row + stride, ni);
    // ---- the places the teacher names in this part, behind the dense stores:
    // w tau (q - the sum of the p of all entries that name the place)
    if (counts) {
      for (int j = tid; j < k; j += ST) {
        const int i = ir[j];
        if (i < 0 || i < e0 || i >= e0 + cnt * E) continue;
        const int first = head[bucket(i)];
        int same = 0;
        for (int l = first; l >= 0; l = next[l]) same += ir[l] == i;
        float p = tr[j];
        if (same > 1) {   // in the order of their entries, whatever the list's
          p = 0.f;
          if (same <= 4) {
            for (int q = 0, done = -1; q < same; ++q) {
              int at = DI_MAXK;
              for (int l = first; l >= 0; l = next[l])
                if (ir[l] == i && l > done && l < at) at = l;
              p += tr[at];
              done = at;
            }
          } else {
            for (int l = 0; l < k; ++l) p += ir[l] == i ? tr[l] : 0.f;
          }
        }
        put(dz + i, zr[j] - p);
      }
    }
    if (FWD && rank == 0 && tid == ST - 1)
      finish_loss(a, row, counts, m, s, ts, loss_s[par], lw);
    w = w1;
    if (stride >= n - row) break;
    row += stride;
  }
  if (abort) {   // a copy may still be in flight
    if (tid == 0) report(a.info, KRONQ_ERR_TIMEOUT);
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(&bar, (copies & 1) ^ 1) && globaltimer() - t0 < kWaitLimitNs) {
    }
  }
  __syncwarp();
  // no CTA leaves while another may still read its pair
  if (clus) cluster_sync_all();
}

// ---------------------------------------------------------------- forward alone
// Nothing needs a row twice, so it is streamed through registers: a CTA per row,
// or a cluster of them when rows are few. Each thread takes FWD_U vectors at a
// time, raises its maximum to theirs (its sum is rescaled only when that rises)
// and adds their exponentials; the pairs meet as above. The places that the
// teacher names are read by the first CTA under the first vectors' way.
constexpr int FWD_U = 4;
template <class T, int ST>
__global__ void __launch_bounds__(ST, 1024 / ST)
    distill_fwd_kernel(const DistillP a, int parts) {
  constexpr int E = VecOf<T>::E, WARPS = ST / 32;
  __shared__ float t_s[DI_MAXK], z_s[DI_MAXK];
  __shared__ __align__(16) float4 wpair[WARPS];
  __shared__ __align__(16) float4 pair;
  __shared__ double loss_s[WARPS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % parts, k = a.k;
  const int64_t row = blockIdx.x / parts;
  const float c2e = a.c;
  pdl_launch();
  pdl_wait();
  const float w = a.weight ? a.weight[row] : 1.f;
  if (w == 0.f) {   // (the whole cluster)
    if (rank == 0 && tid == 0) {
      a.loss[row] = 0.f;
      if (a.lse) a.lse[row] = 0.f;
    }
    return;
  }
  const T *z = static_cast<const T *>(a.Z) + row * a.ldz;
  const int64_t head = static_cast<int64_t>(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
  const int64_t nvec = (a.vocab + head + E - 1) / E, per = (nvec + parts - 1) / parts;
  const int64_t v0 = rank * per, v1 = kq_min<int64_t>(v0 + per, nvec);
  // whole vectors
  const int64_t w0 = v0 == 0 && head ? 1 : v0;
  const int64_t w1 = v1 == nvec && nvec * E - head > a.vocab ? v1 - 1 : v1;
  const uint4 *zv = reinterpret_cast<const uint4 *>(z - head);
  float m = -INFINITY, s = 0.f;
  auto add = [&](const uint4 *x) {
    float top = max_vec<T>(x[0]);
#pragma unroll
    for (int u = 1; u < FWD_U; ++u) top = max_nan(top, max_vec<T>(x[u]));
    top = max_nan(m, top < NO_LOGIT ? NO_LOGIT : top);   // exponents of masked logits: -inf
    if (!(top == m)) {
      s = rescale(s, m, top, c2e);
      m = top;
    }
    const Exponent ex(m, c2e);
    F2 acc0 = f2(0.f, 0.f), acc1 = acc0;
#pragma unroll
    for (int u = 0; u < FWD_U; ++u) {
      F2 y[E / 2];
      unpack2<T>(x[u], y);
#pragma unroll
      for (int t = 0; t < E / 2; t += 2) {
        acc0 = f2_add(acc0, ex(y[t]));
        acc1 = f2_add(acc1, ex(y[t + 1]));
      }
    }
    const float2 sum = f2_get(f2_add(acc0, acc1));
    s += sum.x + sum.y;
  };
  auto load = [&](int64_t v, uint4 *x) {
#pragma unroll
    for (int u = 0; u < FWD_U; ++u) {
      const int64_t at = v + u * ST;
      x[u] = at < w1 ? zv[at] : neg_inf_vec<T>();
    }
  };
  uint4 x[FWD_U];
  int64_t v = w0 + tid;
  load(v, x);
  // ---- the teacher's entries
  float tm = -INFINITY, ts = 0.f;
  if (rank == 0) {
    for (int j = tid; j < k; j += ST) {
      const int64_t at = row * a.ldt + j;
      const int i = a.idx[at];
      float t = a.t_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(a.T)[at])
                         : static_cast<const float *>(a.T)[at];
      if (i >= a.vocab) report(a.info, KRONQ_ERR_INVALID_ARG);
      const bool in = i >= 0 && i < a.vocab;
      if (!in) t = -INFINITY;
      t_s[j] = t;
      z_s[j] = in ? named_logit(to_f(z[i])) : 0.f;
      const float m2 = max_nan(tm, t);
      ts = rescale(ts, tm, m2, c2e) + (t == -INFINITY ? 0.f : ex2((t - m2) * c2e));
      tm = m2;
    }
    if (warp * 32 < k) warp_pair(tm, ts, c2e);
  }
  // ---- (m, s) of this part
  while (v < w1) {   // (the vectors of the next step are on their way)
    uint4 y[FWD_U];
    v += FWD_U * ST;
    load(v, y);
    add(x);
    if (v >= w1) break;
    v += FWD_U * ST;
    load(v, x);
    add(y);
  }
  if (tid == 0 && v0 < w0) {
#pragma unroll
    for (int u = 0; u < FWD_U; ++u) x[u] = neg_inf_vec<T>();
    x[0] = cut_vec(z, -head, a.vocab);
    add(x);
  }
  if (tid == ST - 1 && w1 < v1 && w1 >= w0) {
#pragma unroll
    for (int u = 0; u < FWD_U; ++u) x[u] = neg_inf_vec<T>();
    x[0] = cut_vec(z, w1 * E - head, a.vocab);
    add(x);
  }
  warp_pair(m, s, c2e);
  if (lane == 0) wpair[warp] = make_float4(m, s, tm, ts);
  __syncthreads();
  {
    const float4 q = lane < WARPS ? wpair[lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    m = warp_max_nan(q.x);
    tm = warp_max_nan(q.z);
    s = warp_sum(rescale(q.y, q.x, m, c2e));
    ts = warp_sum(rescale(q.w, q.z, tm, c2e));
  }
  if (parts > 1) {
    if (tid == 0) pair = make_float4(m, s, 0.f, 0.f);
    __syncwarp();
    cluster_sync_all();
    if (rank == 0) {
      const float4 q = lane < parts ? ld_dsmem_f4(mapa_shared(smem_u32(&pair), lane))
                                    : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      m = warp_max_nan(q.x);
      s = warp_sum(rescale(q.y, q.x, m, c2e));
    }
  }
  // ---- the loss
  if (rank == 0) {
    const bool counts = tm != -INFINITY;   // some entry is kept
    if (s == 0.f) m = NAN;   // no logit at all: q has no value
    const float rts = __fdiv_rn(1.f, ts);
    double x0 = 0.0;
    if (counts) {
      for (int j = tid; j < k; j += ST) {
        const float t = t_s[j];
        const float p = t == -INFINITY ? 0.f : ex2((t - tm) * c2e) * rts;
        if (p != 0.f) x0 += double(p) * (double(t) - double(tm) + (double(m) - double(z_s[j])));
      }
    }
    x0 = warp_sum_d(x0);
    if (lane == 0) loss_s[warp] = x0;
    __syncthreads();
    if (tid == 0) finish_loss(a, row, counts, m, s, ts, loss_s, kq_min(WARPS, (k + 31) / 32));
  }
  __syncwarp();
  // no CTA leaves while another may still read its pair
  if (parts > 1) cluster_sync_all();
}

// Threads of a row: as many as fill the chip at 1024 an SM, with four vectors each
// at least and 40 at most; above 512 they are CTAs of a cluster. Measured with 64 |
// 128 | 256 | 512 threads: 4096 rows of 32000 bf16 logits 52.3 | 50.0 | 55.5 | 75.8 us,
// 768 of 128256 60.6 | 51.5 | 40.0 | 40.6, 2048 of 6000 8.6 | 9.9 | 13.8 | 26.2,
// 257 rows of 50257 fp32 logits 31.2 | 19.5 | 14.7 | 12.0; 8 rows of 128256 bf16
// logits 8.1 with 512 and 4.6 with 4096; 100 of 128256 fp32 logits 14.7 with 1024
// and 20.3 with 2048, which take a wave and a third.
template <class T>
kronq_status launch_fwd(cudaStream_t st, const DistillP &p, int64_t n) {
  const int64_t nvec = ceil_div(p.vocab, VecOf<T>::E) + 1;
  int threads = 64;   // the power of two next to a limit by the row's length
  while (threads < 4096 && (threads * 10 < nvec / 40 * 7 ||
                            (threads * 10 < nvec / 4 * 7 && threads * 2 * n <= 148 * 1024)))
    threads *= 2;
  const int parts = kq_max(threads / 512, 1);
  auto go = [&](auto st_c) {
    constexpr int ST = decltype(st_c)::value;
    return launch_kernel(st, distill_fwd_kernel<T, ST>, n * parts, ST, 0, parts, true, p, parts);
  };
  switch (threads) {
    case 64: return go(std::integral_constant<int, 64>());
    case 128: return go(std::integral_constant<int, 128>());
    case 256: return go(std::integral_constant<int, 256>());
    default: return go(std::integral_constant<int, 512>());
  }
}

// How many rows (clusters of `parts` CTAs) are on the chip at once; asked once
// per kernel, device and size.
kronq_status resident_rows(const void *kern, int threads, int smem, int parts, bool clus,
                           int *rows) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void *, int, int>, int> known;
  int dev = 0;
  KQ_CUDA(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(mu);
  int &v = known[std::make_tuple(dev, kern, smem, parts)];
  if (v == 0) {
    int got = 0;
    if (clus) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(parts));
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(parts);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      KQ_CUDA(cudaOccupancyMaxActiveClusters(&got, kern, &cfg));
    } else {
      int sms = 0;
      KQ_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
      KQ_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, kern, threads, smem));
      got = got * sms / parts;
    }
    v = kq_max(got, 1);
  }
  *rows = v;
  return KRONQ_OK;
}

// A launch of distill_wide_kernel with rows over `parts` CTAs: its shared memory
// and how many rows run at once.
struct WidePlan {
  int parts, per, kp, bits, smem, rows;
};
template <class T, bool FWD, int ST>
kronq_status plan_wide(const DistillP &p, int64_t nvec, int parts, WidePlan *w) {
  auto *kern = distill_wide_kernel<T, FWD, ST>;
  w->parts = parts;
  w->per = static_cast<int>(ceil_div(nvec, parts));
  w->kp = (p.k + 3) / 4 * 4;
  w->bits = 5;   // a list an entry
  while (1 << w->bits < p.k) ++w->bits;
  w->smem = (w->per * 16 + 28 * w->kp + (8 << w->bits) + 1023) / 1024 * 1024;
  KQ_TRY(smem_attr(kern, w->smem));
  return resident_rows(reinterpret_cast<const void *>(kern), ST, w->smem, parts, FWD && parts > 1,
                       &w->rows);
}
template <class T, bool FWD, int ST>
kronq_status launch_wide(cudaStream_t st, const DistillP &p, int64_t n, const WidePlan &w) {
  const int64_t rows = kq_min<int64_t>(n, w.rows);
  return launch_kernel(st, distill_wide_kernel<T, FWD, ST>, rows * w.parts, ST, w.smem,
                       FWD ? w.parts : 1, true, p, w.parts, w.per, w.kp, w.bits,
                       static_cast<int>(n));
}

template <class T, bool FWD>
kronq_status launch_grad(cudaStream_t st, const DistillP &p, int64_t n) {
  // a row that starts off a 16-byte boundary touches one vector more
  const int64_t nvec = ceil_div(p.vocab, VecOf<T>::E) + 1;
  WidePlan w;
  if (nvec <= 384) {
    KQ_TRY((plan_wide<T, FWD, 64>(p, nvec, 1, &w)));
    return launch_wide<T, FWD, 64>(st, p, n, w);
  }
  if (nvec <= 1408) {
    KQ_TRY((plan_wide<T, FWD, 128>(p, nvec, 1, &w)));
    return launch_wide<T, FWD, 128>(st, p, n, w);
  }
  if (nvec <= 8 * WIDE_VEC) {
    // Parts of a row: what makes the rounds of rows cheapest. A round costs its
    // part plus about 1500 vectors' time for the barriers and the teacher's
    // entries, 2500 more across a cluster. (Measured with the gradient: one row of
    // 32000 bf16 logits 7.1 us in one part, 5.4 in eight; 300 rows of 50257 fp32
    // logits 36.2 us in three parts, 33.2 in four; 64 rows of 8000 fp32 logits 4.9 us
    // in one part, 6.0 in eight.)
    WidePlan best = {};
    int64_t best_cost = 0;
    for (int parts = static_cast<int>(ceil_div(nvec, WIDE_VEC)); parts <= 8; ++parts) {
      KQ_TRY((plan_wide<T, FWD, 384>(p, nvec, parts, &w)));
      const int64_t cost =
          ceil_div(n, w.rows) * (w.per + 1500 + (FWD && parts > 1 ? 2500 : 0));
      if (best.parts == 0 || cost < best_cost) {
        best = w;
        best_cost = cost;
      }
    }
    return launch_wide<T, FWD, 384>(st, p, n, best);
  }
  return launch_kernel(st, distill_kernel<T, FWD>, n, DI_THREADS, 0, 1, false, p);
}

template <class T>
kronq_status launch(cudaStream_t st, const DistillP &p, int64_t n, bool fwd, bool bwd) {
  return !bwd  ? launch_fwd<T>(st, p, n)
         : fwd ? launch_grad<T, true>(st, p, n)
               : launch_grad<T, false>(st, p, n);
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
  p.c = float(1.4426950408889634074 / double(a.tau));
  p.tau = a.tau;
  p.inv_tau = 1.0 / double(a.tau);
  p.weight = a.weight;
  p.loss = a.loss;
  p.lse = a.lse;
  p.dZ = a.dZ;
  p.info = a.info;
  return a.z_bf16 ? launch<__nv_bfloat16>(st, p, a.n, a.loss != nullptr, a.dZ != nullptr)
                  : launch<float>(st, p, a.n, a.loss != nullptr, a.dZ != nullptr);
}

}  // namespace kronq
