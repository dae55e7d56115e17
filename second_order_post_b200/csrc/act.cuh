// The activations of the dense operators and their derivatives, in fp32.
//   silu       z s(z),                s(z) = 1 / (1 + exp(-z))
//   gelu       z P(z),                P(z) = erfc(-z / sqrt 2) / 2, the normal integral
//   gelu_tanh  z s(2 v),              v = sqrt(2 / pi) (z + 0.044715 z^3):
//              (1 + tanh v) / 2 = s(2 v), which keeps its relative accuracy
//              where tanh v is close to -1
// A NaN stays a NaN.
#pragma once

#include "common.cuh"

namespace kronq {

__device__ __forceinline__ float logistic(float z) {
  return __fdividef(1.f, 1.f + __expf(-z));
}

// The normal integral's tail over its density's exponential: W(a) =
// exp(a^2 / 2) P(-a) for a >= 0, falling like 1 / a. In t = 1 / (1 + 0.24 a), as
// Hastings' approximations (Abramowitz and Stegun 7.1.26) but to a relative error:
// W = t (c0 + ... + c7 t^7), fitted here over all a >= 0 to 4.3e-7, 8e-7 with
// fp32's roundings. One exponential then serves P and the density; with erfcf the
// backward pass of 4096 x 4096 elements was bound by its instructions.
__device__ __forceinline__ float tail_ratio(float a) {
  const float t = __fdividef(1.f, fmaf(0.24f, a, 1.f));
  float w = -0.05299540236592293f;
  w = fmaf(w, t, 0.15280704200267792f);
  w = fmaf(w, t, -0.06572140008211136f);
  w = fmaf(w, t, 0.11840226501226425f);
  w = fmaf(w, t, 0.06339198350906372f);
  w = fmaf(w, t, 0.09283988922834396f);
  w = fmaf(w, t, 0.09552200883626938f);
  w = fmaf(w, t, 0.09575380384922028f);
  return w * t;
}

template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if constexpr (ACT == KRONQ_ACT_RELU) return z < 0.f ? 0.f : z;
  if constexpr (ACT == KRONQ_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  if constexpr (ACT == KRONQ_ACT_GELU) {
    const float tail = __expf(-0.5f * z * z) * tail_ratio(fabsf(z));
    return z * (z < 0.f ? tail : 1.f - tail);
  }
  if constexpr (ACT == KRONQ_ACT_GELU_TANH) {
    const float v2 = 1.5957691216f * fmaf(0.044715f * z * z, z, z);
    return __fdividef(z, 1.f + __expf(-v2));
  }
  return z;
}

// Four values, the activation chosen at run time, for the epilogues that run once
// a CTA (few tokens, split k). Not inlined: what such an epilogue costs is fetching
// its code, and unrolled copies of five activations took longer to fetch (8000 cycles
// a tile) than the tile took to multiply. The pair kernel's epilogue over whole tiles
// has the activation as a template argument and its one act_f inlined: 1021 tokens
// 1351 -> 2003 with gelu_tanh take 14.3 us, 15.1 with calls.
template <int ACT>
__device__ __forceinline__ float4 act4_f(float4 z) {
  return make_float4(act_f<ACT>(z.x), act_f<ACT>(z.y), act_f<ACT>(z.z), act_f<ACT>(z.w));
}
static __device__ __noinline__ float4 act4(int act, float4 z) {
  switch (act) {
    case KRONQ_ACT_RELU: return act4_f<KRONQ_ACT_RELU>(z);
    case KRONQ_ACT_SILU: return act4_f<KRONQ_ACT_SILU>(z);
    case KRONQ_ACT_GELU: return act4_f<KRONQ_ACT_GELU>(z);
    case KRONQ_ACT_GELU_TANH: return act4_f<KRONQ_ACT_GELU_TANH>(z);
    default: return z;
  }
}
// value and derivative
template <int ACT>
__device__ __forceinline__ void act_df(float z, float &h, float &dh) {
  if constexpr (ACT == KRONQ_ACT_RELU) {
    h = z < 0.f ? 0.f : z;
    dh = z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);   // NaN stays
  } else if constexpr (ACT == KRONQ_ACT_SILU) {
    const float s = logistic(z);
    h = z * s;
    dh = fmaf(h, 1.f - s, s);
  } else if constexpr (ACT == KRONQ_ACT_GELU) {
    const float e = __expf(-0.5f * z * z), tail = e * tail_ratio(fabsf(z));
    const float c = z < 0.f ? tail : 1.f - tail;
    h = z * c;
    dh = fmaf(z * 0.39894228f, e, c);
  } else if constexpr (ACT == KRONQ_ACT_GELU_TANH) {
    // beyond |z| = 30 the derivative's second term is 0 in fp32; the clamp
    // keeps its polynomial finite there
    const float zc = fminf(fmaxf(z, -30.f), 30.f);
    const float e = __expf(-1.5957691216f * fmaf(0.044715f * zc * zc, z, z));
    const float s = __fdividef(1.f, 1.f + e);
    // 1 - s is e s: the difference drops up to 2^-23, and z dv2 is 36 at z = 5
    const float r = e < 1.f ? e * s : 1.f - s;
    const float dv2 = 1.5957691216f * fmaf(3.f * 0.044715f * zc, zc, 1.f);
    h = z * s;
    dh = fmaf(h * r, dv2, s);
  } else {
    h = z;
    dh = 1.f;
  }
}

}  // namespace kronq
