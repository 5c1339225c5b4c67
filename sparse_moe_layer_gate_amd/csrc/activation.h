// The activations of the linear maps and their derivatives, in float32: a residual that is added to one, or a sum over many,
// sees no fewer digits. FAST, for tensors of bfloat16, takes the hardware's exponential and reciprocal, each a step or two of
// float32 off.
#pragma once

#include <hip/hip_runtime.h>

#include "moe_internal.h"

namespace moe {

constexpr float kInvSqrt2Pi = 0.3989422804f;
constexpr float kGeluTanhA = 0.7978845608f;   // sqrt(2 / pi)
constexpr float kGeluTanhB = 0.044715f;

template <bool FAST>
__device__ inline float act_sigmoid(float z) {
  return FAST ? __builtin_amdgcn_rcpf(1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
}

// Phi(-a) / exp(-a^2 / 2) for a >= 0: the mass beyond a of the normal distribution over its density's exponential, as a
// polynomial in 1 / (1 + c a) fitted to erfcx(a / sqrt 2) / 2 by relative error up to a = 14, where the exponential
// leaves float32: 1.6e-7 with eight terms. (Five terms, 3.2e-5, round 0.3% of bfloat16 results otherwise, with a residual
// or without, and take 0.3% less time at 8,191 x 5,120 -> 12,288 and 3 to 4% less at 6,517 x 320 -> 7,472.)
__device__ inline float normal_tail_ratio(float a) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.0f));
  float p = fmaf(0.0354239674f, t, -0.156159341f);
  p = fmaf(p, t, 0.204558206f);
  p = fmaf(p, t, -0.0520352263f);
  p = fmaf(p, t, 0.127692364f);
  p = fmaf(p, t, 0.100175782f);
  p = fmaf(p, t, 0.120712161f);
  p = fmaf(p, t, 0.119632006f);
  return p * t;
}

// e^(-x^2 / 2)
template <bool FAST>
__device__ inline float half_gauss(float x) {
  if (!FAST) return expf(-0.5f * x * x);
  const float s = x * 0.84932180028801904f;  // sqrt(log2(e) / 2)
  return __builtin_amdgcn_exp2f(-s * s);
}

// Factors are kept finite where the other one has vanished long before, so that an infinite z gives the limit and not a
// NaN; a NaN passes through the exponential.
template <bool FAST>
__device__ inline float act_gelu(float z) {
  // z Phi(z) = max(z, 0) - |z| Phi(-|z|): both tails keep their relative precision
  const float a = fabsf(z);
  const float q = half_gauss<FAST>(a) * normal_tail_ratio(a);
  return fmaf(-fminf(a, 30.0f), q, fmaxf(z, 0.f));
}

template <bool FAST>
__device__ inline float act_gelu_tanh(float z) {
  // (1 + tanh(u)) / 2 = sigmoid(2 u)
  const float u = kGeluTanhA * z * fmaf(kGeluTanhB * z, z, 1.0f);
  return fmaxf(z, -30.0f) * act_sigmoid<FAST>(2.0f * u);
}

template <bool FAST>
__device__ inline float act_silu(float z) {
  return fmaxf(z, -200.0f) * act_sigmoid<FAST>(z);
}

// N values at once: one branch on the activation (the same for every thread) for all of them.
template <bool FAST, int N>
__device__ inline void act_apply(int act, float* v) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // a NaN stays one
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_silu<FAST>(v[i]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_gelu<FAST>(v[i]);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = act_gelu_tanh<FAST>(v[i]);
      break;
    default:
      break;
  }
}

// d act / d z
template <bool FAST>
__device__ inline float slope_gelu(float z) {
  // Phi(z) + z phi(z)
  const float a = fabsf(z);
  if (a > 30.0f) return z > 0.f ? 1.f : 0.f;
  const float e = half_gauss<FAST>(a);
  const float q = e * normal_tail_ratio(a);
  const float d = a * e * kInvSqrt2Pi;
  return z > 0.f ? 1.0f - q + d : q - d;
}
template <bool FAST>
__device__ inline float slope_gelu_tanh(float z) {
  if (fabsf(z) > 30.0f) return z > 0.f ? 1.f : 0.f;
  const float u2 = 2.0f * kGeluTanhA * z * fmaf(kGeluTanhB * z, z, 1.0f);
  const float du2 = 2.0f * kGeluTanhA * fmaf(3.0f * kGeluTanhB * z, z, 1.0f);
  const float s = act_sigmoid<FAST>(u2);
  return fmaf(z * du2, s * (1.0f - s), s);
}
template <bool FAST>
__device__ inline float slope_silu(float z) {
  if (fabsf(z) > 200.0f) return z > 0.f ? 1.f : 0.f;
  const float s = act_sigmoid<FAST>(z);
  return fmaf(z * s, 1.0f - s, s);
}

// d[i] *= act'(z[i])
template <bool FAST, int N>
__device__ inline void act_slope_times(int act, const float* z, float* d) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] = z[i] > 0.f ? d[i] : z[i] != z[i] ? z[i] : 0.f * d[i];
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] *= z[i] != z[i] ? z[i] : slope_silu<FAST>(z[i]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] *= z[i] != z[i] ? z[i] : slope_gelu<FAST>(z[i]);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) d[i] *= z[i] != z[i] ? z[i] : slope_gelu_tanh<FAST>(z[i]);
      break;
    default:
      break;
  }
}

}  // namespace moe
