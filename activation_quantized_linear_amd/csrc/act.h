// The epilogue of a linear's output, y = act(v) * mul + residual, and its gradients
// (internal to libaql.so): the activations, the term that the W8A16 kernels apply to
// each sum, and the launcher of the gradient kernel. Arguments are validated by the C
// ABI layer.
#pragma once

#include <type_traits>

#include "common.h"

namespace aql {

enum ActKind : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };
constexpr int kActKinds = 5;

// 1 / (1 + e^-z). The hardware's exponential and reciprocal are each within an ulp or so
// (the exponential of |z| <= 88 within 2^-17, from the rounding of z log2 e), far inside the 2^-8 of
// the bf16 value that every result here becomes. e^-z past float32 is infinite
// and the value 0.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

// The argument of the tanh form's sigmoid, 2 sqrt(2 / pi) (z + 0.044715 z^3): past
// |z| = 64 the sigmoid is 0 or 1 whatever it is, and the cube must not overflow.
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  const float c = fminf(fmaxf(z, -64.0f), 64.0f);
  return 1.59576912f * c * fmaf(0.044715f * c, c, 1.0f);
}

// Phi(z) of the normal distribution, and e^(-z^2 / 2). Phi(-|z|) = P(t) e^(-z^2 / 2) with
// t = 1 / (1 + 0.3182 |z|), P fitted for this file: a weighted least-squares fit of degree 8 to
// erfcx(x) / 2, x = |z| / sqrt 2 in [0, 20], its relative error held below 4e-7 over
// the whole tail (the exponent's own rounding adds up to 8e-6 at |z| = 13). A third of
// erfcf's instructions: the linear of M = 2048, N = 14336, K = 4096 with gelu took 256 us with that,
// 224 without an activation.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.318198055f, a, 1.0f));
  float p = 0.0347404033f;
  p = fmaf(p, t, -0.125645936f);
  p = fmaf(p, t, 0.114017196f);
  p = fmaf(p, t, 0.0112389755f);
  p = fmaf(p, t, 0.0990576223f);
  p = fmaf(p, t, 0.112606712f);
  p = fmaf(p, t, 0.127045199f);
  p = fmaf(p, t, 0.126940012f);
  e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
  const float left = p * t * e;
  return z < 0.0f ? left : 1.0f - left;
}

// act(z). The tanh form is z times a sigmoid, 0.5 (1 + tanh u) = 1 / (1 + e^-2u), and the
// erf form computes its left tail as such: neither loses it in a difference from 1.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == kActRelu) return z < 0.0f ? 0.0f : z;  // (NaN stays NaN)
  if constexpr (ACT == kActGelu) {
    float e;
    return z * normal_cdf(z, e);
  }
  if constexpr (ACT == kActGeluTanh) return z * sigmoid(gelu_tanh_arg(z));
  if constexpr (ACT == kActSilu) return z * sigmoid(z);
  return z;
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void act_value_grad(float z, float &a, float &d) {
  if constexpr (ACT == kActRelu) {
    a = act_value<ACT>(z);
    d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    float e;
    const float c = normal_cdf(z, e);
    a = z * c;
    d = fmaf(z * 0.398942280f, e, c);
  } else if constexpr (ACT == kActGeluTanh) {
    const float g = sigmoid(gelu_tanh_arg(z)), c = fminf(fmaxf(z, -64.0f), 64.0f);
    a = z * g;
    d = fmaf(z * g * (1.0f - g), 1.59576912f * fmaf(0.134145f * c, c, 1.0f), g);
  } else if constexpr (ACT == kActSilu) {
    const float g = sigmoid(z);
    a = z * g;
    d = fmaf(a, 1.0f - g, g);
  } else {
    a = z;
    d = 1.0f;
  }
}

// f(constant of the activation): one branch, outside the loops over values.
template <class F>
__device__ __forceinline__ void act_dispatch(int act, F &&f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

// What a W8A16 kernel applies to v = scale * sum + bias, all in float32, before the one
// rounding to bf16. Each output's mul and residual are read by the thread (in the tiled
// kernels: the workgroup, before a barrier) that then writes it, so y may be either.
struct ActTerm {
  static constexpr bool on = false, act = true;
  int kind;
  const uint16_t *mul;  // [M, N] or NULL
  const uint16_t *res;  // [M, N] or NULL
  uint16_t *pre;        // [M, N] or NULL: v itself, rounded
  int64_t N;
  __device__ __forceinline__ float add(int64_t m, int64_t n, float v) const {
    const int64_t i = m * N + n;
    const float f = mul ? bf16_to_f32(mul[i]) : 1.0f;
    const float r = res ? bf16_to_f32(res[i]) : 0.0f;
    if (pre) pre[i] = f32_to_bf16_rne(v);
    act_dispatch(kind, [&](auto k) { v = act_value<decltype(k)::value>(v); });
    if (mul) v *= f;
    return res ? v + r : v;
  }
};

// dv = dy * mul * act'(pre), dmul = dy * act(pre) over n elements, all bf16; mul and
// dmul may be NULL.
hipError_t launch_act_mul_backward(const uint16_t *dy, const uint16_t *pre, int act,
                                   const uint16_t *mul, int64_t n, uint16_t *dv, uint16_t *dmul,
                                   hipStream_t st);

}  // namespace aql
