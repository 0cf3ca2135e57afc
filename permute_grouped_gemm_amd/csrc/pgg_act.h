// Activations of the gated products, and their derivatives, in fp32.
#pragma once

#include "pgg_device.h"

namespace pgg {

namespace {

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// 1 / (1 + exp(-v)) from the hardware's base-2 exponential and reciprocal, each
// within 1 ulp.  The product -v log2 e is rounded, which makes the exponential
// off by |v| 2^-24 of itself; where it is that large a part of the sum, the
// result is near 0.  At the ends the exponential is 0 or inf, the result 1 or 0.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.4426950408889634f));
}

// silu(g) = g sigmoid(g);  gelu_tanh(g) = g sigmoid(2 c (g + a g^3)), which is
// g (1 + tanh(c (g + a g^3))) / 2.
template <int ACT>
__device__ __forceinline__ float activate(float g) {
  if constexpr (ACT == PGG_ACT_SILU) return g * sigmoid(g);
  return g * sigmoid(2.0f * kGeluC * (g + kGeluA * g * g * g));
}

// The same with the derivative: with s = sigmoid(u(g)), d/dg (g s) = s + g s (1 - s) u'(g).
template <int ACT>
__device__ __forceinline__ void activate_grad(float g, float& value, float& slope) {
  float s, du;
  if constexpr (ACT == PGG_ACT_SILU) {
    s = sigmoid(g);
    du = 1.0f;
  } else {
    s = sigmoid(2.0f * kGeluC * (g + kGeluA * g * g * g));
    // finite, so that it keeps the 0 of s (1 - s), which g is far past by then
    du = 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * fminf(g * g, 1e30f));
  }
  value = g * s;
  slope = s + g * s * (1.0f - s) * du;
}

}  // namespace

}  // namespace pgg
