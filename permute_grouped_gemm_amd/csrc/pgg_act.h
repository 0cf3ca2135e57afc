// Activations of the gated products, and their derivatives, in fp32.
#pragma once

#include "pgg_device.h"

namespace pgg {

namespace {

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

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
    du = 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * g * g);
  }
  value = g * s;
  slope = s + g * s * (1.0f - s) * du;
}

}  // namespace

}  // namespace pgg
