// The activation of a gated block: act(g) = g sigmoid(z(g)) with z = g (SiLU)
// or z = 2 sqrt(2 / pi) (g + 0.044715 g^3) (the tanh form of GELU, as
// (1 + tanh(y)) / 2 = sigmoid(2 y)), and its derivative
//   act'(g) = sigmoid(z) + g sigmoid(z) (1 - sigmoid(z)) z'(g).
#pragma once

#include <hip/hip_runtime.h>

#include "qlora_fp8.h"

namespace qlora {

// sigmoid s by the hardware's exponential and reciprocal, one unit in the last place
// each.  The exponent z log2 e is rounded, and so is log2 e, so the relative error
// grows with |z|: at most 2^-24 ((1 - s) (1.4 |z| + 2) + 3).  (exp2 is flushed to 0
// below 2^-126 and infinite above 2^128, where the sigmoid is 1 and 0.)
__device__ __forceinline__ float sigmoid_of(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}

constexpr float kGeluScale = 1.59576912f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

__device__ __forceinline__ float act_value(float g, int act) {
  const float z = act == QLORA_ACT_SILU ? g : kGeluScale * (g + kGeluCubic * g * g * g);
  return g * sigmoid_of(z);
}

// value and derivative
template <int kAct>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
  float z = g, dz = 1.0f;
  if constexpr (kAct != QLORA_ACT_SILU) {
    // g^2 stays finite, so that where the sigmoid is 0 or 1 its slope's 0
    // meets no infinity
    const float g2 = fminf(g * g, 1e30f);
    z = kGeluScale * (g + kGeluCubic * g2 * g);
    dz = kGeluScale * (1.0f + 3.0f * kGeluCubic * g2);
  }
  const float s = sigmoid_of(z);
  value = g * s;
  slope = __builtin_fmaf(value, kAct == QLORA_ACT_SILU ? 1.0f - s : (1.0f - s) * dz, s);
}

}  // namespace qlora
