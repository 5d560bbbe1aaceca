// act.cuh -- the activations of the gated feed-forward block.
//
//   silu(g) = g / (1 + exp(-g))
//   gelu_tanh(g) = g / (1 + exp(-2z)), z = sqrt(2/pi) (g + 0.044715 g^3):
//     0.5 (1 + tanh z) is the logistic function of 2z, which keeps its
//     relative accuracy where 1 + tanh z cancels.
#pragma once

#include <cuda_runtime.h>

#include <cfloat>

#include "rra.h"

namespace rra {

// sigma = logistic(k(g)), *slope = k'(g)
template <int ACT>
__device__ __forceinline__ float gate_sigma(float g, float* slope) {
  float k = g;
  *slope = 1.f;
  if constexpr (ACT == RRA_ACT_GELU_TANH) {
    constexpr float c = 1.5957691216057308f;  // 2 sqrt(2/pi)
    k = c * g * fmaf(0.044715f * g, g, 1.f);
    *slope = c * fmaf(3.f * 0.044715f * g, g, 1.f);
  }
  return __fdividef(1.f, 1.f + __expf(-k));
}

// act'(g) = sigma (1 + g k'(g) (1 - sigma)) of what gate_sigma gave.  gelu's g
// k'(g) grows as g^3 and passes float32's range at |g| = 1.2e13, where sigma
// is 0 or 1: held finite, its product with the 0 is 0 (and the slope 0 or 1).
template <int ACT>
__device__ __forceinline__ float gate_slope(float g, float sigma, float slope) {
  float z = g * slope;
  if constexpr (ACT == RRA_ACT_GELU_TANH) z = fminf(fmaxf(z, -FLT_MAX), FLT_MAX);
  return sigma * fmaf(z, 1.f - sigma, 1.f);
}

}  // namespace rra
