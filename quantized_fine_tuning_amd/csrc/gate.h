// The activations of the gated block: act(g) = g·σ(h(g)) with σ the logistic
// function and h(g) = g (SiLU) or 2·sqrt(2/π)·(g + 0.044715·g³) (the tanh form of
// GELU: (1 + tanh(y))/2 = σ(2y)).
#pragma once

#include "host.h"

namespace qnf4 {

constexpr double kGeluSlope = 1.5957691216057307, kGeluCube = 0.044715;  // 2·sqrt(2/π)

// act(g) within a few ulps of fp32: h, an exponential and a reciprocal of 1 ulp each.
__device__ __forceinline__ float gate_act(int act, float g) {
  float h = g;
  if (act == kActGeluTanh) h = (float)kGeluSlope * __builtin_fmaf((float)kGeluCube * g * g, g, g);
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(h * -1.44269502f));
}

}  // namespace qnf4
