// The activations of the gated block: act(g) = g·σ(h(g)) with σ the logistic
// function and h(g) = g (SiLU) or 2·sqrt(2/π)·(g + 0.044715·g³) (the tanh form of
// GELU: (1 + tanh(y))/2 = σ(2y)).
#pragma once

#include "host.h"

namespace qnf4 {

constexpr double kGeluSlope = 1.5957691216057307, kGeluCube = 0.044715;  // 2·sqrt(2/π)

// act(g), off by its exponent's roundings: with u = 2^-24, (6 + 3|h|)u of itself for SiLU,
// (6 + 8|h|)u for GELU (h is off by 5u of itself); below 2^-126 a step of fp32.  FAR:
// whether g may be below far_gate(act).  There exp(−h) passes 2^95 and more, the
// reciprocal of 1 + exp(−h) is exp(h) in fp32, and exp(h) is taken 2^64 times as large:
// the reciprocal instruction gives 0 for results below 2^-126, from h = −87 on, where g
// times them is still a normal number.
template <bool FAR = true>
__device__ __forceinline__ float gate_act(int act, float g) {
  float h = g;
  if (act == kActGeluTanh) h = (float)kGeluSlope * __builtin_fmaf((float)kGeluCube * g * g, g, g);
  const float x = h * -1.44269502f;
  if constexpr (FAR)
    if (x > 100.f) return g * __builtin_amdgcn_exp2f(64.f - x) * 0x1p-64f;
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x));
}
// (h = −69 and −66, x = 99.5 and 95.8)
__device__ __forceinline__ float far_gate(int act) { return act == kActGeluTanh ? -9.f : -69.f; }

}  // namespace qnf4
