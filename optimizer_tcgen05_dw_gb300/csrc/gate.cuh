// The gate's activation and its gradient, in float32.
//
// The activations are g s with a sigmoid s:  SiLU: s = sigma(g);  GELU (tanh
// form): (1 + tanh z) / 2 = sigma(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3).
// So act' = s + g s (1 - s) d with d = 1 or 2 z'(g): no difference of nearly
// equal numbers at either end, as 1 + tanh would be.
#pragma once

#include "launch.h"

namespace forge {

// s and d of g (see above).  Past |g| = 50 the polynomial's sigmoid is 0 or 1
// to the last bit: the bound keeps its powers finite (an infinite d times a
// zero 1 - s would be NaN).  The fast exponential is off by 2^-22 + |z| 2^-23 of
// itself and the fast quotient by 2^-22, far below bf16's 2^-8; an exponential
// past the largest float, or a sum past 2^126, gives s = 0.
template <int ACT>
__device__ __forceinline__ float gate_sigmoid(float g, float& d) {
  float z = g;
  d = 1.f;
  if (ACT == kActGeluTanh) {
    constexpr float c = 1.5957691216057308f, k = 0.044715f;  // 2 sqrt(2 / pi)
    const float b = fminf(fmaxf(g, -50.f), 50.f), b2 = b * b;
    z = c * b * (1.f + k * b2);
    d = c * (1.f + 3.f * k * b2);
  }
  return __fdividef(1.f, 1.f + __expf(-z));
}

template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
  float d;
  return g * gate_sigmoid<ACT>(g, d) * u;
}
__device__ __forceinline__ float gated(int act, float g, float u) {
  return act == kActSilu ? gated<kActSilu>(g, u) : gated<kActGeluTanh>(g, u);
}

// From dA, G and U: dG, dU and Y.
template <int ACT>
__device__ __forceinline__ void gated_gradient(float da, float g, float u, float& dg, float& du, float& y) {
  float d;
  const float s = gate_sigmoid<ACT>(g, d), a = g * s;
  du = da * a;
  dg = da * u * (s + a * (1.f - s) * d);
  y = a * u;
}

}  // namespace forge
