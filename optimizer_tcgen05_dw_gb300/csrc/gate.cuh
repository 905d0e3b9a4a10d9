// The gate's activation and its gradient, in float32.
//
// The activations are g s with a sigmoid s:  SiLU: s = sigma(g);  GELU (tanh
// form): (1 + tanh z) / 2 = sigma(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3).
// So act' = s + g s (1 - s) d with d = 1 or 2 z'(g).  With e = exp(-|x|) the
// sigmoid and its complement are 1 / (1 + e) and e / (1 + e), whichever x's sign
// makes which: no end is a difference of nearly equal numbers, as 1 + tanh or
// 1 - s would be, and e only gets small, so that s keeps float32's whole range
// (1 / (1 + exp(-x)) is 0 from x = -87.3 on, where g s is still 1e-36).
#pragma once

#include "launch.h"

namespace forge {

struct Gate {
  float s, c, d;  // the sigmoid, 1 - s, and d (see above)
};

// Past |g| = 50 the polynomial's sigmoid is 0 or 1 to the last bit: the bound
// keeps its powers finite (an infinite d times a zero c would be NaN).  The fast
// exponential is off by 2^-22 + |x| 2^-23 of itself (by a few 2^-149 below
// 2^-126) and the fast quotient, of 1 + e in [1, 2], by 2^-22: far below bf16's 2^-8.
template <int ACT>
__device__ __forceinline__ Gate gate(float g) {
  float x = g;
  Gate r = {0.f, 0.f, 1.f};
  if (ACT == kActGeluTanh) {
    constexpr float c = 1.5957691216057308f, k = 0.044715f;  // 2 sqrt(2 / pi)
    const float b = fminf(fmaxf(g, -50.f), 50.f), b2 = b * b;
    x = c * b * (1.f + k * b2);
    r.d = c * (1.f + 3.f * k * b2);
  }
  const float e = __expf(-fabsf(x)), most = __fdividef(1.f, 1.f + e), least = e * most;
  r.s = x > 0.f ? most : least;
  r.c = x > 0.f ? least : most;
  return r;
}

template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
  return g * gate<ACT>(g).s * u;
}
__device__ __forceinline__ float gated(int act, float g, float u) {
  return act == kActSilu ? gated<kActSilu>(g, u) : gated<kActGeluTanh>(g, u);
}

// From dA, G and U: dG, dU and Y.
template <int ACT>
__device__ __forceinline__ void gated_gradient(float da, float g, float u, float& dg, float& du, float& y) {
  const Gate r = gate<ACT>(g);
  const float a = g * r.s;
  du = da * a;
  dg = da * u * (r.s + a * r.c * r.d);
  y = a * u;
}

}  // namespace forge
