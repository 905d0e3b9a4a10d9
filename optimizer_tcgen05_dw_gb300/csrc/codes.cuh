// E4M3 codes in blocks of 128: the scale of a block is max|x| / 448, at least
// the smallest normal float (so that it and its reciprocal keep their bits; a
// block whose largest magnitude is below 448 * 2^-126 then uses only the lower
// codes), 0 for a block of zeros, NaN for one that holds a value that is not
// finite.  A code is E4M3(x r), to the nearest, ties to even, with r the float32
// reciprocal of the scale (one division a block).  Reciprocal and product are
// rounded once each, so x r is x / scale to within 2^-23 of itself, and the code
// differs from that of the quotient only where this lies that close to the
// middle between two codes.
// (5 in 10^4 of 17 M bf16 values did, every one an exact tie of 448 x / max|x|:
// the two codes are equally near, and a quantiser that divides takes the other.)
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace forge {
namespace codes {

constexpr int kBlock = 128;
constexpr float kE4M3Max = 448.f;

// The larger of two magnitudes; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float block_scale(float amax) {
  const float a = amax + (amax - amax);  // an infinite maximum is no scale
  return a > 0.f ? fmaxf(__fdiv_rn(a, kE4M3Max), 0x1p-126f) : a;
}
__device__ __forceinline__ float inverse_scale(float scale) { return scale == 0.f ? 0.f : __frcp_rn(scale); }

// Two floats to codes, the first in the low byte: saturating at the largest
// finite code, NaN kept.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  return encode2(a, b) | (encode2(c, d) << 16);
}

// The values of the two codes in the low half of `c` (exact: every E4M3 value is a half).
__device__ __forceinline__ float2 decode2(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// A sum of code products is scaled by its blocks' two scales.  Their product
// may leave float32's range where the value does not, so the factor comes in
// two parts, value = (sum * p) * f, p a power of two: 1 unless xs * ws is below
// 2^-100 or above 2^100.  (Past the largest float f is that: sums that are not
// 0 go to infinity, 0 stays.)  A scale that is 0 or NaN gives that factor.
struct Factor {
  float f, p;
};
__device__ __forceinline__ Factor factor(float xs, float ws) {
  Factor r = {xs * ws, 1.f};
  if ((r.f <= 0x1p-100f || r.f >= 0x1p100f) && xs > 0.f && ws > 0.f) {
    const bool low = r.f < 1.f;
    const float k = low ? 0x1p32f : 0x1p-32f;
    r.f = fminf((xs * k) * (ws * k), 0x1.fffffep127f);
    r.p = low ? 0x1p-64f : 0x1p64f;
  }
  return r;
}

}  // namespace codes
}  // namespace forge
