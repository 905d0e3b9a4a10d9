// E4M3 codes in blocks of 128: the scale of a block is max|x| / 448, at least
// the smallest normal float (so that it and its reciprocal keep their bits; a
// block whose largest magnitude is below 448 * 2^-126 then uses only the lower
// codes), 0 for a block of zeros, NaN for one that holds a value that is not
// finite.  A code is E4M3(x * (1 / scale)), to the nearest, ties to even: x
// times the rounded reciprocal is within 1.5 float32 roundings of x / scale, so
// a code differs from that of the exact quotient only where this lies that
// close to the middle between two codes.
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
__device__ __forceinline__ float inverse_scale(float scale) { return scale == 0.f ? 0.f : __fdiv_rn(1.f, scale); }

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

}  // namespace codes
}  // namespace forge
