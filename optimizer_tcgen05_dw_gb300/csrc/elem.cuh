// Groups of eight consecutive elements of a weight, gradient or state tensor:
// vector loads and stores, the INT8 code of a block shared by the lanes that
// hold it, and the stochastic rounding of eight weights.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "optim.cuh"

namespace forge {

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Max over the `lanes` lanes (a power of two up to 32) of an aligned lane
// group; all 32 lanes call it.
__device__ __forceinline__ float group_max(float a, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  return a;
}

// Codes are formed and read without the conversion unit (int <-> float casts
// and rint run there at a quarter of the float rate): code_f32, and
// code_round_fast with all eight redone from the exact quotient when one lies
// near a half-integer or is not finite.  The values are dequant's and quant's
// for any v that `a` is the absmax of: an unsigned code clamps at 0 itself (a
// quantiser's caller may give negative values, a second moment has none).
template <bool SIGNED>
__device__ __forceinline__ void decode8(uint2 c, float a, float (&v)[8]) {
  const float s = dev::dvd(a, SIGNED ? 127.f : 255.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = dev::mul(dev::code_f32<SIGNED>(j < 4 ? c.x : c.y, j & 3), s);
}

template <bool SIGNED>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float a) {
  if (a == 0.f) return make_uint2(0u, 0u);
  const float st = dev::dvd(a, SIGNED ? 127.f : 255.f), inv = dev::dvd(1.f, st);
  uint32_t k[8];  // the low byte of each is the code
  bool any = !(fabsf(inv) <= 3.0e38f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bool redo;
    const float y = dev::mul(v[j], inv);
    k[j] = dev::code_round_fast<SIGNED>(SIGNED ? y : fmaxf(y, 0.f), redo);  // a NaN's code is 0 too
    any |= redo;
  }
  if (any) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bool near;
      k[j] = static_cast<uint32_t>(dev::code_round<SIGNED>(dev::dvd(v[j], st), near));
    }
  }
  return make_uint2(__byte_perm(__byte_perm(k[0], k[1], 0x0040u), __byte_perm(k[2], k[3], 0x0040u), 0x5410u),
                    __byte_perm(__byte_perm(k[4], k[5], 0x0040u), __byte_perm(k[6], k[7], 0x0040u), 0x5410u));
}

template <bool SIGNED>
__device__ __forceinline__ void load_codes8(const void* base, int64_t e0, float a, float (&v)[8]) {
  decode8<SIGNED>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + e0), a, v);
}

template <bool SIGNED>
__device__ __forceinline__ void store_codes8(void* base, int64_t e0, float a, const float (&v)[8]) {
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + e0) = encode8<SIGNED>(v, a);
}

__device__ __forceinline__ void load_bf16x8(const void* base, int64_t e0, float (&v)[8]) {
  const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + e0);
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = dev::bf16_to_f32(w[j] & 0xFFFFu);
    v[2 * j + 1] = dev::bf16_to_f32(w[j] >> 16);
  }
}

// Eight values to bf16 (dev::bf16_rne), packed in pairs: by the conversion
// instruction, which rounds the same way and differs only in the NaN it gives,
// so when none of the eight is a NaN.
__device__ __forceinline__ uint4 pack_rne_bf16x8(const float (&v)[8]) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) nan |= v[j] != v[j];
  uint32_t o[4];
  if (!nan) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = dev::bf16_rne(v[2 * j]) | (dev::bf16_rne(v[2 * j + 1]) << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void store_bf16x8_rne(void* base, int64_t e0, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e0) = pack_rne_bf16x8(v);
}

// Eight weights to bf16 by stochastic rounding (dev::bf16_sr), packed in
// pairs.  When all eight are finite (w * 0 is then 0; an infinite or NaN w
// makes the sum NaN), each is its bit pattern plus its 16 random bits, upper
// half kept: the two halves of a word come from one byte permutation.
__device__ __forceinline__ uint4 pack_sr_bf16x8(const float* w, uint4 rnd) {
  float probe = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) probe = __fmaf_rn(w[j], 0.f, probe);
  const uint32_t rw[4] = {rnd.x, rnd.y, rnd.z, rnd.w};
  uint32_t o[4];
  if (probe == probe) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = __byte_perm(__float_as_uint(w[2 * j]) + (rw[j] & 0xFFFFu),
                         __float_as_uint(w[2 * j + 1]) + (rw[j] >> 16), 0x7632u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = dev::bf16_sr(w[2 * j], dev::sr_bits(rnd, 2 * j)) |
             (dev::bf16_sr(w[2 * j + 1], dev::sr_bits(rnd, 2 * j + 1)) << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace forge
