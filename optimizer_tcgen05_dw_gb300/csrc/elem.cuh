// Groups of eight consecutive elements of a weight, gradient or state tensor:
// vector loads and stores, and the INT8 code of a block shared by the lanes
// that hold it.  Used by the elementwise kernels (elementwise.cu, multi.cu).
#pragma once

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

template <bool SIGNED>
__device__ __forceinline__ void load_codes8(const void* base, int64_t e0, float a, float (&v)[8]) {
  const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(base) + e0);
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = (w[j >> 2] >> (8 * (j & 3))) & 0xFFu;
    const int code = SIGNED ? static_cast<int>(static_cast<int8_t>(b)) : static_cast<int>(b);
    v[j] = dev::dequant<SIGNED>(code, a);
  }
}

template <bool SIGNED>
__device__ __forceinline__ void store_codes8(void* base, int64_t e0, float a, const float (&v)[8]) {
  uint32_t w[2] = {0u, 0u};
  const float st = dev::dvd(a, SIGNED ? 127.f : 255.f), inv = dev::dvd(1.f, st);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j >> 2] |= (static_cast<uint32_t>(dev::quant_recip<SIGNED>(v[j], a, st, inv)) & 0xFFu) << (8 * (j & 3));
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + e0) = make_uint2(w[0], w[1]);
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

__device__ __forceinline__ void store_bf16x8_rne(void* base, int64_t e0, const float (&v)[8]) {
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = dev::bf16_rne(v[2 * j]) | (dev::bf16_rne(v[2 * j + 1]) << 16);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + e0) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace forge
