// Activations and weights to E4M3 codes in blocks of 128 and back (codes.cuh
// has the format): a scale for each 128 elements of a row, or for each
// 128 x 128 of a matrix.  The last block of a row, and the last rows' blocks,
// may be short.
//
// The floor is the traffic: 2 (bf16) or 4 (float32) bytes an element on one
// side, 1 on the other, 4 / 128 of scales.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "elem.cuh"
#include "launch.h"

namespace forge {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;  // vectors of codes a thread has in flight (16384 x 14336 to bf16: 104 us, one 123)

__device__ __forceinline__ void store_x8(uint16_t* x, int64_t e, const float (&v)[8]) { store_bf16x8_rne(x, e, v); }
__device__ __forceinline__ void store_x8(float* x, int64_t e, const float (&v)[8]) { store8(x + e, v); }

__device__ __forceinline__ float max8(const float (&v)[8]) {
  float a = codes::max_nan(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
  for (int j = 2; j < 8; ++j) a = codes::max_nan(a, fabsf(v[j]));
  return a;
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  return make_uint2(codes::encode4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    codes::encode4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// Eight values as they were loaded (zeros where `at` is negative).  The largest
// magnitude of bf16 is that of its bits without the sign, a NaN's above all.
template <typename X>
struct Eight;
template <>
struct Eight<uint16_t> {
  uint4 r;
  __device__ __forceinline__ void load(const uint16_t* x, int64_t at) {
    r = at >= 0 ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float top() const {
    constexpr uint32_t m = 0x7FFF7FFFu;
    const uint32_t t = __vmaxu2(__vmaxu2(r.x & m, r.y & m), __vmaxu2(r.z & m, r.w & m));
    return __uint_as_float(max(t << 16, t & 0xFFFF0000u));
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* x, int64_t at) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    a = at >= 0 ? reinterpret_cast<const float4*>(x + at)[0] : zero;
    b = at >= 0 ? reinterpret_cast<const float4*>(x + at)[1] : zero;
  }
  __device__ __forceinline__ float top() const {
    float v[8];
    values(v);
    return max8(v);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// Blocks of one row: half a warp takes a block, eight elements a lane, and a
// warp eight blocks one after the other, loaded together.  The maxima of a
// half's four blocks are reduced in one tree, every lane ending with one of
// them: five exchanges in place of sixteen, and one scale and reciprocal a lane
// in place of four (16384 x 14336 bf16: 132 us so; 102 with
// the values kept as they were loaded, in half the registers).
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const X* x, uint8_t* out, float* scale, int64_t blocks,
                                                                 int V, int NB) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  const int lane = threadIdx.x & 31, l = lane & 15;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * 8 + (lane >> 4);
  const bool whole = V == NB * 16;
  Eight<X> v[4];
  float a[4];
  int64_t at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t b = first + 2 * i;
    at[i] = -1;
    if (b < blocks) {
      if (whole) {
        at[i] = (b * 16 + l) * 8;
      } else {
        const int64_t t = b / NB;
        const int c = static_cast<int>(b - t * NB) * 16 + l;
        if (c < V) at[i] = (t * V + c) * 8;
      }
    }
    v[i].load(x, at[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = v[i].top();
  const bool b0 = l & 1, b1 = l & 2;  // this lane ends with block 2 b0 + b1 of the four
  const float k0 = codes::max_nan(b0 ? a[2] : a[0], __shfl_xor_sync(kAll, b0 ? a[0] : a[2], 1));
  const float k1 = codes::max_nan(b0 ? a[3] : a[1], __shfl_xor_sync(kAll, b0 ? a[1] : a[3], 1));
  float k = codes::max_nan(b1 ? k1 : k0, __shfl_xor_sync(kAll, b1 ? k0 : k1, 2));
  k = codes::max_nan(k, __shfl_xor_sync(kAll, k, 4));
  k = codes::max_nan(k, __shfl_xor_sync(kAll, k, 8));
  const float s = codes::block_scale(k), inv = codes::inverse_scale(s);
  const int64_t mine = first + 2 * (2 * b0 + b1);
  if (l < 4 && mine < blocks) scale[mine] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f = __shfl_sync(kAll, inv, (lane & 16) | (i >> 1) | ((i & 1) << 1));
    float w[8];
    v[i].values(w);
    if (at[i] >= 0) *reinterpret_cast<uint2*>(out + at[i]) = encode8(w, f);
  }
}

// Blocks of 128 x 128: a block of threads takes one, half a warp a row of it.
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_square_kernel(const X* x, uint8_t* out, float* scale, int64_t T, int V,
                                                                   int NB) {
  constexpr int kRows = codes::kBlock / (kThreads / 16);  // rows a thread has a vector of
  __shared__ float top[kThreads / 32];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / NB) * codes::kBlock;
  const int nb = blockIdx.x % NB, c = nb * 16 + (threadIdx.x & 15);
  Eight<X> v[kRows];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t t = t0 + i * (kThreads / 16) + (threadIdx.x >> 4);
    v[i].load(x, t < T && c < V ? (t * V + c) * 8 : -1);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) a = codes::max_nan(a, v[i].top());
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) a = codes::max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = codes::max_nan(a, top[i]);
  const float s = codes::block_scale(a), inv = codes::inverse_scale(s);
  if (threadIdx.x == 0) scale[blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t t = t0 + i * (kThreads / 16) + (threadIdx.x >> 4);
    float w[8];
    v[i].values(w);
    if (t < T && c < V) *reinterpret_cast<uint2*>(out + (t * V + c) * 8) = encode8(w, inv);
  }
}

// Codes to values, eight a lane, a warp 32 U vectors of them one after the
// other: value = code * scale (float32), rounded once.
template <typename X, int U>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* in, const float* scale, X* x, int64_t vectors,
                                                              int V, int NB, bool square) {
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 * U) + (threadIdx.x & 31);
  const bool flat = !square && V == NB * 16;
  uint2 c[U];
  float s[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t at = first + 32 * i;
    if (at >= vectors) break;
    c[i] = reinterpret_cast<const uint2*>(in)[at];
    int64_t b = at >> 4;
    if (!flat) {
      const int64_t t = vectors <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(V)) : at / V;
      b = (square ? t / codes::kBlock : t) * NB + ((at - t * V) >> 4);
    }
    s[i] = scale[b];
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t at = first + 32 * i;
    if (at >= vectors) break;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 d = codes::decode2((j < 2 ? c[i].x : c[i].y) >> (16 * (j & 1)));
      v[2 * j] = d.x * s[i];
      v[2 * j + 1] = d.y * s[i];
    }
    store_x8(x, at * 8, v);
  }
}

// Blocks of threads for `items` of which one takes `each`.
unsigned blocks_for(int64_t items, int each) { return static_cast<unsigned>((items + each - 1) / each); }

template <typename X>
cudaError_t quantize(const CodesParams& p, cudaStream_t s) {
  const int V = static_cast<int>(p.cols / 8), NB = (V + 15) / 16;
  const X* x = static_cast<const X*>(p.x);
  if (p.square) {
    const int64_t tiles = (p.rows + codes::kBlock - 1) / codes::kBlock * NB;
    quantize_square_kernel<X><<<static_cast<unsigned>(tiles), kThreads, 0, s>>>(x, p.codes, p.scale, p.rows, V, NB);
  } else {
    const int64_t blocks = p.rows * NB;
    quantize_rows_kernel<X><<<blocks_for(blocks, kThreads / 4), kThreads, 0, s>>>(x, p.codes, p.scale, blocks, V, NB);
  }
  return cudaGetLastError();
}

template <typename X>
cudaError_t dequantize(const CodesParams& p, cudaStream_t s) {
  const int V = static_cast<int>(p.cols / 8), NB = (V + 15) / 16;
  const int64_t vectors = p.rows * V;
  dequantize_kernel<X, kAhead><<<blocks_for(vectors, kThreads * kAhead), kThreads, 0, s>>>(
      p.codes, p.scale, static_cast<X*>(const_cast<void*>(p.x)), vectors, V, NB, p.square != 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_e4m3(bool fp32, const CodesParams& p, cudaStream_t s) {
  return fp32 ? quantize<float>(p, s) : quantize<uint16_t>(p, s);
}

cudaError_t launch_dequantize_e4m3(bool fp32, const CodesParams& p, cudaStream_t s) {
  return fp32 ? dequantize<float>(p, s) : dequantize<uint16_t>(p, s);
}

}  // namespace forge
