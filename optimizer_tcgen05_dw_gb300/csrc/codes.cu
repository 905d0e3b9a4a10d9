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
constexpr int kAhead = 4;  // blocks (vectors, in the other direction) a thread has in flight

__device__ __forceinline__ void load_x8(const uint16_t* x, int64_t e, float (&v)[8]) { load_bf16x8(x, e, v); }
__device__ __forceinline__ void load_x8(const float* x, int64_t e, float (&v)[8]) { load8(x + e, v); }
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

// Blocks of one row: half a warp takes a block, eight elements a lane.
template <typename X>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const X* x, uint8_t* out, float* scale, int64_t blocks,
                                                                 int V, int NB) {
  const int l = threadIdx.x & 15;
  const int64_t half = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
  const bool whole = V == NB * 16;
  for (int64_t b0 = half; b0 - half < blocks; b0 += step * kAhead) {  // uniform over the warp but for its end
    float v[kAhead][8];
    int64_t at[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t b = b0 + i * step;
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
      if (at[i] >= 0) {
        load_x8(x, at[i], v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float a = max8(v[i]);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) a = codes::max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
      const float s = codes::block_scale(a);
      const int64_t b = b0 + i * step;
      if (l == 0 && b < blocks) scale[b] = s;
      if (at[i] >= 0) *reinterpret_cast<uint2*>(out + at[i]) = encode8(v[i], codes::inverse_scale(s));
    }
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
  float v[kRows][8], a = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t t = t0 + i * (kThreads / 16) + (threadIdx.x >> 4);
    if (t < T && c < V) {
      load_x8(x, (t * V + c) * 8, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) a = codes::max_nan(a, max8(v[i]));
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
    if (t < T && c < V) *reinterpret_cast<uint2*>(out + (t * V + c) * 8) = encode8(v[i], inv);
  }
}

// Codes to values, eight a thread: value = code * scale (float32), rounded once.
template <typename X>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* in, const float* scale, X* x, int64_t vectors,
                                                              int V, int NB, bool square) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  const bool flat = !square && V == NB * 16;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i0 < vectors; i0 += step * kAhead) {
    uint2 c[kAhead];
    float s[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = i0 + i * step;
      if (at >= vectors) continue;
      c[i] = reinterpret_cast<const uint2*>(in)[at];
      int64_t b = at >> 4;
      if (!flat) {
        const int64_t t = vectors <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(at) / static_cast<uint32_t>(V)) : at / V;
        b = (square ? t / codes::kBlock : t) * NB + ((at - t * V) >> 4);
      }
      s[i] = scale[b];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = i0 + i * step;
      if (at >= vectors) continue;
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
}

int blocks_for(int64_t threads, int num_sms) {
  const int64_t need = (threads + kThreads - 1) / kThreads, most = int64_t{8} * num_sms;
  return static_cast<int>(need < most ? need : most);
}

template <typename X>
cudaError_t quantize(const CodesParams& p, int num_sms, cudaStream_t s) {
  const int V = static_cast<int>(p.cols / 8), NB = (V + 15) / 16;
  const X* x = static_cast<const X*>(p.x);
  if (p.square) {
    const int64_t tiles = (p.rows + codes::kBlock - 1) / codes::kBlock * NB;
    quantize_square_kernel<X><<<static_cast<unsigned>(tiles), kThreads, 0, s>>>(x, p.codes, p.scale, p.rows, V, NB);
  } else {
    const int64_t blocks = p.rows * NB;
    quantize_rows_kernel<X><<<blocks_for(blocks * 16, num_sms), kThreads, 0, s>>>(x, p.codes, p.scale, blocks, V, NB);
  }
  return cudaGetLastError();
}

template <typename X>
cudaError_t dequantize(const CodesParams& p, int num_sms, cudaStream_t s) {
  const int V = static_cast<int>(p.cols / 8), NB = (V + 15) / 16;
  const int64_t vectors = p.rows * V;
  dequantize_kernel<X><<<blocks_for(vectors, num_sms), kThreads, 0, s>>>(p.codes, p.scale, static_cast<X*>(const_cast<void*>(p.x)),
                                                                       vectors, V, NB, p.square != 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_e4m3(bool fp32, const CodesParams& p, int num_sms, cudaStream_t s) {
  return fp32 ? quantize<float>(p, num_sms, s) : quantize<uint16_t>(p, num_sms, s);
}

cudaError_t launch_dequantize_e4m3(bool fp32, const CodesParams& p, int num_sms, cudaStream_t s) {
  return fp32 ? dequantize<float>(p, num_sms, s) : dequantize<uint16_t>(p, num_sms, s);
}

}  // namespace forge
