// Root-mean-square norm over the K columns of each token, with the residual's
// addition in front of it, its output in bf16 or E4M3, and its gradient.
//
//   h = bf16(x + residual)      (h = x without one; the stream the next
//                                layers and the gradient read)
//   r = 1 / sqrt(mean_k h^2 + eps)
//   y = h r w
//   dx = r (g - n mean_k(g n)) + dh,  g = dy w,  n = h r;   dw = sum_t dy n
//
// Everything between loads and stores is float32; h, y and dx are rounded to
// bf16 (nearest even) and codes to E4M3 (nearest even, saturating) once.
//
// The floor of each is its traffic: x, residual, h, y 2 B an element each,
// codes 1 B.  So a row is read once and held in registers (or, for the token-contiguous
// codes, shared memory between its reduction and its output.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "optim.cuh"
#include "ptx.cuh"

namespace forge {

namespace {

constexpr float kE4M3Max = 448.f;

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = dev::bf16_to_f32(a[j] & 0xFFFFu);
    f[2 * j + 1] = __uint_as_float(a[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Two floats to E4M3 codes (a in the low byte): nearest even, saturating at
// the largest finite value, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  float x[8], y[8];
  unpack8(a, x);
  unpack8(b, y);
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] += y[j];
  return pack8(x);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// 1 / sqrt(sum / K + eps)
__device__ __forceinline__ float inv_rms(float sum, int K, float eps) {
  return __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(K)) + eps);
}

// ---------------------------------------------------------------- forward

// A block takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; thread i holds
// vectors i, i + blockDim.x, .. (NV of them, eight columns each) of the row and
// of the weight.  Sum and maximum are reduced together: one barrier a row, the
// partials in alternating halves of `red`.
template <int NV, bool RES>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormParams p) {
  __shared__ float red[2][2][16];  // [row parity][sum, max][warp]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int V = p.K >> 3;
  const bool want_max = p.q != nullptr;
  const uint4* W = static_cast<const uint4*>(p.w);
  uint4 w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * blockDim.x;
    w[i] = v < V ? W[v] : make_uint4(0, 0, 0, 0);
  }
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    const uint4* x = static_cast<const uint4*>(p.x) + t * V;
    uint4 h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      h[i] = v < V ? x[v] : make_uint4(0, 0, 0, 0);
    }
    if (RES) {
      const uint4* res = static_cast<const uint4*>(p.res) + t * V;
      uint4* ho = static_cast<uint4*>(p.h) + t * V;
      uint4 r[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        r[i] = v < V ? res[v] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        h[i] = add_bf16x8(h[i], r[i]);
        if (v < V) ho[v] = h[i];
      }
    }
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float f[8], g[8];
      unpack8(h[i], f);
      unpack8(w[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = __fmaf_rn(f[j], f[j], sum);
        if (want_max) top = fmaxf(top, fabsf(f[j] * g[j]));
      }
    }
    sum = warp_sum(sum);
    if (want_max) top = warp_max(top);
    if (warps > 1) {
      if (lane == 0) {
        red[par][0][warp] = sum;
        red[par][1][warp] = top;
      }
      __syncthreads();
      sum = 0.f;
      top = 0.f;
      for (int i = 0; i < warps; ++i) {
        sum += red[par][0][i];
        top = fmaxf(top, red[par][1][i]);
      }
    }
    const float rstd = inv_rms(sum, p.K, p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[t] = rstd;
    // A token's codes: scale = max|y| / 448 (0 and zero codes for a zero row;
    // NaN, and NaN codes, when the row holds a value that is not finite).
    float inv = 0.f;
    if (want_max) {
      const float amax = top * rstd;
      inv = amax == 0.f ? 0.f : fminf(__fdiv_rn(kE4M3Max, amax), 3.4e38f) + (amax - amax);
      if (tid == 0) p.q_scale[t] = __fdiv_rn(amax, kE4M3Max);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      if (v >= V) continue;
      float f[8], g[8];
      unpack8(h[i], f);
      unpack8(w[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * g[j];
      if (p.y != nullptr) static_cast<uint4*>(p.y)[t * V + v] = pack8(f);
      if (want_max) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= inv;
        static_cast<uint2*>(p.q)[t * V + v] =
            make_uint2(e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16),
                       e4m3x2(f[4], f[5]) | (e4m3x2(f[6], f[7]) << 16));
      }
    }
  }
}

// Token-contiguous codes [K x T].  One token's codes are single bytes a row
// apart, so a cluster of blocks takes 32 tokens at a time, each block a
// segment of the columns, and keeps its h in shared memory between the two
// passes: rows are read (and h written) along K, reduced in the block and then
// across the cluster through distributed shared memory; then each thread
// takes two columns down the 32 tokens and writes 32 consecutive codes of
// each, a whole sector.  Nothing is read from global memory twice: 7 B an
// element with a residual.
constexpr int kTransTokens = 32;
constexpr int kTransCols = 2048;  // of a segment, at most: 128 KiB of shared memory

// A float of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ float cluster_float(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(ptx::mapa(ptx::smem_addr(p), rank)) : "memory");
  return v;
}

template <bool RES>
__global__ void __launch_bounds__(256) norm_fwd_t_kernel(const NormParams p, const int cluster, const int seg) {
  extern __shared__ __align__(16) uint4 s_h[];  // [32][seg / 8]
  __shared__ float s_sum[kTransTokens], s_top[kTransTokens], s_rstd[kTransTokens];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = p.K >> 3, SV = seg >> 3;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int v0 = rank * SV;
  const int mine = min(SV, V - v0);  // vectors of this block's segment (at least one: host)
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / cluster) * kTransTokens;
  const int rows = static_cast<int>(p.T - t0 < kTransTokens ? p.T - t0 : kTransTokens);  // 16 or 32
  const uint4* w = static_cast<const uint4*>(p.w) + v0;
  for (int r = warp; r < rows; r += 8) {
    const int64_t at = (t0 + r) * V + v0;
    const uint4* x = static_cast<const uint4*>(p.x) + at;
    const uint4* res = static_cast<const uint4*>(p.res) + at;
    uint4* ho = static_cast<uint4*>(p.h) + at;
    float sum = 0.f, top = 0.f;
#pragma unroll 4
    for (int v = lane; v < mine; v += 32) {
      uint4 h = x[v];
      if (RES) {
        h = add_bf16x8(h, res[v]);
        ho[v] = h;
      }
      s_h[r * SV + v] = h;
      float f[8], g[8];
      unpack8(h, f);
      unpack8(w[v], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sum = __fmaf_rn(f[j], f[j], sum);
        top = fmaxf(top, fabsf(f[j] * g[j]));
      }
    }
    sum = warp_sum(sum);
    top = warp_max(top);
    if (lane == 0) {
      s_sum[r] = sum;
      s_top[r] = top;
    }
  }
  ptx::cluster_sync();  // every block's shares are there
  if (tid < rows) {     // each block adds them in the same order
    float sum = 0.f, top = 0.f;
    for (int c = 0; c < cluster; ++c) {
      sum += cluster_float(&s_sum[tid], c);
      top = fmaxf(top, cluster_float(&s_top[tid], c));
    }
    const float rstd = inv_rms(sum, p.K, p.eps);
    s_rstd[tid] = rstd;
    if (rank == 0) {
      if (p.rstd != nullptr) p.rstd[t0 + tid] = rstd;
      if (p.amax != nullptr) {
        const float amax = top * rstd;
        const uint32_t bits = amax == amax ? __float_as_uint(amax) : 0x7FC00000u;  // a NaN wins
        const uint32_t most = __reduce_max_sync(rows == 32 ? 0xFFFFFFFFu : 0xFFFFu, bits);
        if (tid == 0) atomicMax(reinterpret_cast<unsigned int*>(p.amax), most);
      }
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // done with the others' shares
  const uint32_t* src = reinterpret_cast<const uint32_t*>(s_h);
  const uint32_t* w2 = reinterpret_cast<const uint32_t*>(w);
  uint8_t* out = static_cast<uint8_t*>(p.qt) + static_cast<int64_t>(v0) * 8 * p.T + t0;
  for (int c = tid; c < mine * 4; c += 256) {
    const float w0 = dev::bf16_to_f32(w2[c] & 0xFFFFu), w1 = __uint_as_float(w2[c] & 0xFFFF0000u);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half * 16 >= rows) break;
      uint32_t o0[4], o1[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = half * 16 + 4 * q + j;
          const uint32_t u = src[t * (seg >> 1) + c];
          const float r = s_rstd[t];
          a[j] = dev::bf16_to_f32(u & 0xFFFFu) * r * w0 * p.inv_scale;
          b[j] = __uint_as_float(u & 0xFFFF0000u) * r * w1 * p.inv_scale;
        }
        o0[q] = e4m3x2(a[0], a[1]) | (e4m3x2(a[2], a[3]) << 16);
        o1[q] = e4m3x2(b[0], b[1]) | (e4m3x2(b[2], b[3]) << 16);
      }
      uint8_t* to = out + static_cast<int64_t>(2 * c) * p.T + half * 16;
      *reinterpret_cast<uint4*>(to) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
      *reinterpret_cast<uint4*>(to + p.T) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // nobody reads this block's shares any more
}

// ---------------------------------------------------------------- gradient

// As the forward's rows; each thread keeps its columns' share of dw over the
// block's rows in registers and writes it to the block's row of `partial`.
// The next row is loaded before the present one is reduced (PRE), so that the
// barrier does not leave memory idle.
template <int NV, bool DH, bool PRE, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(const NormParams p) {
  __shared__ float red[2][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int V = p.K >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 w[NV];
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * blockDim.x;
    w[i] = v < V ? static_cast<const uint4*>(p.w)[v] : zero;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  }
  uint4 dy[NV], h[NV], dh[NV], dy2[NV], h2[NV], dh2[NV];
  float rs = 0.f, rs2 = 0.f;
  auto load = [&](int64_t t, uint4 (&a)[NV], uint4 (&b)[NV], uint4 (&c)[NV], float& r) {
    r = p.rstd[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      a[i] = v < V ? static_cast<const uint4*>(p.dy)[t * V + v] : zero;
      b[i] = v < V ? static_cast<const uint4*>(p.x)[t * V + v] : zero;
      if (DH) c[i] = v < V ? static_cast<const uint4*>(p.dh)[t * V + v] : zero;
    }
  };
  int par = 0;
  if (blockIdx.x < p.T) load(blockIdx.x, dy, h, dh, rs);
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    const bool more = t + gridDim.x < p.T;
    if (PRE && more) load(t + gridDim.x, dy2, h2, dh2, rs2);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8], g[8];
      unpack8(dy[i], a);
      unpack8(h[i], b);
      unpack8(w[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = b[j] * rs;
        dot = __fmaf_rn(a[j] * g[j], n, dot);
        acc[i][j] = __fmaf_rn(a[j], n, acc[i][j]);
      }
    }
    dot = warp_sum(dot);
    if (warps > 1) {
      if (lane == 0) red[par][warp] = dot;
      __syncthreads();
      dot = 0.f;
      for (int i = 0; i < warps; ++i) dot += red[par][i];
    }
    const float mean = __fdiv_rn(dot, static_cast<float>(p.K));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      if (v >= V) continue;
      float a[8], b[8], g[8], d[8];
      unpack8(dy[i], a);
      unpack8(h[i], b);
      unpack8(w[i], g);
      if (DH) unpack8(dh[i], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = rs * __fmaf_rn(-b[j] * rs, mean, a[j] * g[j]);
        a[j] = DH ? x + d[j] : x;
      }
      static_cast<uint4*>(p.y)[t * V + v] = pack8(a);
    }
    if (PRE) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        dy[i] = dy2[i];
        h[i] = h2[i];
        if (DH) dh[i] = dh2[i];
      }
      rs = rs2;
    } else if (more) {
      load(t + gridDim.x, dy, h, dh, rs);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * blockDim.x;
    if (v >= V) continue;
    float4* o = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * p.K + 8 * v);
    o[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    o[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
}

// dw = the sum of the blocks' shares, always in the same order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* partial, float* dw, int K, int rows) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  float sum = 0.f;
  if (k < K)
    for (int r = part; r < rows; r += 8) sum += partial[static_cast<int64_t>(r) * K + k];
  s[part][lane] = sum;
  __syncthreads();
  if (part == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum += s[i][lane];
    dw[k] = sum;
  }
}

int round32(int n) { return (n + 31) / 32 * 32; }

template <int NV>
void run_fwd(const NormParams& p, int grid, int threads, cudaStream_t s) {
  if (p.res != nullptr) norm_fwd_kernel<NV, true><<<grid, threads, 0, s>>>(p);
  else norm_fwd_kernel<NV, false><<<grid, threads, 0, s>>>(p);
}

template <bool RES>
cudaError_t run_fwd_t(const NormParams& p, cudaStream_t s) {
  const int V = p.K / 8;
  int cluster = 1;  // segments of at most 1024 columns (64 KiB: three blocks an SM) up to K = 8192
  while (cluster < 8 && V > 128 * cluster) cluster *= 2;
  const int seg = (V + cluster - 1) / cluster * 8;
  const int smem = kTransTokens * seg * 2;
  auto* k = norm_fwd_t_kernel<RES>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTransTokens * kTransCols * 2);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T + kTransTokens - 1) / kTransTokens * cluster), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p, cluster, seg);
}

template <int NV, bool PRE, int MAXT, int MINB>
void run_bwd(const NormParams& p, int grid, int threads, cudaStream_t s) {
  if (p.dh != nullptr) norm_bwd_kernel<NV, true, PRE, MAXT, MINB><<<grid, threads, 0, s>>>(p);
  else norm_bwd_kernel<NV, false, PRE, MAXT, MINB><<<grid, threads, 0, s>>>(p);
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p0, int num_sms, cudaStream_t s) {
  NormParams p = p0;
  const int V = p.K / 8;
  cudaError_t e;
  if (p.qt == nullptr || p.y != nullptr || p.q != nullptr) {
    // Few rows: as many threads a row as it has vectors, up to 512, for the
    // shortest time to one row.  Else two vectors a thread (four past
    // K = 8192), so that a block's reduction is spread over more loads.
    int nv = p.T < num_sms ? 1 : (V >= 128 ? 2 : 1);
    while ((V + nv - 1) / nv > 512) nv *= 2;
    const int threads = round32((V + nv - 1) / nv);
    const int per_sm = static_cast<int>(least(32, 2048 / threads));
    const int grid = static_cast<int>(least(p.T, static_cast<int64_t>(num_sms) * per_sm));
    if (nv == 1) run_fwd<1>(p, grid, threads, s);
    else if (nv == 2) run_fwd<2>(p, grid, threads, s);
    else run_fwd<4>(p, grid, threads, s);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (p.res != nullptr) p.x = p.h;  // for the codes below
    p.res = nullptr;
    p.rstd = nullptr;
  }
  if (p.qt != nullptr) {
    if (p.amax != nullptr && (e = cudaMemsetAsync(p.amax, 0, sizeof(float), s)) != cudaSuccess) return e;
    if ((e = p.res != nullptr ? run_fwd_t<true>(p, s) : run_fwd_t<false>(p, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int64_t norm_bwd_blocks(int64_t T, int K, int num_sms) {
  return least(T, static_cast<int64_t>(num_sms) * (K >= 2048 ? 2 : 8));
}

cudaError_t launch_norm_bwd(const NormParams& p, int num_sms, cudaStream_t s) {
  const int V = p.K / 8;
  const int nv = V <= 256 ? 1 : (V <= 1024 ? 2 : 4);
  const int threads = round32((V + nv - 1) / nv);
  const int grid = static_cast<int>(norm_bwd_blocks(p.T, p.K, num_sms));
  if (grid > 0) {
    if (nv == 1) run_bwd<1, true, 256, 4>(p, grid, threads, s);
    else if (nv == 2 && threads <= 320) run_bwd<2, true, 320, 2>(p, grid, threads, s);
    else if (nv == 2) run_bwd<2, true, 512, 1>(p, grid, threads, s);
    else run_bwd<4, false, 512, 1>(p, grid, threads, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  norm_dw_kernel<<<(p.K + 31) / 32, 256, 0, s>>>(p.partial, p.dw, p.K, grid);
  return cudaGetLastError();
}

}  // namespace forge
