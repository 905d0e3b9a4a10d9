// Root-mean-square norm over the K columns of each token, with the residual's
// addition in front of it, its output in bf16 or E4M3, and its gradient.
//
//   h = bf16(x + residual)      (h = x without one; the stream the next
//                                layers and the gradient read)
//   r = 1 / sqrt(mean_k h^2 + eps)      (0 where that is 1 / 0)
//   y = h r w
//   dx = r (g - n mean_k(g n)) + dh,  g = dy w,  n = h r;   dw = sum_t dy n
//
// Everything between loads and stores is float32; h, y and dx are rounded to
// bf16 (nearest even) and codes to E4M3 (nearest even, saturating) once.
//
// The floor of each is its traffic: x, residual, h, y 2 B an element each,
// codes 1 B.  So a row is read once and held in registers (or, for the token-contiguous
// codes, shared memory) between its reduction and its output.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "launch.h"
#include "optim.cuh"
#include "ptx.cuh"

namespace forge {

namespace {

constexpr float kE4M3Max = 448.f;

// Elements are handled in pairs (dev::f2): at these rates a dozen scalar
// operations per element would take as long as its bytes.
using dev::f2;
using dev::pair;
using dev::unpair;

__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return dev::mul(a, b); }
__device__ __forceinline__ f2 both(float a) { return pair(a, a); }

// Eight bf16 as four pairs.
__device__ __forceinline__ void unpack8(uint4 v, f2 (&f)[4]) {
  const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) f[j] = pair(dev::bf16_to_f32(a[j]), __uint_as_float(a[j] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(f2 p) {
  float a, b;
  unpair(p, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const f2 (&f)[4]) {
  return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}

// Two floats to E4M3 codes (the first in the low byte): nearest even,
// saturating at the largest finite value, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x2(f2 p) {
  float a, b;
  unpair(p, a, b);
  return e4m3x2(a, b);
}

// Sums of bf16 pairs, rounded once to bf16.  (Rounding through float32 gives
// the same: a float32 holds the sum of two 8-bit significands exactly unless
// one is below half a bf16 ulp of the other, and then both give the larger.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}
__device__ __forceinline__ uint4 add_bf16x8(uint4 a, uint4 b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

// The larger of two magnitudes; a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest of `top` and the pairs' magnitudes.
__device__ __forceinline__ float max_abs(float top, const f2 (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    unpair(f[j], a, b);
    top = max_nan(top, max_nan(fabsf(a), fabsf(b)));
  }
  return top;
}
__device__ __forceinline__ float sum2(f2 p) {
  float a, b;
  unpair(p, a, b);
  return a + b;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// An infinite maximum is no scale.
__device__ __forceinline__ float nan_unless_finite(float a) { return a + (a - a); }

// 1 / sqrt(sum / K + eps), or 0 where that root is 0 (eps = 0, a row whose
// squares are): such a row's y and codes are zeros and its gradient is dh, where
// 0 / 0 would make them NaN.
__device__ __forceinline__ float inv_rms(float sum, int K, float eps) {
  const float square = __fdiv_rn(sum, static_cast<float>(K)) + eps;
  return square == 0.f ? 0.f : __frsqrt_rn(square);
}

// ---------------------------------------------------------------- forward

// A block takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; thread i holds
// vectors i, i + blockDim.x, .. (NV of them, eight columns each) of the row;
// the weight comes from L1.  What keeps memory busy is rows in flight, so many
// rows run on few threads each (one warp up to K = 2048: no barrier) and the
// blocks of an SM are at different points of theirs; few rows run on many
// threads each, for the shortest time to one.  Sum and maximum are reduced
// together: one barrier a row, the partials in alternating halves of `red`.
// The row is kept as the products h w, so that the output is one factor away.
template <int NV, bool RES, bool MANY>
__global__ void __launch_bounds__(MANY ? 256 : 512, MANY ? (NV >= 8 ? 2 : NV >= 6 ? 3 : 4) : 1) norm_fwd_kernel(const NormParams p) {
  __shared__ float red[2][2][16];  // [row parity][sum, max][warp]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int V = p.K >> 3;
  const bool want_max = p.q != nullptr;
  const uint4* w = static_cast<const uint4*>(p.w);
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int par = 0;
  for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, par ^= 1) {
    const uint4* x = static_cast<const uint4*>(p.x) + t * V;
    uint4 h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      h[i] = v < V ? x[v] : zero;
    }
    if (RES) {
      const uint4* res = static_cast<const uint4*>(p.res) + t * V;
      uint4* ho = static_cast<uint4*>(p.h) + t * V;
      uint4 r[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        r[i] = v < V ? res[v] : zero;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        h[i] = add_bf16x8(h[i], r[i]);
        if (v < V) ho[v] = h[i];
      }
    }
    f2 sums = both(0.f);
    float top = 0.f;
    f2 hw[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      f2 f[4], g[4];
      unpack8(h[i], f);
      unpack8(v < V ? w[v] : zero, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sums = fma2(f[j], f[j], sums);
        hw[i][j] = mul2(f[j], g[j]);
      }
      if (want_max) top = max_abs(top, hw[i]);
    }
    float sum = warp_sum(sum2(sums));
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
        top = max_nan(top, red[par][1][i]);
      }
    }
    const float rstd = inv_rms(sum, p.K, p.eps);
    if (tid == 0 && p.rstd != nullptr) p.rstd[t] = rstd;
    // A token's codes: scale = max|y| / 448 (0 and zero codes for a zero row;
    // NaN, and NaN codes, when the row or the weight holds a value that is not
    // finite).
    // Near the smallest floats the scale is a denormal of few bits and its
    // reciprocal past the largest float: there the codes are of the stored scale,
    // with it and the row brought up by the same power of two.
    float by = rstd, by2 = 0.f;  // codes: (h w) by by2
    if (want_max) {
      const float amax = nan_unless_finite(top * rstd), scale = __fdiv_rn(amax, kE4M3Max);
      if (tid == 0) p.q_scale[t] = scale;
      const bool tiny = scale < 0x1p-120f;
      const float inv = __fdiv_rn(tiny ? 1.f : kE4M3Max, tiny ? scale * 0x1p100f : amax);
      by = tiny ? 0x1p100f : rstd;
      by2 = tiny ? (scale > 0.f ? inv * rstd : 0.f) : inv;
    }
    const bool to_y = p.y != nullptr;
    if (!to_y && !want_max) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      if (v >= V) continue;
      if (to_y) {
        f2 y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = mul2(hw[i][j], both(rstd));
        static_cast<uint4*>(p.y)[t * V + v] = pack8(y);
      }
      if (want_max) {
#pragma unroll
        for (int j = 0; j < 4; ++j) hw[i][j] = mul2(mul2(hw[i][j], both(by)), both(by2));
        static_cast<uint2*>(p.q)[t * V + v] = make_uint2(e4m3x2(hw[i][0]) | (e4m3x2(hw[i][1]) << 16),
                                                         e4m3x2(hw[i][2]) | (e4m3x2(hw[i][3]) << 16));
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
constexpr int kTransSmem = 131072;  // bytes of a block, at most

// 32 aligned bytes.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Store a pair of floats to the same shared variable of the cluster's block
// `rank`, counted on that block's mbarrier when it has landed.
__device__ __forceinline__ void cluster_store2(const void* dst, uint64_t* bar, uint32_t rank, float a, float b) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2, %3}, [%1];"
      ::"r"(ptx::mapa(ptx::smem_addr(dst), rank)), "r"(ptx::mapa(ptx::smem_addr(bar), rank)), "f"(a), "f"(b)
      : "memory");
}

// Until the mbarrier's first phase completes (true) or the limit passes.
__device__ __forceinline__ bool shares_landed(uint64_t* bar, uint64_t limit_ns) {
  if (ptx::mbar_try_wait_cluster(bar, 0u)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (!ptx::mbar_try_wait_cluster(bar, 0u))
    if (ptx::global_timer_ns() - t0 > limit_ns) return false;
  return true;
}

// The blocks of a cluster hand their rows' shares to each other with counted
// stores: a cluster barrier would have to wait for the h just written to
// reach L2 as well.  Two barriers of the cluster stand around them, neither of
// which waits for memory: that every block's mbarrier exists (entered before
// the loads, left after them), and that every block has sent its shares
// (entered then, left at the end).  A block whose shares did not land within
// the limit writes nothing more and leaves only after the second barrier and
// another bounded wait for them, so that none comes to a block that is gone.
template <bool RES, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? 5 : WARPS == 8 ? 3 : 1) norm_fwd_t_kernel(const NormParams p, const int cluster, const int seg) {
  extern __shared__ __align__(16) uint4 s_h[];  // [rows][seg / 8]
  __shared__ __align__(8) float2 s_part[8][kTransTokens];  // [block of the cluster][row]: sum, max
  __shared__ float s_rstd[kTransTokens];
  __shared__ __align__(8) uint64_t s_bar;
  constexpr int kRows = WARPS == 16 ? 2 : 4;  // rows of a warp loaded together
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int V = p.K >> 3, SV = seg >> 3;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int v0 = rank * SV;
  const int mine = min(SV, V - v0);  // vectors of this block's segment (at least one: host)
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / cluster) * kTransTokens;
  const int rows = static_cast<int>(p.T - t0 < kTransTokens ? p.T - t0 : kTransTokens);  // 16 or 32
  if (tid == 0) {
    ptx::mbar_init(&s_bar, 1);
    ptx::fence_mbar_init();
    ptx::mbar_arrive_expect_tx(&s_bar, static_cast<uint32_t>(cluster * rows * 8));
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // this block's barrier is there
  const uint4* w = static_cast<const uint4*>(p.w) + v0;
  const bool want_max = p.amax != nullptr;
  // A warp's rows, four at a time: warp, warp + WARPS, ..  Of 16 tokens,
  // those past the last repeat an earlier row and are not kept.
  bool met = false;
  for (int first = warp; first < rows; first += kRows * WARPS) {
    const int64_t at = (t0 + first) * V + v0;
    const uint4* x = static_cast<const uint4*>(p.x) + at;
    const uint4* res = static_cast<const uint4*>(p.res) + at;
    uint4* ho = static_cast<uint4*>(p.h) + at;
    f2 sums[kRows];
    float top[kRows];
    int step[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      sums[i] = both(0.f);
      top[i] = 0.f;
      step[i] = first + i * WARPS < rows ? i * WARPS * V : 0;
    }
    for (int v = lane; v < mine; v += 32) {
      uint4 h[kRows], q[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) h[i] = x[v + step[i]];
      if (RES) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) q[i] = res[v + step[i]];
      }
      f2 g[4];
      unpack8(want_max ? w[v] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = first + i * WARPS;
        if (RES) h[i] = add_bf16x8(h[i], q[i]);
        if (r < rows) {
          if (RES) ho[v + step[i]] = h[i];
          s_h[r * SV + v] = h[i];
        }
        f2 f[4];
        unpack8(h[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sums[i] = fma2(f[j], f[j], sums[i]);
          f[j] = mul2(f[j], g[j]);
        }
        if (want_max) top[i] = max_abs(top[i], f);
      }
    }
    if (!met) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // every block's barrier is there
    met = true;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int r = first + i * WARPS;
      const float sum = warp_sum(sum2(sums[i])), most = want_max ? warp_max(top[i]) : 0.f;
      if (r < rows && lane < cluster && !p.skip_sends) cluster_store2(&s_part[rank][r], &s_bar, lane, sum, most);
    }
  }
  if (!met) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // this thread's shares are sent
  const bool landed = tid >= rows || shares_landed(&s_bar, p.wait_limit_ns);
  if (__syncthreads_or(!landed)) {  // (else s_h is whole as well)
    if (!landed) atomicCAS(p.status, 0u, static_cast<uint32_t>(kStatusTimeout));
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    shares_landed(&s_bar, p.wait_limit_ns);
    return;
  }
  if (tid < rows) {
    float sum = 0.f, most = 0.f;
    for (int c = 0; c < cluster; ++c) {  // the same order in each block
      sum += s_part[c][tid].x;
      most = max_nan(most, s_part[c][tid].y);
    }
    const float rstd = inv_rms(sum, p.K, p.eps);
    const float factor = rstd * p.inv_scale;  // past the largest float every code but zero's saturates
    s_rstd[tid] = factor > 3.4e38f ? 3.4e38f : factor;
    if (rank == 0) {
      if (p.rstd != nullptr) p.rstd[t0 + tid] = rstd;
      if (want_max) {
        const float amax = nan_unless_finite(most * rstd);
        const uint32_t bits = amax == amax ? __float_as_uint(amax) : 0x7FC00000u;  // a NaN wins
        const uint32_t all = __reduce_max_sync(rows == 32 ? 0xFFFFFFFFu : 0xFFFFu, bits);
        if (tid == 0) atomicMax(reinterpret_cast<unsigned int*>(p.amax), all);
      }
    }
  }
  __syncthreads();
  const uint32_t* src = reinterpret_cast<const uint32_t*>(s_h);
  const uint32_t* w2 = reinterpret_cast<const uint32_t*>(w);
  uint8_t* out = static_cast<uint8_t*>(p.qt) + static_cast<int64_t>(v0) * 8 * p.T + t0;
  const bool whole = p.T % 32 == 0 && (reinterpret_cast<uintptr_t>(p.qt) & 31u) == 0;
  for (int c = tid; c < mine * 4; c += 32 * WARPS) {
    const f2 wp = pair(dev::bf16_to_f32(w2[c]), __uint_as_float(w2[c] & 0xFFFF0000u));
    uint8_t* to = out + static_cast<int64_t>(2 * c) * p.T;
    uint32_t o0[8], o1[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float a[4], b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 4 * q + j;  // past `rows`: not stored
        const uint32_t u = src[t * (seg >> 1) + c];
        const f2 y = mul2(mul2(pair(dev::bf16_to_f32(u), __uint_as_float(u & 0xFFFF0000u)), both(s_rstd[t])), wp);
        unpair(y, a[j], b[j]);
      }
      o0[q] = e4m3x2(a[0], a[1]) | (e4m3x2(a[2], a[3]) << 16);
      o1[q] = e4m3x2(b[0], b[1]) | (e4m3x2(b[2], b[3]) << 16);
    }
    if (whole) {  // rows of whole 32-byte sectors: one a store
      store32(to, o0);
      store32(to + p.T, o1);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (16 * i < rows) {
          *reinterpret_cast<uint4*>(to + 16 * i) = make_uint4(o0[4 * i], o0[4 * i + 1], o0[4 * i + 2], o0[4 * i + 3]);
          *reinterpret_cast<uint4*>(to + p.T + 16 * i) = make_uint4(o1[4 * i], o1[4 * i + 1], o1[4 * i + 2], o1[4 * i + 3]);
        }
    }
  }
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// ---------------------------------------------------------------- gradient

// A block takes rows blockIdx.x, blockIdx.x + gridDim.x, ...; each thread keeps
// its columns' share of dw over them in registers and writes it to the block's
// row of `partial` at the end.  The next row is loaded before the present one is
// reduced (PRE), so that the barrier does not leave memory idle; the weight
// waits in shared memory.
template <int NV, bool DH, bool PRE, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint4 s_w[];  // [NV * blockDim.x]
  __shared__ float red[2][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5;
  const int V = p.K >> 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  f2 acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * blockDim.x;
    s_w[v] = v < V ? static_cast<const uint4*>(p.w)[v] : zero;  // its own reader
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
  }
  struct Row {
    uint4 dy[NV], h[NV], dh[NV];
    float rs;
  };
  auto load = [&](int64_t t, Row& r) {
    r.rs = p.rstd[t];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      r.dy[i] = v < V ? static_cast<const uint4*>(p.dy)[t * V + v] : zero;
      r.h[i] = v < V ? static_cast<const uint4*>(p.x)[t * V + v] : zero;
      if (DH) r.dh[i] = v < V ? static_cast<const uint4*>(p.dh)[t * V + v] : zero;
    }
  };
  int par = 0;
  auto row = [&](int64_t t, const Row& r) {
    f2 dots = both(0.f), g[NV][4];
    const f2 r2 = both(r.rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f2 a[4], b[4], w[4];
      unpack8(r.dy[i], a);
      unpack8(r.h[i], b);
      unpack8(s_w[tid + i * blockDim.x], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 n = mul2(b[j], r2);
        g[i][j] = mul2(a[j], w[j]);
        dots = fma2(g[i][j], n, dots);
        acc[i][j] = fma2(a[j], n, acc[i][j]);
      }
    }
    float dot = warp_sum(sum2(dots));
    if (warps > 1) {
      if (lane == 0) red[par][warp] = dot;
      __syncthreads();
      dot = 0.f;
      for (int i = 0; i < warps; ++i) dot += red[par][i];
      par ^= 1;
    }
    // dx = rs (g - n mean) + dh, n mean = h (rs mean): rs itself may be past the
    // root of the largest float (a tiny row without eps), n is near one
    const f2 back = both(-r.rs * __fdiv_rn(dot, static_cast<float>(p.K)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * blockDim.x;
      if (v >= V) continue;
      f2 b[4], d[4];
      unpack8(r.h[i], b);
      if (DH) unpack8(r.dh[i], d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f2 inner = fma2(b[j], back, g[i][j]);
        b[j] = DH ? fma2(inner, r2, d[j]) : mul2(inner, r2);
      }
      static_cast<uint4*>(p.y)[t * V + v] = pack8(b);
    }
  };
  const int64_t G = gridDim.x;
  int64_t t = blockIdx.x;
  Row r0;
  if (PRE) {  // two rows' registers take turns
    Row r1;
    if (t < p.T) load(t, r0);
    while (t < p.T) {
      if (t + G < p.T) load(t + G, r1);
      row(t, r0);
      t += G;
      if (t >= p.T) break;
      if (t + G < p.T) load(t + G, r0);
      row(t, r1);
      t += G;
    }
  } else {
    for (; t < p.T; t += G) {
      load(t, r0);
      row(t, r0);
    }
  }
  ptx::grid_dep_launch();  // the sum over blocks may start as they end
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = tid + i * blockDim.x;
    if (v >= V) continue;
    float4* o = reinterpret_cast<float4*>(p.partial + static_cast<int64_t>(blockIdx.x) * p.K + 8 * v);
    float a[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) unpair(acc[i][j], a[2 * j], a[2 * j + 1]);
    o[0] = make_float4(a[0], a[1], a[2], a[3]);
    o[1] = make_float4(a[4], a[5], a[6], a[7]);
  }
}

// dw = the sum of the blocks' shares, always in the same order: sixteen groups
// of rows in parallel, eight loads ahead in each.
constexpr int kDwParts = 16;
__global__ void __launch_bounds__(32 * kDwParts) norm_dw_kernel(const float* partial, float* dw, int K, int rows) {
  __shared__ float s[kDwParts][33];
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int k = blockIdx.x * 32 + lane;
  float sum = 0.f;
  ptx::grid_dep_wait();
  if (k < K) {
#pragma unroll 8
    for (int r = part; r < rows; r += kDwParts) sum += partial[static_cast<int64_t>(r) * K + k];
  }
  s[part][lane] = sum;
  __syncthreads();
  if (part == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < kDwParts; ++i) sum += s[i][lane];
    dw[k] = sum;
  }
}

int round32(int n) { return (n + 31) / 32 * 32; }

template <int NV, bool MANY>
void run_fwd(const NormParams& p, int grid, int threads, cudaStream_t s) {
  if (p.res != nullptr) norm_fwd_kernel<NV, true, MANY><<<grid, threads, 0, s>>>(p);
  else norm_fwd_kernel<NV, false, MANY><<<grid, threads, 0, s>>>(p);
}

template <bool RES>
cudaError_t run_fwd_t(const NormParams& p, cudaStream_t s) {
  const int V = p.K / 8;
  int cluster = 1;  // segments of at most 512 columns (32 KiB) up to K = 4096
  while (cluster < 8 && V > 64 * cluster) cluster *= 2;
  const int seg = (V + cluster - 1) / cluster * 8;
  const int smem = kTransTokens * seg * 2;
  // Five blocks of four warps an SM overlap their passes better than three of
  // eight (16384 x 4096: 90 and 102 us) as long as their memory lets five in;
  // where it lets one in (K > 8192), sixteen warps (2048 x 16384: 74 and 84).
  const int warps = smem <= 40960 ? 4 : (smem <= 65536 ? 8 : 16);
  auto* k = warps == 4 ? norm_fwd_t_kernel<RES, 4> : (warps == 8 ? norm_fwd_t_kernel<RES, 8> : norm_fwd_t_kernel<RES, 16>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kTransSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T + kTransTokens - 1) / kTransTokens * cluster), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps), 1, 1);
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
  if (p.dh != nullptr) norm_bwd_kernel<NV, true, PRE, MAXT, MINB><<<grid, threads, NV * threads * 16, s>>>(p);
  else norm_bwd_kernel<NV, false, PRE, MAXT, MINB><<<grid, threads, NV * threads * 16, s>>>(p);
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

}  // namespace

cudaError_t launch_norm_fwd(const NormParams& p0, int num_sms, cudaStream_t s) {
  NormParams p = p0;
  const int V = p.K / 8;
  cudaError_t e;
  if (p.qt != nullptr) {  // first: y may lie over x or the residual
    if (p.amax != nullptr && (e = cudaMemsetAsync(p.amax, 0, sizeof(float), s)) != cudaSuccess) return e;
    if ((e = p.res != nullptr ? run_fwd_t<true>(p, s) : run_fwd_t<false>(p, s)) != cudaSuccess) return e;
    if (p.y == nullptr && p.q == nullptr) return cudaSuccess;
    if (p.res != nullptr) p.x = p.h;  // the sum is there
    p.res = nullptr;
    p.rstd = nullptr;
  }
  if (p.T < 2 * num_sms) {  // few rows
    int nv = 1;
    while ((V + nv - 1) / nv > 512) nv *= 2;
    const int threads = round32((V + nv - 1) / nv);
    const int grid = static_cast<int>(p.T);
    if (nv == 1) run_fwd<1, false>(p, grid, threads, s);
    else if (nv == 2) run_fwd<2, false>(p, grid, threads, s);
    else run_fwd<4, false>(p, grid, threads, s);
  } else {
    int warps = 1;
    while (V > 32 * 8 * warps) warps *= 2;
    const int nv = (V + 32 * warps - 1) / (32 * warps);
    const int grid = static_cast<int>(least(p.T, static_cast<int64_t>(num_sms) * (32 / warps)));
    if (nv <= 1) run_fwd<1, true>(p, grid, 32 * warps, s);
    else if (nv <= 2) run_fwd<2, true>(p, grid, 32 * warps, s);
    else if (nv <= 4) run_fwd<4, true>(p, grid, 32 * warps, s);
    else if (nv <= 5) run_fwd<5, true>(p, grid, 32 * warps, s);
    else if (nv <= 6) run_fwd<6, true>(p, grid, 32 * warps, s);
    else run_fwd<8, true>(p, grid, 32 * warps, s);
  }
  return cudaGetLastError();
}

int64_t norm_bwd_blocks(int64_t T, int K, int num_sms) {
  // two blocks an SM, or eight of narrow rows (few threads each); every block adds a row to `partial`
  return least(T, static_cast<int64_t>(num_sms) * (K >= 2048 ? 2 : 8));
}

cudaError_t launch_norm_bwd(const NormParams& p, int num_sms, cudaStream_t s) {
  const int V = p.K / 8;
  // Loading a row ahead pays where its registers leave room for it: with one
  // vector a thread (16384 x 2048: 60 us, 69 without) and with two in one block
  // an SM (4096 x 8192: 50 and 69); two blocks of two vectors a thread are
  // faster without (12289 x 5120: 88 and 106, spilled), and four do not fit.
  const int nv = V <= 256 ? 1 : (V <= 1024 ? 2 : 4);
  const int threads = round32((V + nv - 1) / nv);
  const int grid = static_cast<int>(norm_bwd_blocks(p.T, p.K, num_sms));
  if (grid > 0) {
    if (nv == 1) run_bwd<1, true, 256, 4>(p, grid, threads, s);
    else if (nv == 2 && threads <= 320) run_bwd<2, false, 320, 2>(p, grid, threads, s);
    else if (nv == 2) run_bwd<2, true, 512, 1>(p, grid, threads, s);
    else run_bwd<4, false, 512, 1>(p, grid, threads, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.K + 31) / 32), 1, 1);
  cfg.blockDim = dim3(32 * kDwParts, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = grid > 0 ? 1 : 0;
  const float* partial = p.partial;
  return cudaLaunchKernelEx(&cfg, norm_dw_kernel, partial, p.dw, static_cast<int>(p.K), grid);
}

}  // namespace forge
