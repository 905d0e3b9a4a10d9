// The gated product and the product of block-scaled codes for a few token rows
// (decoding).  The weights are read once for a handful of tokens, so the floor
// is that read and what matters is to spread it evenly and keep it streaming:
// a block takes the weight rows of 8 (gated: gate and up), 16 or 32 features, its
// 8 or 16 warps share the reduction, and the warp-level matrix instruction takes
// the weights from the registers they were loaded to (each is used once: staging
// it through shared memory for a larger instruction would only lengthen its way).
// The instruction's k order is free as long as both operands agree: a lane loads
// 16 contiguous bytes of its row and of its token and feeds them to two
// instructions.  The warps' sums meet in shared memory, in warp order.
//
// Tokens past the last repeat it, rows past the last feature repeat it; their
// results are not stored.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "gate.cuh"
#include "launch.h"
#include "optim.cuh"

namespace forge {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;

__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Rows 0-7 (lane >> 2) and 8-15 of the first operand against eight columns:
// c[0], c[1] are row lane >> 2, columns 2 (lane & 3) and the next, c[2], c[3] row + 8.
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes, in order, as two pairs of halves, each 2^-8 of its value: sign,
// four exponent and three mantissa bits move to their places in a half (bias 15
// for 7; numbers smaller than normal come out right too).  Of NaN's seven set
// bits this makes 0x3F80, the largest magnitude there is: `top` keeps the
// largest seen.
__device__ __forceinline__ uint32_t halves2(uint32_t high, uint32_t& top) {  // two codes, each the high byte of a half
  const uint32_t mag = (high >> 1) & 0x3F803F80u;
  top = __vmaxu2(top, mag);
  return mag | (high & 0x80008000u);
}
__device__ __forceinline__ void halves16(uint4 c, uint32_t (&h)[8], uint32_t& top) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[2 * j] = halves2(__byte_perm(w[j], 0, 0x1404), top);
    h[2 * j + 1] = halves2(__byte_perm(w[j], 0, 0x3424), top);
  }
}
// The same by the conversion instruction: the values themselves.
__device__ __forceinline__ void converted16(uint4 c, uint32_t (&h)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h[2 * j]), "=r"(h[2 * j + 1]) : "r"(w[j]));
  }
}
__device__ __forceinline__ bool has_nan(uint32_t top) { return (top & 0xFFFFu) == 0x3F80u || (top >> 16) == 0x3F80u; }

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  const __nv_bfloat16 b = __float2bfloat16_rn(v);
  return *reinterpret_cast<const uint16_t*>(&b);
}

// ---------------------------------------------------------------- gated

// Features 8 blockIdx.x .. of up to 8 tokens.  The gate's rows are rows 0-7 of
// the instruction and the up projection's rows 8-15, so a lane holds both
// projections of a feature.
__global__ void __launch_bounds__(kThreads) gated_few_kernel(const uint16_t* W, const uint16_t* X, const GatedParams p,
                                                             const int K) {
  constexpr int kTok = 8;
  __shared__ float s_sum[kWarps * kTok * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int V = K >> 3, f0 = blockIdx.x * 8;
  const int64_t f_own = min(f0 + g, p.F - 1);
  const uint4* wg = reinterpret_cast<const uint4*>(W + f_own * K);
  const uint4* wu = reinterpret_cast<const uint4*>(W + (p.F + f_own) * K);
  const uint4* x = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(min(g, p.T - 1)) * K);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll 2
  for (int v = warp * 4 + q; v - q < V; v += kWarps * 4) {  // uniform over the warp
    const bool in = v < V;
    const uint4 a = in ? ld_once(wg + v) : zero, b = in ? ld_once(wu + v) : zero, t = in ? x[v] : zero;
    mma_bf16(acc, a.x, b.x, a.y, b.y, t.x, t.y);
    mma_bf16(acc, a.z, b.z, a.w, b.w, t.z, t.w);
  }
  // [warp][token][gate's features, then the up projection's]
#pragma unroll
  for (int j = 0; j < 4; ++j) s_sum[(warp * kTok + 2 * q + (j & 1)) * 16 + (j >> 1) * 8 + g] = acc[j];
  __syncthreads();
  const int t = threadIdx.x >> 3, c = threadIdx.x & 7, f = f0 + c;
  if (t >= p.T || t >= kTok || f >= p.F) return;
  float gate = 0.f, up = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    gate += s_sum[(w * kTok + t) * 16 + c];
    up += s_sum[(w * kTok + t) * 16 + 8 + c];
  }
  static_cast<uint16_t*>(p.Y)[static_cast<int64_t>(t) * p.F + f] = bf16_bits(gated(p.act, gate, up));
  if (p.gu != nullptr) {
    uint16_t* kept = static_cast<uint16_t*>(p.gu) + static_cast<int64_t>(t) * 2 * p.F + f;
    kept[0] = bf16_bits(gate);
    kept[p.F] = bf16_bits(up);
  }
}

// ---------------------------------------------------------------- codes

// Features 16 MT blockIdx.x .. of up to 8 NT tokens; a warp takes a block of
// 128 of the reduction at a time, and its sum meets the block's two scales.  The
// codes are multiplied as halves: the warp-level instruction on E4M3 itself ran
// at a fraction of that one's rate (5 rows of 4096 x 14336: 33 us and more).
// Weights are converted by the instruction for it and tokens by integer
// operations, to share the time between the two pipes; the tokens' serve MT
// instructions, and the next block's loads, 2 MT KB a warp, are under way meanwhile
// (5 rows of 4096 x 14336: 14.7 us; MT = 1 in twice as many blocks of eight warps 18.2).
constexpr int kCodeWarps = 16, kCodeThreads = 32 * kCodeWarps;
template <int NT, int MT>
__global__ void __launch_bounds__(kCodeThreads, 1) product_few_kernel(const uint8_t* W, const uint8_t* X, const ProductParams p,
                                                                   const int K) {
  constexpr int kTok = 8 * NT, kFeat = 16 * MT;
  __shared__ float s_sum[kCodeWarps * kTok * kFeat];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * kFeat, V = K >> 4;
  const uint4* w[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      w[m][r] = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(min(f0 + 16 * m + 8 * r + g, p.N - 1)) * K) + q;
  const float* sw = p.w_scale + static_cast<int64_t>(f0 / codes::kBlock) * p.num_kb;
  const uint4* x[NT];
  const float* sx[NT][2];
  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    x[i] = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(min(8 * i + g, p.T - 1)) * K) + q;
#pragma unroll
    for (int j = 0; j < 2; ++j) sx[i][j] = p.x_scale + static_cast<int64_t>(min(8 * i + 2 * q + j, p.T - 1)) * p.num_kb;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.f;
  }
  struct Block {
    uint4 a[MT][2][2], t[NT][2];
    float ws, xs[NT][2];
  };
  Block ahead;
  uint32_t top_t[NT];  // largest magnitudes of this lane's tokens
#pragma unroll
  for (int i = 0; i < NT; ++i) top_t[i] = 0;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](Block& o, int b) {
    const bool in = b < p.num_kb;
    const int at = in ? b : 0;
    o.ws = sw[at];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = at * 8 + h * 4;
      const bool there = in && v + q < V;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 2; ++r) o.a[m][r][h] = there ? ld_once(w[m][r] + v) : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i) o.t[i][h] = there ? x[i][v] : zero;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) o.xs[i][j] = sx[i][j][at];
  };
  load(ahead, warp);
  for (int b = warp; b < p.num_kb; b += kCodeWarps) {
    const Block o = ahead;
    load(ahead, b + kCodeWarps);
    float c[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[m][i][j] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t t[NT][8];
#pragma unroll
      for (int i = 0; i < NT; ++i) halves16(o.t[i][h], t[i], top_t[i]);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        uint32_t r0[8], r1[8];
        converted16(o.a[m][0][h], r0);
        converted16(o.a[m][1][h], r1);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int k = 0; k < 8; k += 2) mma_f16(c[m][i], r0[k], r1[k], r0[k + 1], r1[k + 1], t[i][k], t[i][k + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const codes::Factor f = codes::factor(o.xs[i][j], o.ws);
        const float part = f.p * 256.f;  // the tokens were 2^-8 of their values
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          acc[m][i][j] = fmaf(c[m][i][j] * part, f.f, acc[m][i][j]);
          acc[m][i][j + 2] = fmaf(c[m][i][j + 2] * part, f.f, acc[m][i][j + 2]);
        }
      }
  }
  // A NaN code among this warp's makes its token's sums NaN: the token is with
  // the four lanes whose g is its number.
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint32_t nan_t = __ballot_sync(0xFFFFFFFFu, has_nan(top_t[i]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (((nan_t >> (4 * (2 * q + (j & 1)))) & 0xFu) != 0)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m][i][j] = __uint_as_float(0x7FC00000u);
    }
  }
  // [warp][token][feature]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s_sum[(warp * kTok + 8 * i + 2 * q + (j & 1)) * kFeat + 16 * m + g + 8 * (j >> 1)] = acc[m][i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < kTok * kFeat; o += kCodeThreads) {
    const int t = o / kFeat, f = f0 + o % kFeat;
    if (t >= p.T || f >= p.N) continue;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kCodeWarps; ++i) sum += s_sum[i * kTok * kFeat + o];
    static_cast<uint16_t*>(p.Y)[static_cast<int64_t>(t) * p.N + f] = bf16_bits(sum);
  }
}

template <int NT, int MT>
cudaError_t run_product(const void* W, const void* X, const ProductParams& p, int K, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.N + 16 * MT - 1) / (16 * MT));
  product_few_kernel<NT, MT><<<grid, kCodeThreads, 0, s>>>(static_cast<const uint8_t*>(W), static_cast<const uint8_t*>(X), p, K);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_few(const void* W, const void* X, const GatedParams& p, int K, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.F + 7) / 8);
  gated_few_kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint16_t*>(W), static_cast<const uint16_t*>(X), p, K);
  return cudaGetLastError();
}

// Blocks of 32 features, or of 16 where all of them have an SM each.
cudaError_t launch_product_few(const void* W, const void* X, const ProductParams& p, int K, int num_sms, cudaStream_t s) {
  if ((p.N + 15) / 16 <= num_sms) return p.T <= 8 ? run_product<1, 1>(W, X, p, K, s) : run_product<2, 1>(W, X, p, K, s);
  return p.T <= 8 ? run_product<1, 2>(W, X, p, K, s) : run_product<2, 2>(W, X, p, K, s);
}

}  // namespace forge
