// The gated product and the product of block-scaled codes for a few token rows
// (decoding).  The weights are read once for a handful of tokens, so the floor
// is that read and what matters is to spread it evenly and keep it streaming:
// a block takes the weight rows of 8 (gated: gate and up) or 16 features, its
// eight warps share the reduction, and the warp-level matrix instruction takes
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

// Four codes as two pairs of halves, codes 1 and 3 first, then 0 and 2, each
// 2^-8 of its value: sign, four exponent and three mantissa bits move to their
// places in a half (bias 15 for 7; numbers smaller than normal come out right
// too).  Of NaN's seven set bits this makes 0x3F80, the largest magnitude there
// is: `top` keeps the largest seen.
__device__ __forceinline__ void halves4(uint32_t w, uint32_t& odd, uint32_t& even, uint32_t& top) {
  constexpr uint32_t kMag = 0x3F803F80u, kSign = 0x80008000u;
  const uint32_t mo = (w >> 1) & kMag, me = (w << 7) & kMag;
  top = __vmaxu2(top, __vmaxu2(mo, me));
  odd = mo | (w & kSign);
  even = me | ((w << 8) & kSign);
}
__device__ __forceinline__ void halves16(uint4 c, uint32_t (&h)[8], uint32_t& top) {
  halves4(c.x, h[0], h[1], top);
  halves4(c.y, h[2], h[3], top);
  halves4(c.z, h[4], h[5], top);
  halves4(c.w, h[6], h[7], top);
}
// The same by the conversion instruction: values themselves, in order.
__device__ __forceinline__ void converted16(uint4 c, uint32_t (&h)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 x;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %1, lo;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(h[2 * j]), "=r"(h[2 * j + 1]) : "r"(w[j]));
    const uint32_t a = h[2 * j], b = h[2 * j + 1];  // codes 2, 3 and 0, 1 -> 1, 3 and 0, 2
    h[2 * j] = __byte_perm(b, a, 0x7632);
    h[2 * j + 1] = __byte_perm(b, a, 0x5410);
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

// Features 16 blockIdx.x .. of up to 8 NT tokens; a warp takes a block of 128
// of the reduction at a time, and its sum meets the block's two scales.  The
// codes are multiplied as halves: the warp-level instruction on E4M3 itself ran
// at a fraction of that one's rate (5 rows of 4096 x 14336: 33 us and more).
// Weights are converted by the instruction for it and tokens by integer
// operations, to share the time between the two pipes (all converted 22.6 us, all
// by integers 26, so 17.9); the next block's loads are under way meanwhile.
template <int NT>
__global__ void __launch_bounds__(kThreads, 2) product_few_kernel(const uint8_t* W, const uint8_t* X, const ProductParams p,
                                                               const int K) {
  constexpr int kTok = 8 * NT;
  __shared__ float s_sum[kWarps * kTok * 16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * 16, V = K >> 4;
  const uint4* w0 = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(min(f0 + g, p.N - 1)) * K) + q;
  const uint4* w1 = reinterpret_cast<const uint4*>(W + static_cast<int64_t>(min(f0 + g + 8, p.N - 1)) * K) + q;
  const float* sw = p.w_scale + static_cast<int64_t>(f0 / codes::kBlock) * p.num_kb;
  const uint4* x[NT];
  const float* sx[NT][2];
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    x[i] = reinterpret_cast<const uint4*>(X + static_cast<int64_t>(min(8 * i + g, p.T - 1)) * K) + q;
#pragma unroll
    for (int j = 0; j < 2; ++j) sx[i][j] = p.x_scale + static_cast<int64_t>(min(8 * i + 2 * q + j, p.T - 1)) * p.num_kb;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  }
  struct Block {
    uint4 a0[2], a1[2], t[NT][2];
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
      o.a0[h] = there ? ld_once(w0 + v) : zero;
      o.a1[h] = there ? ld_once(w1 + v) : zero;
#pragma unroll
      for (int i = 0; i < NT; ++i) o.t[i][h] = there ? x[i][v] : zero;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) o.xs[i][j] = sx[i][j][at];
  };
  load(ahead, warp);
  for (int b = warp; b < p.num_kb; b += kWarps) {
    const Block o = ahead;
    load(ahead, b + kWarps);
    float c[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r0[8], r1[8];
      converted16(o.a0[h], r0);
      converted16(o.a1[h], r1);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        uint32_t t[8];
        halves16(o.t[i][h], t, top_t[i]);
#pragma unroll
        for (int k = 0; k < 8; k += 2) mma_f16(c[i], r0[k], r1[k], r0[k + 1], r1[k + 1], t[k], t[k + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const codes::Factor f = codes::factor(o.xs[i][j], o.ws);
        const float part = f.p * 256.f;  // the tokens were 2^-8 of their values
        acc[i][j] = fmaf(c[i][j] * part, f.f, acc[i][j]);
        acc[i][j + 2] = fmaf(c[i][j + 2] * part, f.f, acc[i][j + 2]);
      }
  }
  // A NaN code among this warp's makes its token's sums NaN: the token is with
  // the four lanes whose g is its number.
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const uint32_t nan_t = __ballot_sync(0xFFFFFFFFu, has_nan(top_t[i]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (((nan_t >> (4 * (2 * q + (j & 1)))) & 0xFu) != 0) acc[i][j] = __uint_as_float(0x7FC00000u);
    }
  }
  // [warp][token][feature]
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s_sum[(warp * kTok + 8 * i + 2 * q + (j & 1)) * 16 + g + 8 * (j >> 1)] = acc[i][j];
  __syncthreads();
  for (int o = threadIdx.x; o < kTok * 16; o += kThreads) {
    const int t = o / 16, f = f0 + o % 16;
    if (t >= p.T || f >= p.N) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_sum[w * kTok * 16 + o];
    static_cast<uint16_t*>(p.Y)[static_cast<int64_t>(t) * p.N + f] = bf16_bits(sum);
  }
}

template <int NT>
cudaError_t run_product(const void* W, const void* X, const ProductParams& p, int K, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.N + 15) / 16);
  product_few_kernel<NT><<<grid, kThreads, 0, s>>>(static_cast<const uint8_t*>(W), static_cast<const uint8_t*>(X), p, K);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_few(const void* W, const void* X, const GatedParams& p, int K, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((p.F + 7) / 8);
  gated_few_kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint16_t*>(W), static_cast<const uint16_t*>(X), p, K);
  return cudaGetLastError();
}

cudaError_t launch_product_few(const void* W, const void* X, const ProductParams& p, int K, cudaStream_t s) {
  return p.T <= 8 ? run_product<1>(W, X, p, K, s) : run_product<2>(W, X, p, K, s);
}

}  // namespace forge
