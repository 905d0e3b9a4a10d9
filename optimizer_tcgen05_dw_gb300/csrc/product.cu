// The product of block-scaled 8-bit codes: X [T x K] with a scale for each 128
// elements of a row, W [N x K] with one for each 128 x 128,
//   Y[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k].
//
// The inner sum is one ring stage on the tensor cores (128 E4M3 of the
// reduction: 128-byte rows), float32 in tensor memory; the outer one is kept in
// registers: after every stage the accumulator changes hands, and sixteen
// epilogue warps of each CTA fold it in with the block's factor while the next
// stage fills the other one.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "pair_gemm.cuh"

namespace forge {

namespace {

using dev::f2;

__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

template <int W>
struct ProductOp {
  using Params = ProductParams;
  struct Maps { int unused; };
  static constexpr int kW = W, kStg = 6, kEpiBytes = 0;
  static constexpr bool kFp8 = true, kBMajorMN = false, kBlockwise = true;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }

  static __device__ __forceinline__ void epilogue(const Maps&, const Params& p, SharedState* ss, uint8_t*, int warp,
                                                  int lane, uint32_t rank) {
    constexpr int NC = W / 2;                // columns a warp folds
    constexpr int LD = NC < 16 ? NC : 16;    // columns a load
    const int quarter = warp & 3, sub = (warp - 2) >> 2;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    uint32_t use = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * kPairM + static_cast<int>(rank) * kTileM + quarter * 32 + lane;
      const int64_t col = static_cast<int64_t>(tn) * 2 * W + sub * NC;
      // rows and columns past the end repeat the last one's scales; nothing of theirs is stored
      const float* sx = p.x_scale + min(row, static_cast<int64_t>(p.T) - 1) * p.num_kb;
      const float* sw = p.w_scale + min(col, static_cast<int64_t>(p.N) - 1) / codes::kBlock * p.num_kb;
      f2 acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = dev::pair(0.f, 0.f);
      float ax = sx[0], aw = sw[0];
      for (int kb = 0; kb < p.num_kb; ++kb, ++use) {
        const int next = min(kb + 1, p.num_kb - 1);
        const float nx = sx[next], nw = sw[next];
        const uint32_t buf = use & 1u;
        if (!pairs::warp_wait(&ss->tmem_full[buf], (use >> 1) & 1u, p, ss, lane)) return;
        ptx::tc_fence_after();
        const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + buf * kTileN +
                               static_cast<uint32_t>(sub * NC);
        // The factor, where it has all its bits (or is 0 or NaN); else the two
        // scales one after the other in 64 bits.
        const float f = ax * aw;
        const bool plain = (f > 0x1p-100f && f < 0x1p100f) || !(ax > 0.f) || !(aw > 0.f);
#pragma unroll
        for (int h = 0; h < NC / LD; ++h) {
          float v[LD];
          pairs::tmem_load<LD>(taddr + h * LD, v);
          if (!plain) {
#pragma unroll
            for (int j = 0; j < LD; ++j)
              v[j] = static_cast<float>(static_cast<double>(v[j]) * static_cast<double>(ax) * static_cast<double>(aw));
          }
          const f2 ff = dev::pair(plain ? f : 1.f, plain ? f : 1.f);
#pragma unroll
          for (int j = 0; j < LD / 2; ++j)
            acc[h * LD / 2 + j] = fma2(dev::pair(v[2 * j], v[2 * j + 1]), ff, acc[h * LD / 2 + j]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + buf * 8u);
        ax = nx;
        aw = nw;
      }
      if (row >= p.T) continue;
      uint16_t* out = static_cast<uint16_t*>(p.Y) + row * p.N + col;
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        if (col + i * 8 >= p.N) break;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) dev::unpair(acc[i * 4 + j], v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4*>(out + i * 8) = pack_rne_bf16x8(v);
      }
    }
  }
};

}  // namespace

cudaError_t launch_product(int width, const CUtensorMap& x, const CUtensorMap& w, const ProductParams& p, int pairs_n,
                           cudaStream_t s) {
  if (width == 128) return pairs::launch<ProductOp<128>>(x, w, {}, p, pairs_n, s);
  if (width == 64) return pairs::launch<ProductOp<64>>(x, w, {}, p, pairs_n, s);
  return pairs::launch<ProductOp<32>>(x, w, {}, p, pairs_n, s);
}

}  // namespace forge
