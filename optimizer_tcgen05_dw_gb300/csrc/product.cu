// The product of block-scaled 8-bit codes: X [T x K] with a scale for each 128
// elements of a row, W [N x K] with one for each 128 x 128,
//   Y[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k].
//
// The inner sum is one ring stage on the tensor cores (128 E4M3 of the
// reduction: 128-byte rows), float32 in tensor memory; the outer one is kept in
// registers: after every stage the accumulator changes hands, and eight
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

__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return dev::mul(a, b); }

// A warp holds 32 token rows x W columns of the sum in registers.  The row
// is a lane of tensor memory and the columns lie in one block of W's scales, so
// a lane has one factor a stage.
template <int W, int AROWS = kTileM>
struct ProductOp {
  using Params = ProductParams;
  struct Maps { CUtensorMap y; };
  static constexpr int kW = W, kARows = AROWS, kBufs = 256 / W, kEpiWarps = 8;
  static constexpr int kStg = AROWS < kTileM ? (W == 128 ? 10 : W == 64 ? 16 : 24) : (W == 128 ? 5 : W == 64 ? 8 : 10);
  static constexpr int NC = W;                              // columns a warp holds
  static constexpr bool kStaged = W == 128 && AROWS == kTileM;
  static constexpr int kStage = kStaged ? 32 * NC * 2 : 0;  // bytes a warp stages its rows in
  static constexpr int kEpiBytes = kEpiWarps * kStage;
  static constexpr bool kFp8 = true, kBMajorMN = false, kBlockwise = true;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }

  // acc += v times the block's factor f = xs ws (codes::factor where that is not
  // an ordinary number in some lane).
  static __device__ __forceinline__ void fold(f2* acc, const uint32_t (&v)[32], float f, float xs, float ws, bool ordinary) {
    if (ordinary) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        acc[j] = fma2(dev::pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), dev::pair(f, f), acc[j]);
    } else {
      const codes::Factor c = codes::factor(xs, ws);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        acc[j] = fma2(mul2(dev::pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), dev::pair(c.p, c.p)),
                      dev::pair(c.f, c.f), acc[j]);
    }
  }

  static __device__ __forceinline__ void epilogue(const Maps& maps, const Params& p, pairs::Shared* ss, uint8_t* epi,
                                                  int warp, int lane, uint32_t rank) {
    const int quarter = warp & 3, sub = (warp - pairs::kFirstEpiWarp) >> 2;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    const uint32_t tbase = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(sub * NC);
    uint8_t* stage = epi + (warp - pairs::kFirstEpiWarp) * kStage;
    uint32_t buf = 0, ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = tm * kPairM + static_cast<int>(rank) * kTileM + quarter * 32, col = tn * 2 * W + sub * NC;
      const bool live = row0 < p.T && col < p.N;  // else the warp hands the accumulators on unread
      // rows past the end repeat the last one's scales; nothing of theirs is stored
      const float* sx = p.x_scale + static_cast<int64_t>(min(row0 + lane, p.T - 1)) * p.num_kb;
      const float* sw = p.w_scale + static_cast<int64_t>(min(col, p.N - 1) / codes::kBlock) * p.num_kb;
      f2 acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = dev::pair(0.f, 0.f);
      float ax = sx[0], aw = sw[0];
      for (int kb = 0; kb < p.num_kb; ++kb) {
        const float xs = ax, ws = aw;
        const float f = xs * ws;
        if (kb + 1 < p.num_kb) {
          ax = sx[kb + 1];
          aw = sw[kb + 1];
        }
        const bool ordinary = __all_sync(0xFFFFFFFFu, f > 0x1p-100f && f < 0x1p100f);
        if (!pairs::warp_wait(&ss->tmem_full[buf], ph, p, ss, lane)) return;
        ptx::tc_fence_after();
        if (live) {
          const uint32_t taddr = tbase + buf * pairs::Layout<ProductOp>::kBufCols;
          uint32_t v[2][32];
          pairs::tmem_issue32(taddr, v[0]);
          pairs::tmem_wait32(v[0]);
#pragma unroll
          for (int h = 0; h < NC / 32; ++h) {
            if (h + 1 < NC / 32) pairs::tmem_issue32(taddr + (h + 1) * 32, v[(h + 1) & 1]);
            if (h + 1 == NC / 32) {  // all of it is in registers
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + buf * 8u);
            }
            fold(acc + h * 16, v[h & 1], f, xs, ws, ordinary);
            if (h + 1 < NC / 32) pairs::tmem_wait32(v[(h + 1) & 1]);
          }
        } else {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + buf * 8u);
        }
        if (++buf == kBufs) {
          buf = 0;
          ph ^= 1u;
        }
      }
      if constexpr (kStaged) {
        // 32 rows x 64 columns of bf16 a copy: 128-byte rows
        if (lane == 0) ptx::bulk_wait_group_read0();  // the last tile's copies have read them
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) dev::unpair(acc[i * 4 + j], v[2 * j], v[2 * j + 1]);
          *reinterpret_cast<uint4*>(stage + (i >> 3) * 4096 + sw128(lane, i & 7)) = pack_rne_bf16x8(v);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && live) {
          ptx::tma_store_2d(&maps.y, stage, col, row0);
          if (col + 64 < p.N) ptx::tma_store_2d(&maps.y, stage + 4096, col + 64, row0);
          ptx::bulk_commit_group();
        }
      } else if (row0 + lane < p.T) {
        uint16_t* out = static_cast<uint16_t*>(p.Y) + static_cast<int64_t>(row0 + lane) * p.N + col;
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
    if (kStaged && lane == 0) ptx::bulk_wait_group0();
  }
};

}  // namespace

cudaError_t launch_product(int width, const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& y, const ProductParams& p,
                           int pairs_n, cudaStream_t s) {
  if (p.T <= kShortRows) {
    if (width == 128) return pairs::launch<ProductOp<128, kShortRows>>(x, w, {y}, p, pairs_n, s);
    if (width == 64) return pairs::launch<ProductOp<64, kShortRows>>(x, w, {y}, p, pairs_n, s);
    return pairs::launch<ProductOp<32, kShortRows>>(x, w, {y}, p, pairs_n, s);
  }
  if (width == 128) return pairs::launch<ProductOp<128>>(x, w, {y}, p, pairs_n, s);
  if (width == 64) return pairs::launch<ProductOp<64>>(x, w, {y}, p, pairs_n, s);
  return pairs::launch<ProductOp<32>>(x, w, {y}, p, pairs_n, s);
}

}  // namespace forge
