// The gated feed-forward products.
//
// Forward, both projections of a token, the gate's activation and the product
// in one kernel:
//   G = X Wg^T,  U = X Wu^T,  Y = act(G) U          (W = [Wg; Wu], 2F x K)
// The pair's two CTAs hold the two halves of the matrix instruction's B
// operand, so one loads gate rows and the other up rows of the same features:
// every CTA's accumulator then has G in its first W columns and U in the next,
// and the activation meets its factor in one thread.  What the gradient needs
// (G and U) leaves in bf16 or as E4M3 codes; the 128 features of a tile are one
// block of the codes.
//
// Gradient, through the down projection's weight Wd [N x F], the product dY Wd
// with the activation's gradient as its epilogue (dA never reaches memory):
//   dA = dY Wd,  dU = dA act(G),  dG = dA U act'(G),  and Y = act(G) U again,
// which the down projection's own step reads: the forward need not keep it.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "gate.cuh"
#include "pair_gemm.cuh"

namespace forge {

namespace {

constexpr int kQuarterBarrier = 2;  // + 0 .. 3: the four warps of a tensor-memory quarter

// ---------------------------------------------------------------- forward

template <int W, bool CODES, int AROWS = kTileM>
struct GatedOp {
  static_assert(!CODES || W == codes::kBlock, "a block of the codes is a tile's features");
  using Params = GatedParams;
  struct Maps { int unused; };
  static constexpr int kW = W, kARows = AROWS, kBufs = W == 128 ? 2 : 4, kSplit = 1;
  static constexpr int kStg = AROWS < kTileM ? (W == 128 ? 10 : W == 64 ? 16 : 24) : (W == 128 ? 6 : W == 64 ? 9 : 11);
  static constexpr int kEpiBytes = CODES ? 2 * 4 * kTileM * 4 : 0;
  static constexpr bool kMoreRegs = false, kFp8 = false, kBMajorMN = false, kBlockwise = false;

  // rank 0: gate rows, rank 1: up rows of the same features (rows of another
  // half past a ragged end give columns that are not stored)
  static __device__ __forceinline__ int b_row(int tn, int rank, const Params& p) { return rank * p.F + tn * W; }

  static __device__ __forceinline__ void init_barriers(pairs::Shared*) {}
  static __device__ __forceinline__ void helper(const Params&, pairs::Shared*, uint8_t*, int, int, uint32_t) {}

  static __device__ __forceinline__ void epilogue(const Maps&, const Params& p, pairs::Shared* ss, uint8_t* epi, int warp,
                                                  int lane, uint32_t rank) {
    constexpr int NC = W / 4;  // features a warp takes
    const int quarter = warp & 3, sub = (warp - pairs::kFirstEpiWarp) >> 2, r = quarter * 32 + lane;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    float* red = reinterpret_cast<float*>(epi);  // [gate, up][warp of the quarter][row]
    uint32_t acc = 0, ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * kPairM + static_cast<int>(rank) * kTileM + r;
      const int f0 = tn * W + sub * NC;
      const bool ok = pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane);
      if (CODES) {  // the quarter's warps meet below: they stop together
        if (ptx::bar_red_or(kQuarterBarrier + quarter, 128, !ok)) return;
        __syncwarp();
      } else if (!ok) {
        return;
      }
      ptx::tc_fence_after();
      const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
                             static_cast<uint32_t>(sub * NC);
      float g[NC], u[NC];
      pairs::tmem_load<NC>(taddr, g);
      pairs::tmem_load<NC>(taddr + W, u);
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
      if (++acc == kBufs) {
        acc = 0;
        ph ^= 1u;
      }
      float gs = 0.f, us = 0.f;
      if (CODES) {
        float ga = 0.f, ua = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {  // (columns past F are of other rows)
          if (f0 + j < p.F) {
            ga = codes::max_nan(ga, fabsf(g[j]));
            ua = codes::max_nan(ua, fabsf(u[j]));
          }
        }
        red[sub * kTileM + r] = ga;
        red[(4 + sub) * kTileM + r] = ua;
        ptx::bar_sync(kQuarterBarrier + quarter, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ga = codes::max_nan(ga, red[i * kTileM + r]);
          ua = codes::max_nan(ua, red[(4 + i) * kTileM + r]);
        }
        gs = codes::block_scale(ga);
        us = codes::block_scale(ua);
        // (the next tile's first barrier keeps its sums from overtaking these reads)
      }
      if (row < p.T) {
        if (p.gu != nullptr) {
          uint16_t* out = static_cast<uint16_t*>(p.gu) + row * 2 * p.F + f0;
#pragma unroll
          for (int j = 0; j < NC / 8; ++j) {
            if (f0 + 8 * j >= p.F) break;
            *reinterpret_cast<uint4*>(out + 8 * j) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(g[8 * j]));
            *reinterpret_cast<uint4*>(out + p.F + 8 * j) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(u[8 * j]));
          }
        }
        if (CODES) {
          const float gi = codes::inverse_scale(gs), ui = codes::inverse_scale(us);
          uint8_t* out = static_cast<uint8_t*>(p.codes) + row * 2 * p.F + f0;
#pragma unroll
          for (int j = 0; j < NC / 8; ++j) {
            if (f0 + 8 * j >= p.F) break;
            const float* a = g + 8 * j;
            const float* b = u + 8 * j;
            *reinterpret_cast<uint2*>(out + 8 * j) = make_uint2(codes::encode4(a[0] * gi, a[1] * gi, a[2] * gi, a[3] * gi),
                                                                codes::encode4(a[4] * gi, a[5] * gi, a[6] * gi, a[7] * gi));
            *reinterpret_cast<uint2*>(out + p.F + 8 * j) =
                make_uint2(codes::encode4(b[0] * ui, b[1] * ui, b[2] * ui, b[3] * ui),
                           codes::encode4(b[4] * ui, b[5] * ui, b[6] * ui, b[7] * ui));
          }
          if (sub < 2) p.scale[(row * 2 + sub) * p.tiles_n + tn] = sub == 0 ? gs : us;
        }
        uint16_t* y = static_cast<uint16_t*>(p.Y) + row * p.F + f0;
#pragma unroll
        for (int j = 0; j < NC / 8; ++j) {
          if (f0 + 8 * j >= p.F) break;
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = gated(p.act, g[8 * j + i], u[8 * j + i]);
          *reinterpret_cast<uint4*>(y + 8 * j) = pack_rne_bf16x8(v);
        }
      }
    }
  }
};

// ---------------------------------------------------------------- gradient

template <int W, bool CODES>
struct GatedGradOp {
  using Params = GatedParams;
  struct Maps { int unused; };
  static constexpr int kW = W, kARows = kTileM, kStg = W == 128 ? 6 : 9, kBufs = W == 128 ? 2 : 4, kSplit = 1, kEpiBytes = 0;
  static constexpr bool kMoreRegs = false, kFp8 = false, kBMajorMN = true, kBlockwise = false;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }

  static __device__ __forceinline__ void init_barriers(pairs::Shared*) {}
  static __device__ __forceinline__ void helper(const Params&, pairs::Shared*, uint8_t*, int, int, uint32_t) {}

  static __device__ __forceinline__ void epilogue(const Maps&, const Params& p, pairs::Shared* ss, uint8_t*, int warp,
                                                  int lane, uint32_t rank) {
    constexpr int NC = W / 2;  // features a warp takes
    const int quarter = warp & 3, sub = (warp - pairs::kFirstEpiWarp) >> 2, r = quarter * 32 + lane;
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    const int NB = (p.F + codes::kBlock - 1) / codes::kBlock;
    uint32_t acc = 0, ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int64_t row = static_cast<int64_t>(tm) * kPairM + static_cast<int>(rank) * kTileM + r;
      const int f0 = tn * 2 * W + sub * NC;
      if (!pairs::warp_wait(&ss->tmem_full[acc], ph, p, ss, lane)) return;
      ptx::tc_fence_after();
      const uint32_t taddr = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * (kTmemCols / kBufs) +
                             static_cast<uint32_t>(sub * NC);
      const bool live = row < p.T && f0 < p.F;
      float gs = 0.f, us = 0.f;
      if (CODES && live) {
        gs = p.scale[row * 2 * NB + f0 / codes::kBlock];
        us = p.scale[(row * 2 + 1) * NB + f0 / codes::kBlock];
      }
#pragma unroll 1
      for (int c = 0; c < NC; c += 8) {
        float da[8];
        pairs::tmem_load<8>(taddr + c, da);
        if (row >= p.T || f0 + c >= p.F) continue;
        const int64_t at = row * 2 * p.F + f0 + c;
        float g[8], u[8], y[8];
        if (CODES) {
          const uint2 gc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.codes) + at);
          const uint2 uc = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.codes) + at + p.F);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = codes::decode2((j < 2 ? gc.x : gc.y) >> (16 * (j & 1)));
            const float2 b = codes::decode2((j < 2 ? uc.x : uc.y) >> (16 * (j & 1)));
            g[2 * j] = a.x * gs;
            g[2 * j + 1] = a.y * gs;
            u[2 * j] = b.x * us;
            u[2 * j + 1] = b.y * us;
          }
        } else {
          load_bf16x8(p.gu, at, g);
          load_bf16x8(p.gu, at + p.F, u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) gated_gradient(p.act, da[j], g[j], u[j], g[j], u[j], y[j]);
        // (dGU may be gu itself: this thread alone reads and writes these eight of each)
        store_bf16x8_rne(p.dGU, at, g);
        store_bf16x8_rne(p.dGU, at + p.F, u);
        if (p.Y != nullptr) store_bf16x8_rne(p.Y, row * p.F + f0 + c, y);
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + acc * 8u);
      if (++acc == kBufs) {
        acc = 0;
        ph ^= 1u;
      }
    }
  }
};

}  // namespace

cudaError_t launch_gated(int width, const CUtensorMap& x, const CUtensorMap& w, const GatedParams& p, int pairs_n,
                         cudaStream_t s) {
  if (p.codes != nullptr) return pairs::launch<GatedOp<128, true>>(x, w, {}, p, pairs_n, s);
  if (p.T <= kShortRows) {
    if (width == 128) return pairs::launch<GatedOp<128, false, kShortRows>>(x, w, {}, p, pairs_n, s);
    if (width == 64) return pairs::launch<GatedOp<64, false, kShortRows>>(x, w, {}, p, pairs_n, s);
    return pairs::launch<GatedOp<32, false, kShortRows>>(x, w, {}, p, pairs_n, s);
  }
  if (width == 128) return pairs::launch<GatedOp<128, false>>(x, w, {}, p, pairs_n, s);
  if (width == 64) return pairs::launch<GatedOp<64, false>>(x, w, {}, p, pairs_n, s);
  return pairs::launch<GatedOp<32, false>>(x, w, {}, p, pairs_n, s);
}

cudaError_t launch_gated_grad(int width, const CUtensorMap& dy, const CUtensorMap& w, const GatedParams& p, int pairs_n,
                              cudaStream_t s) {
  const bool kept8 = p.codes != nullptr;
  if (width == 128)
    return kept8 ? pairs::launch<GatedGradOp<128, true>>(dy, w, {}, p, pairs_n, s)
                 : pairs::launch<GatedGradOp<128, false>>(dy, w, {}, p, pairs_n, s);
  return kept8 ? pairs::launch<GatedGradOp<64, true>>(dy, w, {}, p, pairs_n, s)
               : pairs::launch<GatedGradOp<64, false>>(dy, w, {}, p, pairs_n, s);
}

}  // namespace forge
