// The product of block-scaled 8-bit codes: X [T x K] with a scale for each 128
// elements of a row, W [N x K] with one for each 128 x 128,
//   Y[t, n] = sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k].
//
// The inner sum is one ring stage on the tensor cores (128 E4M3 of the
// reduction: 128-byte rows), float32 in tensor memory; the outer one is kept in
// registers: after every stage the accumulator changes hands, and the epilogue
// warps fold it in with the block's factor while the next ones are filled.
#include <cuda_bf16.h>

#include "codes.cuh"
#include "pair_gemm.cuh"

namespace forge {

namespace {

// An epilogue warp holds 32 token rows (the lanes of its quarter of tensor
// memory) x W / 2 columns of the sum in registers.  What it does besides folding is
// kept small, as it is this loop that the tensor cores wait for: the factors, a
// product of two scales each, come through shared memory from the two helper
// warps, kGroup stages at a time and up to kSlots of these ahead (16384 x 14336 x
// 4096: 790 us; 832 where those copied the scales and the epilogue multiplied them).
// At W = 128 a stage is multiplied in two halves (kSplit), each with accumulators
// of its own, so that four are under way: an accumulator's way through commit,
// epilogue and back is longer than the instructions of two.
template <int W, int AROWS = kTileM>
struct ProductOp {
  using Params = ProductParams;
  struct Maps { CUtensorMap y; };
  static constexpr int kW = W, kARows = AROWS, kSplit = W == 128 ? 2 : 1, kBufs = W == 32 ? 8 : 4, kEpiWarps = pairs::kEpiWarps;
  static constexpr int kStg = AROWS < kTileM ? (W == 128 ? 9 : W == 64 ? 14 : 22) : (W == 128 ? 5 : W == 64 ? 8 : 10);
  static constexpr int NC = W / 2, LD = NC < 32 ? NC : 32;     // columns a warp holds, and takes at a time
  static constexpr int kBlk = W == 128 ? 2 : 1;                // blocks of W's scales they lie in
  static constexpr bool kStaged = W == 128 && AROWS == kTileM;
  static constexpr int kStage = kStaged ? 32 * LD * 2 : 0;     // bytes a warp stages its rows in
  static constexpr int kGroup = 4, kSlots = 4;                 // stages in a slot of factors, slots
  static constexpr int kStageFloats = kBlk * kTileM;           // a stage's factors: [W's block][row]
  static constexpr int kWide = kBlk * 4;                       // a slot's flags: [W's block][quarter of the rows]
  static constexpr int kSlotFloats = kGroup * kStageFloats + kWide;
  static constexpr int kEpiBytes = kEpiWarps * kStage + ((kSlots * kSlotFloats * 4 + 127) & ~127);
  static constexpr bool kMoreRegs = true, kFp8 = true, kBMajorMN = false;
  static constexpr int kFold = 1;

  static __device__ __forceinline__ int b_row(int tn, int rank, const Params&) { return (2 * tn + rank) * W; }

  static __device__ __forceinline__ void init_barriers(pairs::Shared* ss) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&ss->epi[i], 64);                  // a slot's factors are there: both helper warps' lanes
      ptx::mbar_init(&ss->epi[kSlots + i], kEpiWarps);  // and have been read
    }
  }
  static __device__ __forceinline__ float* factors(uint8_t* epi) { return reinterpret_cast<float*>(epi + kEpiWarps * kStage); }

  // Helper warp 2 + i forms the factors of rows 64 i .. 64 i + 63, two a lane, and
  // says of each quarter of the tile's rows whether some factor in a slot is not
  // an ordinary number.  Rows and columns past the end repeat the last one's;
  // nothing of theirs is stored.
  static __device__ __forceinline__ void helper(const Params& p, pairs::Shared* ss, uint8_t* epi, int warp, int lane,
                                                uint32_t rank) {
    const int row = (warp - 2) * 64 + lane;
    int slot = 0;
    uint32_t ph = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = tm * kPairM + static_cast<int>(rank) * kTileM + row;
      const float* sx0 = p.x_scale + static_cast<int64_t>(min(row0, p.T - 1)) * p.num_kb;
      const float* sx1 = p.x_scale + static_cast<int64_t>(min(row0 + 32, p.T - 1)) * p.num_kb;
      const float* sw[kBlk];
#pragma unroll
      for (int b = 0; b < kBlk; ++b)
        sw[b] = p.w_scale + static_cast<int64_t>(min(tn * 2 * W + b * W, p.N - 1) / codes::kBlock) * p.num_kb;
      for (int kb = 0; kb < p.num_kb; kb += kGroup) {
        if (!pairs::warp_wait(&ss->epi[kSlots + slot], ph ^ 1u, p, ss, lane)) return;
        float* to = factors(epi) + slot * kSlotFloats;
        uint32_t odd = 0;  // bit 2 b + i: some factor of this lane's row i with block b is
#pragma unroll 1
        for (int j = 0; j < kGroup; j += 2) {  // (two stages at a time: the warp has 32 registers)
          float x[2][2], ws[2][kBlk];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int at = min(kb + j + h, p.num_kb - 1);
            x[h][0] = sx0[at];
            x[h][1] = sx1[at];
#pragma unroll
            for (int b = 0; b < kBlk; ++b) ws[h][b] = sw[b][at];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < kBlk; ++b)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float f = x[h][i] * ws[h][b];
                // (blocks of zeros, as padding rows have, are ordinary: their factor is 0 itself)
                if (!((f > 0x1p-100f && f < 0x1p100f) || x[h][i] == 0.f || ws[h][b] == 0.f)) odd |= 1u << (2 * b + i);
                to[(j + h) * kStageFloats + b * kTileM + 32 * i + row] = f;
              }
        }
        odd = __reduce_or_sync(0xFFFFFFFFu, odd);
        if (lane < 2 * kBlk)
          to[kGroup * kStageFloats + (lane >> 1) * 4 + (warp - 2) * 2 + (lane & 1)] = (odd >> lane) & 1u ? 1.f : 0.f;
        ptx::mbar_arrive(&ss->epi[slot]);
        if (++slot == kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
  }

  // acc += v f; where some lane's factor is not an ordinary number, in two parts.
  // (One column an instruction: in pairs every value was moved once more, to
  // where a pair of registers begins, and a block took 173 instructions of the
  // multiply pipe in place of 128.)
  static __device__ __forceinline__ void fold(float* acc, const float (&v)[LD], float f) {
#pragma unroll
    for (int j = 0; j < LD; ++j) acc[j] = fmaf(v[j], f, acc[j]);
  }
  static __device__ __forceinline__ void fold_wide(float* acc, const float (&v)[LD], const Params& p, int row, int col, int kb) {
    const codes::Factor c = codes::factor(p.x_scale[static_cast<int64_t>(min(row, p.T - 1)) * p.num_kb + kb],
                                          p.w_scale[static_cast<int64_t>(min(col, p.N - 1) / codes::kBlock) * p.num_kb + kb]);
#pragma unroll
    for (int j = 0; j < LD; ++j) acc[j] = fmaf(v[j] * c.p, c.f, acc[j]);
  }

  static __device__ __forceinline__ void epilogue(const Maps& maps, const Params& p, pairs::Shared* ss, uint8_t* epi,
                                                  int warp, int lane, uint32_t rank) {
    constexpr int kBufCols = pairs::Layout<ProductOp>::kBufCols;
    const int quarter = warp & 3, w = warp - pairs::kFirstEpiWarp, sub = w >> 2;
    // With kSplit, warps 2 h and 2 h + 1 of a quarter take half h: 64 columns in each block of W's scales.
    const int half = kSplit == 2 ? sub >> 1 : 0, blk = kSplit == 2 ? sub & 1 : 0;
    const int first = kSplit == 2 ? blk * W + half * NC : sub * NC;  // its first column of the tile
    const uint32_t empty0 = ptx::mapa(ptx::smem_addr(&ss->tmem_empty[0]), 0);
    const uint32_t tbase = ss->tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                           static_cast<uint32_t>(kSplit == 2 ? blk * NC : sub * NC);
    uint8_t* stage = epi + w * kStage;
    const float* own = factors(epi) + blk * kTileM + quarter * 32 + lane;
    const float* flag = factors(epi) + kGroup * kStageFloats + blk * 4 + quarter;
    uint32_t buf = half, ph = 0, slot_ph = 0;
    int slot = 0;
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = tm * kPairM + static_cast<int>(rank) * kTileM + quarter * 32, col0 = tn * 2 * W + first;
      const bool live = row0 < p.T && col0 < p.N;  // else nothing of the warp's is stored
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[i] = 0.f;
#pragma unroll 1
      for (int kb0 = 0; kb0 < p.num_kb; kb0 += kGroup) {
        if (!pairs::warp_wait(&ss->epi[slot], slot_ph, p, ss, lane)) goto drain;
        float f[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j) f[j] = own[slot * kSlotFloats + j * kStageFloats];
        const bool wide = flag[slot * kSlotFloats] != 0.f;
        __syncwarp();  // the slot has been read
        if (lane == 0) ptx::mbar_arrive(&ss->epi[kSlots + slot]);
        if (++slot == kSlots) {
          slot = 0;
          slot_ph ^= 1u;
        }
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          if (kb0 + j >= p.num_kb) break;
          if (!pairs::warp_wait(&ss->tmem_full[buf], ph, p, ss, lane)) goto drain;
          ptx::tc_fence_after();
          const uint32_t taddr = tbase + buf * kBufCols;
#pragma unroll
          for (int c = 0; c < NC / LD; ++c) {
            float v[LD];
            pairs::tmem_load<LD>(taddr + c * LD, v);
            if (c == NC / LD - 1) {  // all of it is in registers
              ptx::tc_fence_before();
              __syncwarp();  // (every lane's reads, not only lane 0's, come before the arrival)
              if (lane == 0) ptx::mbar_arrive_cluster_tmem(empty0 + buf * 8u);
            }
            if (!wide) fold(acc + c * LD, v, f[j]);
            else fold_wide(acc + c * LD, v, p, row0 + lane, col0, kb0 + j);
          }
          buf += kSplit;
          if (buf >= kBufs) {
            buf -= kBufs;
            ph ^= 1u;
          }
        }
      }
      if constexpr (kStaged) {
        // 32 rows x 32 columns of bf16 a copy: 64-byte rows, one half of the columns after the other
#pragma unroll
        for (int h = 0; h < NC / LD; ++h) {
          if (lane == 0) ptx::bulk_wait_group_read0();  // the last copy has read them
          __syncwarp();
#pragma unroll
          for (int i = 0; i < LD / 8; ++i)
            *reinterpret_cast<uint4*>(stage + sw64(lane, i)) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(acc[h * LD + i * 8]));
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && live && col0 + h * LD < p.N) {
            ptx::tma_store_2d(&maps.y, stage, col0 + h * LD, row0);
            ptx::bulk_commit_group();
          }
        }
      } else if (row0 + lane < p.T) {
        uint16_t* out = static_cast<uint16_t*>(p.Y) + static_cast<int64_t>(row0 + lane) * p.N + col0;
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) {
          if (col0 + i * 8 >= p.N) break;
          *reinterpret_cast<uint4*>(out + i * 8) = pack_rne_bf16x8(reinterpret_cast<const float(&)[8]>(acc[i * 8]));
        }
      }
    }
  drain:  // (after a wait that ran out too: the copies under way read this block's shared memory)
    if (kStaged && lane == 0) ptx::bulk_wait_group0();
    __syncwarp();
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
