// The skeleton shared by the products of this directory that have TOKENS as the
// 256 rows of the matrix instruction: the gated feed-forward products (gated.cu)
// and the product of block-scaled 8-bit codes (product.cu).
//
// One persistent kernel on CTA pairs, as the linear step's (tc_kernel.cuh: the
// same ring of TMA stages, two accumulators in tensor memory, roles per warp):
//   warp 0      TMA loads: of each stage this CTA's 128 token rows of A and its
//               W columns of B, 128 bytes of the reduction each (64 bf16 or 128
//               E4M3 elements);
//   warp 1      tcgen05.mma of the pair, 256 x 2 W x (16 or 32);
//   warps 2..17 the epilogue, four warps to each 32-lane quarter of tensor memory.
// An operator (Op) says what its B rows are and what its epilogue does:
//   Op::Params                    with PairParams as its base
//   kW, kFp8, kBMajorMN           columns of B per CTA; E4M3 operands; B stored
//                                 with its columns contiguous
//   kBlockwise                    the accumulator is handed over after every
//                                 stage (and starts from zero), not after a tile
//   kStg, kEpiBytes, kMaps        ring stages, epilogue's shared memory
//   b_row(tile_n, rank, p)        first B row (or column) of this CTA's half
//   epilogue(...)                 see pair_kernel
// W narrower than 128 gives more and smaller units when there are few.
#pragma once

#include "launch.h"
#include "tc_kernel.cuh"

namespace forge {
namespace pairs {

constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kA = kTileM * 128;  // bytes of A per stage and CTA

template <class Op>
struct Layout {
  static constexpr int kBK = Op::kFp8 ? 128 : 64;
  static constexpr int kB = Op::kW * 128;  // bytes of B per stage and CTA
  static constexpr int kSmem = Op::kStg * (kA + kB) + Op::kEpiBytes + 512 + 1024;
  static_assert(kSmem <= 232448, "dynamic shared memory limit");
  static_assert(Op::kStg <= 8, "barrier arrays");
};

template <class Op>
__device__ void producer(const CUtensorMap* mA, const CUtensorMap* mB, const typename Op::Params& p, uint8_t* smA,
                         uint8_t* smB, SharedState* ss, uint32_t rank) {
  constexpr int STG = Op::kStg, BK = Layout<Op>::kBK, kB = Layout<Op>::kB, W = Op::kW;
  uint32_t it = 0, issued_mask = 0, last_parity = 0;
  const uint32_t full0 = ptx::mapa(ptx::smem_addr(&ss->full[0]), 0);
  if (!p.skip_loads) {
    for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
      int tm, tn;
      tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
      const int m0 = tm * kPairM + static_cast<int>(rank) * kTileM;
      const int b0 = Op::b_row(tn, static_cast<int>(rank), p);
      for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
        const int s = static_cast<int>(it % STG);
        const uint32_t ph = (it / STG) & 1u;
        if (!bounded_wait(&ss->empty[s], ph ^ 1u, p, ss)) goto drain;
        const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&ss->full[s], 2u * (kA + kB));
        uint8_t* b = smB + s * kB;
        ptx::tma_load_2d_pair(mA, bar, smA + s * kA, kb * BK, m0);
        if (!Op::kBMajorMN) {
          ptx::tma_load_2d_pair(mB, bar, b, kb * BK, b0);
        } else if (p.op3d) {  // [W / 64 column blocks][64 rows][64 columns] in one copy
          ptx::tma_load_3d_pair(mB, bar, b, 0, kb * BK, b0 / 64);
        } else {
#pragma unroll
          for (int i = 0; i < W / 64; ++i) ptx::tma_load_2d_pair(mB, bar, b + i * 64 * BK * 2, b0 + 64 * i, kb * BK);
        }
        issued_mask |= 1u << s;
        last_parity = (last_parity & ~(1u << s)) | (ph << s);
      }
    }
  }
drain:
  if (rank == 0)  // every issued copy lands before the pair can exit
    for (int s = 0; s < STG; ++s)
      if (issued_mask & (1u << s)) bounded_wait(&ss->full[s], (last_parity >> s) & 1u, p, ss, false);
}

// Leader CTA only.
template <class Op>
__device__ void mma(const typename Op::Params& p, uint8_t* smA, uint8_t* smB, SharedState* ss) {
  constexpr int STG = Op::kStg, BK = Layout<Op>::kBK, kB = Layout<Op>::kB;
  constexpr uint32_t idesc = Op::kFp8 ? ptx::idesc_e4m3_f32(kPairM, 2 * Op::kW)
                                      : ptx::idesc_bf16_f32(kPairM, 2 * Op::kW, false, Op::kBMajorMN);
  uint32_t it = 0, use = 0;  // use: accumulators handed over
  for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
    for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
      const uint32_t acc = use & 1u;
      if (Op::kBlockwise || kb == 0) {
        if (!bounded_wait(&ss->tmem_empty[acc], ((use >> 1) & 1u) ^ 1u, p, ss)) goto done;
        ptx::tc_fence_after();
      }
      const int s = static_cast<int>(it % STG);
      if (!bounded_wait(&ss->full[s], (it / STG) & 1u, p, ss)) goto done;
      ptx::tc_fence_after();
      const uint32_t d_tmem = ss->tmem_base + acc * kTileN;
      const uint32_t a0 = ptx::smem_addr(smA + s * kA), b0 = ptx::smem_addr(smB + s * kB);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {  // 32 bytes of the reduction an instruction
        const uint64_t adesc = ptx::smem_desc_sw128(a0 + kk * 32, 16, 1024);
        const uint64_t bdesc = Op::kBMajorMN ? ptx::smem_desc_sw128(b0 + kk * 2048, BK * 128, 1024)
                                             : ptx::smem_desc_sw128(b0 + kk * 32, 16, 1024);
        const uint32_t add = Op::kBlockwise ? (kk != 0 ? 1u : 0u) : ((kb | kk) != 0 ? 1u : 0u);
        if (Op::kFp8) ptx::mma_e4m3_pair(d_tmem, adesc, bdesc, idesc, add);
        else ptx::mma_bf16_pair(d_tmem, adesc, bdesc, idesc, add);
      }
      ptx::mma_commit_pair_multicast(&ss->empty[s], 0x3);
      if (Op::kBlockwise || kb == p.num_kb - 1) {
        ptx::mma_commit_pair_multicast(&ss->tmem_full[acc], 0x3);
        ++use;
      }
    }
  }
done:
  ptx::mma_commit_pair_multicast(&ss->mma_done, 0x1);
  bounded_wait(&ss->mma_done, 0u, p, ss, false);
}

// A warp's wait: lane 0 waits, the warp gets its verdict together, and what
// lane 0 saw is ordered before the other lanes' reads.
template <class P>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const P& p, SharedState* ss, int lane) {
  const bool ok = __all_sync(0xFFFFFFFFu, lane != 0 || bounded_wait(bar, parity, p, ss));
  __syncwarp();
  return ok;
}

// NC consecutive fp32 columns of this warp's 32 tensor-memory lanes.
template <int NC>
__device__ __forceinline__ void tmem_load(uint32_t taddr, float (&v)[NC]) {
  static_assert(NC == 8 || NC == 16 || NC == 32, "8, 16 or 32 columns");
  if constexpr (NC == 8) ptx::tmem_ld_32x32b_x8(taddr, v);
  else if constexpr (NC == 16) ptx::tmem_ld_32x32b_x16(taddr, v);
  else ptx::tmem_ld_32x32b_x32(taddr, v);
}

template <class Op>
__global__ void __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ typename Op::Maps maps, const typename Op::Params p) {
  using L = Layout<Op>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + Op::kStg * kA;
  uint8_t* epi = smB + Op::kStg * L::kB;
  SharedState* ss = reinterpret_cast<SharedState*>(epi + Op::kEpiBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < Op::kStg; ++s) {
      ptx::mbar_init(&ss->full[s], 1);
      ptx::mbar_init(&ss->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&ss->tmem_full[a], 1);
      ptx::mbar_init(&ss->tmem_empty[a], 2 * kEpiWarps);
    }
    ptx::mbar_init(&ss->mma_done, 1);
    ss->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&mapA);
    ptx::prefetch_tensormap(&mapB);
  }
  if (warp == 1) {
    __syncwarp();
    ptx::tmem_alloc_pair(&ss->tmem_base, kTmemCols);
    ptx::tmem_relinquish_pair();
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // both CTAs' barriers exist before either signals the other's
  ptx::tc_fence_after();
  if (warp == 0) {
    if (lane == 0) producer<Op>(&mapA, &mapB, p, smA, smB, ss, rank);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) mma<Op>(p, smA, smB, ss);
  } else {
    Op::epilogue(maps, p, ss, epi, warp, lane, rank);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer's shared and tensor memory stay valid until the pair is done
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(ss->tmem_base, kTmemCols);
  }
}

template <class Op>
inline cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const typename Op::Maps& maps,
                          const typename Op::Params& p, int pairs, cudaStream_t s) {
  auto* k = pair_kernel<Op>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<Op>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Layout<Op>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, a, b, maps, p);
}

}  // namespace pairs
}  // namespace forge
