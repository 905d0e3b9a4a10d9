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
//   warps 2, 3  what an operator has for them (Op::helper);
//   warps 4..19 the epilogue, four warps to each 32-lane quarter of tensor
//               memory (registers are dealt by warpgroups of four, and the
//               epilogue may have what the first gives up).
// An operator (Op) says what its B rows are and what its epilogue does:
//   Op::Params                    with PairParams as its base
//   kW, kFp8, kBMajorMN           columns of B per CTA; E4M3 operands; B stored
//                                 with its columns contiguous
//   kFold                         stages after which the accumulator is handed over
//                                 (and starts from zero), 0: after a tile
//   kEpiBytes, kMoreRegs          the epilogue's shared memory; whether it takes
//                                 registers from the first warpgroup
//   kStg, kBufs                   ring stages, accumulators
//   kSplit                        2: a stage is multiplied in two halves of W
//                                 columns, an accumulator each (columns [0, W / 2)
//                                 are of this CTA's half of B's rows, or the other's
//                                 for the next), so that more of them are under way
//   kARows                        128, or fewer token rows that a stage holds when
//                                 there are no more: the stages of A then lie
//                                 kARows rows apart, so the ring is deeper.  The
//                                 instruction reads 128 rows all the same, the next
//                                 stages' (or, in the second CTA, which loads no A,
//                                 whatever lies there): rows of the accumulator that
//                                 belong to no token, and rows do not mix.
//   Maps                          tensor maps of the epilogue
//   b_row(tile_n, rank, p)        first B row (or column) of this CTA's half
//   epilogue(...), helper(...)    see pair_kernel
//   init_barriers(ss)             the epilogue's own mbarriers (Shared::epi)
// W narrower than 128 gives more and smaller units when there are few; the ring
// then has more stages, so that as many bytes are on their way.
#pragma once

#include "launch.h"
#include "tc_kernel.cuh"

namespace forge {
namespace pairs {

constexpr int kEpiWarps = 16, kFirstEpiWarp = 4;
constexpr int kMaxStages = 24, kMaxBufs = 8;
constexpr int kA = kTileM * 128;  // bytes of A per stage and CTA

struct Shared {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[kMaxBufs];
  uint64_t tmem_empty[kMaxBufs];
  uint64_t mma_done;
  uint64_t epi[32];  // the epilogue's own
  uint32_t tmem_base;
  int32_t abort;
};
constexpr int kSharedBytes = 1024;
static_assert(sizeof(Shared) <= kSharedBytes, "shared state region");

// Bounded wait on an mbarrier phase.  Returns false if the CTA is aborting
// or the wait expired (the first expiry records the timeout).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const PairParams& p, Shared* ss,
                                     bool honour_abort = true) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::global_timer_ns();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (honour_abort && *reinterpret_cast<volatile int32_t*>(&ss->abort)) return false;
    if (ptx::global_timer_ns() - t0 > p.wait_limit_ns) {
      *reinterpret_cast<volatile int32_t*>(&ss->abort) = 1;
      atomicCAS(p.status, 0u, static_cast<uint32_t>(kStatusTimeout));
      return false;
    }
  }
}

// try_wait without a time to suspend for: 15 clocks where the phase is over, 50 with.
__device__ __forceinline__ bool try_once(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

// The same for a whole warp, which gets one verdict.  Every lane looks for
// itself first (what it saw is then ordered before its own reads); only when
// some lane saw nothing does lane 0 wait for all of them.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const PairParams& p, Shared* ss, int lane) {
  if (__all_sync(0xFFFFFFFFu, try_once(ptx::smem_addr(bar), parity))) return true;
  const bool ok = __all_sync(0xFFFFFFFFu, lane != 0 || wait(bar, parity, p, ss));
  __syncwarp();
  return ok;
}

template <class Op>
struct Layout {
  static constexpr int kBK = Op::kFp8 ? 128 : 64;
  static constexpr bool kShort = Op::kARows < kTileM;
  static constexpr int kAStage = Op::kARows * 128;  // bytes of A per stage and CTA
  static constexpr int kABytes = (Op::kStg - 1) * kAStage + kA;
  static constexpr int kB = Op::kW * 128;           // of B
  static constexpr uint32_t kTx = kShort ? kAStage + 2 * kB : 2 * (kAStage + kB);  // a stage's bytes, both CTAs'
  static constexpr int kSmem = kABytes + Op::kStg * kB + Op::kEpiBytes + kSharedBytes + 1024;
  static_assert(kSmem <= 232448, "dynamic shared memory limit");
  static_assert(Op::kStg <= kMaxStages && Op::kBufs <= kMaxBufs, "barrier arrays");
  static constexpr int kBufCols = kTmemCols / Op::kBufs;  // tensor-memory columns of an accumulator
  static_assert(kBufCols * Op::kSplit >= 2 * Op::kW && Op::kBufs % Op::kSplit == 0, "accumulators");
  static_assert(Op::kSplit == 1 || (Op::kFold == 1 && !Op::kBMajorMN), "halves of a stage");
  static constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
  // 65536 registers give 640 threads 96 each, five warpgroups 480; kMoreRegs:
  // the first keeps 32 and the epilogue's take 112 (32 + 4 x 112 = 480).
  static constexpr int kLoadRegs = 32, kEpiRegs = 112;
};

// One lane of the warp, which arrives converged.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// Both roles below run on their whole warp, one lane elected for each copy or
// instruction: addresses and descriptors are then the same in all lanes by
// construction, and live in the uniform registers these instructions read.
// (One lane alone in a branch had them moved there for every instruction: a
// stage's four narrow instructions, its wait and its commit took 389 clocks to
// issue, 212 so.)
template <class Op>
__device__ __forceinline__ void producer(const CUtensorMap* mA, const CUtensorMap* mB, const typename Op::Params& p,
                                         uint8_t* smA, uint8_t* smB, Shared* ss, int lane, uint32_t rank) {
  using L = Layout<Op>;
  constexpr int STG = Op::kStg, BK = L::kBK, kB = L::kB, W = Op::kW;
  uint32_t s = 0, ph = 0, issued_mask = 0, last_parity = 0;
  const uint32_t full0 = ptx::mapa(ptx::smem_addr(&ss->full[0]), 0);  // the leader's barriers
  // (the test hook: no loads, or those of each pair's first tile alone)
  const int end = p.skip_loads == 0 ? p.num_tiles : p.skip_loads == 2 ? min(p.num_tiles, num_pairs()) : 0;
  for (int tile = pair_id(); tile < end; tile += num_pairs()) {
    int tm, tn;
    tile_coords_of(tile, p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * kPairM + static_cast<int>(rank) * kTileM;
    const int b0 = Op::b_row(tn, static_cast<int>(rank), p);
    for (int kb = 0; kb < p.num_kb; ++kb) {
      if (!warp_wait(&ss->empty[s], ph ^ 1u, p, ss, lane)) goto drain;
      const uint32_t bar = full0 + s * 8u;
      uint8_t* a = smA + s * L::kAStage;
      uint8_t* b = smB + s * kB;
      if (elect_one()) {
        if (rank == 0) ptx::mbar_arrive_expect_tx(&ss->full[s], L::kTx);
        if (!L::kShort || rank == 0) ptx::tma_load_2d_pair(mA, bar, a, kb * BK, m0);
        if (!Op::kBMajorMN) {
          ptx::tma_load_2d_pair(mB, bar, b, kb * BK, b0);
        } else if (p.op3d) {  // [W / 64 column blocks][64 rows][64 columns] in one copy
          ptx::tma_load_3d_pair(mB, bar, b, 0, kb * BK, b0 / 64);
        } else {
#pragma unroll
          for (int i = 0; i < W / 64; ++i) ptx::tma_load_2d_pair(mB, bar, b + i * 64 * BK * 2, b0 + 64 * i, kb * BK);
        }
      }
      __syncwarp();
      issued_mask |= 1u << s;
      last_parity = (last_parity & ~(1u << s)) | (ph << s);
      if (++s == STG) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
drain:
  if (rank == 0 && lane == 0)  // every issued copy lands before the pair can exit
    for (int i = 0; i < STG; ++i)
      if (issued_mask & (1u << i)) wait(&ss->full[i], (last_parity >> i) & 1u, p, ss, false);
  __syncwarp();
}

// A stage's four instructions of the pair (32 bytes of the reduction each) and
// the commits that free its ring stage (with `free`) and hand the accumulator
// over (with `last`).  The upper halves of the descriptors are constant; the lower ones
// (address and leading offset) move by additions.
template <bool FP8, uint32_t BSTEP>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc, uint32_t add,
                                            uint32_t empty, uint32_t full, uint32_t free, uint32_t last) {
#define FORGE_STAGE(KIND)                                                                                              \
  asm volatile(                                                                                                        \
      "{\n\t.reg .pred e, f, g, p, t;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t.reg .b16 m;\n\t"                            \
      "mov.b16 m, 3;\n\tsetp.ne.b32 p, %5, 0;\n\tsetp.eq.u32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"              \
      "setp.ne.and.b32 f, %8, 0, e;\n\tsetp.ne.and.b32 g, %12, 0, e;\n\t"                                              \
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %4, p;\n\t" \
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"                    \
      "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %4, t;\n\t"                                             \
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, %10;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"                   \
      "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %4, t;\n\t"                                             \
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, %11;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"                   \
      "@e tcgen05.mma.cta_group::2.kind::" KIND " [%0], a, b, %4, t;\n\t"                                             \
      "@g tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%6], m;\n\t"       \
      "@f tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%7], m;\n\t}"      \
      ::"r"(d), "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(add), "r"(empty), "r"(full), "r"(last), "n"(BSTEP),       \
      "n"(2 * BSTEP), "n"(3 * BSTEP), "r"(free)                                                                        \
      : "memory")
  if constexpr (FP8) FORGE_STAGE("f8f6f4");
  else FORGE_STAGE("f16");
#undef FORGE_STAGE
}

// Leader CTA only.
template <class Op>
__device__ __forceinline__ void mma(const typename Op::Params& p, uint8_t* smA, uint8_t* smB, Shared* ss, int lane) {
  using L = Layout<Op>;
  constexpr int STG = Op::kStg, BK = L::kBK, kFold = Op::kFold > 0 ? Op::kFold : 1 << 30;
  constexpr uint32_t idesc = Op::kFp8 ? ptx::idesc_e4m3_f32(kPairM, 2 * Op::kW / Op::kSplit)
                                      : ptx::idesc_bf16_f32(kPairM, 2 * Op::kW, false, Op::kBMajorMN);
  // 8-row (or 8-column-atom) groups 1 KiB apart; B stored by columns: atoms of
  // 64 columns BK * 128 bytes apart, 16 rows of the reduction 2 KiB.
  const uint64_t ad = ptx::smem_desc_sw128(ptx::smem_addr(smA), 16, 1024);
  const uint64_t bd = ptx::smem_desc_sw128(ptx::smem_addr(smB), Op::kBMajorMN ? BK * 128 : 16, 1024);
  const uint32_t alo = static_cast<uint32_t>(ad), blo = static_cast<uint32_t>(bd), hi = static_cast<uint32_t>(ad >> 32);
  const uint32_t tmem = ss->tmem_base, empty0 = ptx::smem_addr(&ss->empty[0]), full0 = ptx::smem_addr(&ss->tmem_full[0]);
  uint32_t s = 0, ph = 0, acc = 0, aph = 0;
  for (int tile = pair_id(); tile < p.num_tiles; tile += num_pairs()) {
    for (int kb = 0; kb < p.num_kb; ++kb) {
      const bool first = kb % kFold == 0, last = kb % kFold == kFold - 1 || kb == p.num_kb - 1;
#pragma unroll
      for (uint32_t h = 0; h < Op::kSplit; ++h) {
        if (first && !warp_wait(&ss->tmem_empty[acc], aph ^ 1u, p, ss, lane)) goto done;
        if (h == 0 && !warp_wait(&ss->full[s], ph, p, ss, lane)) goto done;
        ptx::tc_fence_after();
        issue_stage<Op::kFp8, Op::kBMajorMN ? 2048 / 16 : 2>(
            tmem + acc * L::kBufCols, alo + s * (L::kAStage / 16), blo + s * (L::kB / 16) + h * (L::kB / Op::kSplit / 16), hi,
            idesc, first ? 0u : 1u, empty0 + s * 8u, full0 + acc * 8u, h == Op::kSplit - 1 ? 1u : 0u,
            last ? 1u : 0u);
        if (last && ++acc == Op::kBufs) {
          acc = 0;
          aph ^= 1u;
        }
      }
      if (++s == STG) {
        s = 0;
        ph ^= 1u;
      }
    }
  }
done:
  if (elect_one()) ptx::mma_commit_pair_multicast(&ss->mma_done, 0x1);
  __syncwarp();
  if (lane == 0) wait(&ss->mma_done, 0u, p, ss, false);
  __syncwarp();
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
__global__ void __launch_bounds__(Layout<Op>::kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB,
                const __grid_constant__ typename Op::Maps maps, const typename Op::Params p) {
  using L = Layout<Op>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + L::kABytes;
  uint8_t* epi = smB + Op::kStg * L::kB;
  Shared* ss = reinterpret_cast<Shared*>(epi + Op::kEpiBytes);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (the same in a warp's lanes)
  const uint32_t rank = ptx::cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < Op::kStg; ++s) {
      ptx::mbar_init(&ss->full[s], 1);
      ptx::mbar_init(&ss->empty[s], 1);
    }
    for (int a = 0; a < Op::kBufs; ++a) {
      ptx::mbar_init(&ss->tmem_full[a], 1);
      ptx::mbar_init(&ss->tmem_empty[a], 2 * kEpiWarps / Op::kSplit);
    }
    Op::init_barriers(ss);
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
  if (warp < kFirstEpiWarp) {
    if (Op::kMoreRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kLoadRegs));
    if (warp == 0) producer<Op>(&mapA, &mapB, p, smA, smB, ss, lane, rank);
    else if (warp >= 2) Op::helper(p, ss, epi, warp, lane, rank);
    else if (rank == 0) mma<Op>(p, smA, smB, ss, lane);
  } else {
    if (Op::kMoreRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kEpiRegs));
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
  cfg.blockDim = dim3(Layout<Op>::kThreads, 1, 1);
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
