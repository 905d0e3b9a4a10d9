// Instantiations of the tensor-core kernel for the grouped FORGE step (bf16
// weights): every expert's weight gradient and optimizer step in one launch.
#include "launch.h"
#include "tc_kernel.cuh"

namespace forge {

template <int SDT>
static cudaError_t run_grouped_step(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& s1,
                                    const CUtensorMap& s2, const CUtensorMap& w, const GemmParams& p, int grid,
                                    cudaStream_t s, bool after_dx) {
  auto* k = tc_kernel<kModeGrouped, kWBf16, SDT>;
  using Cfg = KCfg<kModeGrouped, kWBf16, SDT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pair(k, grid, Cfg::kThreads, Cfg::kSmem, s, a, b, a, b, s1, s2, a, w, p, after_dx);
}

cudaError_t launch_tc_grouped(int sdt, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& s1,
                              const CUtensorMap& s2, const CUtensorMap& w, const GemmParams& p, int grid,
                              cudaStream_t s, bool after_dx) {
  const bool d = after_dx;
  return sdt == kSInt8W    ? run_grouped_step<kSInt8W>(a, b, s1, s2, w, p, grid, s, d)
         : sdt == kSInt8WX ? run_grouped_step<kSInt8WX>(a, b, s1, s2, w, p, grid, s, d)
         : sdt == kSBf16   ? run_grouped_step<kSBf16>(a, b, s1, s2, w, p, grid, s, d)
                           : run_grouped_step<kSFp32>(a, b, s1, s2, w, p, grid, s, d);
}

}  // namespace forge
