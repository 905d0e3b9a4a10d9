// The launch of one instantiation of the grouped FORGE step.
#pragma once

#include "launch.h"
#include "tc_kernel.cuh"

namespace forge {

template <int MODE, int SDT>
cudaError_t run_grouped_step(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& s1,
                             const CUtensorMap& s2, const CUtensorMap& w, const GemmParams& p, int grid,
                             cudaStream_t s, bool after_dx) {
  auto* k = tc_kernel<MODE, kWBf16, SDT>;
  using Cfg = KCfg<MODE, kWBf16, SDT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pair(k, grid, Cfg::kThreads, Cfg::kSmem, s, a, b, a, b, s1, s2, a, w, p, after_dx);
}

}  // namespace forge
