// Instantiations of the tensor-core kernel for the grouped FORGE step (bf16
// weights): every expert's weight gradient and optimizer step in one launch.
// Short groups; tc_grouped_long.cu holds the long ones.
#include "tc_grouped.cuh"

namespace forge {

cudaError_t launch_tc_grouped(int mode, int sdt, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& s1,
                              const CUtensorMap& s2, const CUtensorMap& w, const GemmParams& p, int grid,
                              cudaStream_t s, bool after_dx) {
  const bool d = after_dx;
  if (mode != kModeGrouped) return launch_tc_grouped_long(mode, sdt, a, b, s1, s2, w, p, grid, s, d);
  return sdt == kSBf16 ? run_grouped_step<kModeGrouped, kSBf16>(a, b, s1, s2, w, p, grid, s, d)
                       : run_grouped_step<kModeGrouped, kSFp32>(a, b, s1, s2, w, p, grid, s, d);
}

}  // namespace forge
