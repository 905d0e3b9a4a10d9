// Instantiations of the tensor-core kernel for the grouped FORGE step over
// longer groups, and with INT8 states.
#include "tc_grouped.cuh"

namespace forge {

cudaError_t launch_tc_grouped_long(int mode, int sdt, const CUtensorMap& a, const CUtensorMap& b,
                                   const CUtensorMap& s1, const CUtensorMap& s2, const CUtensorMap& w,
                                   const GemmParams& p, int grid, cudaStream_t s, bool after_dx) {
  const bool d = after_dx;
  if (mode == kModeGroupedMid)
    return sdt == kSBf16 ? run_grouped_step<kModeGroupedMid, kSBf16>(a, b, s1, s2, w, p, grid, s, d)
                         : run_grouped_step<kModeGroupedMid, kSFp32>(a, b, s1, s2, w, p, grid, s, d);
  return sdt == kSInt8W    ? run_grouped_step<kModeGroupedLong, kSInt8W>(a, b, s1, s2, w, p, grid, s, d)
         : sdt == kSInt8WX ? run_grouped_step<kModeGroupedLong, kSInt8WX>(a, b, s1, s2, w, p, grid, s, d)
         : sdt == kSBf16   ? run_grouped_step<kModeGroupedLong, kSBf16>(a, b, s1, s2, w, p, grid, s, d)
                           : run_grouped_step<kModeGroupedLong, kSFp32>(a, b, s1, s2, w, p, grid, s, d);
}

}  // namespace forge
