// The widths of the pair kernels' tiles (pair_gemm.cuh), chosen on the host.
#pragma once

#include <cstdint>

#include "common.h"

namespace forge {

constexpr int kLeastWidth = 32;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The width of a CTA's B half (128, 64 or `least`): the one whose rounds of
// tiles over the pairs cost least by one estimate for every kernel.  A narrow
// tile costs more than its share (the token operand is loaded and read again
// for each, and its stages are short): 62 and 54 where the widest costs 100.
// us at widths 128, 64 and 32, the one taken in brackets (product: codes; else
// the gated forward, of 2 F rows of weights):
//   300 x 14336 x 4096  [66]  78  137      128 x 14336 x 4096   52  [48]  72
//   24 x 2048 x 4096     25   19  [21]     product 33 x 4096 x 14336   58  38  [37]
//   product 1531 x 5120 x 17408  [135]  166  261
//   product 300 x 14336 x 4096   40  [38]  58
// So it is a fit, and 24 x 2048 x 4096, a narrow block's decoding, is 2 us off
// its best.
// `halves`: B halves side by side in a tile's output columns (2), or on top of
// each other (1: gate and up).
inline int pick_width(int64_t rows, int64_t cols, int halves, int least, int pairs) {
  constexpr int kCost[3] = {100, 62, 54};
  int best = 128;
  int64_t cost = 0;
  for (int w = 128, i = 0; w >= least; w /= 2, ++i) {
    const int64_t units = ceil_div(rows, 2 * kTileM) * ceil_div(cols, halves * w);
    const int64_t c = ceil_div(units, pairs) * kCost[i];
    if (w == 128 || c < cost) {
      cost = c;
      best = w;
    }
  }
  return best;
}

}  // namespace forge
