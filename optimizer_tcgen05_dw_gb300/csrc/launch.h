// Host-side launchers of the kernels, one per translation unit, called by the
// C ABI in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.h"

namespace forge {

// Parameters of the elementwise (non-tensor-core) kernels.
struct ElemParams {
  const float* dW;   // optimizer step: fp32 gradient (nullptr = zero); quantise: input
  void* W;
  void* s1;
  void* s2;
  float* s1_scale;
  float* s2_scale;
  int64_t N, K;      // rows, columns
  OptScalars sc;
  uint64_t seed, step;
  uint64_t sr_base;  // added to each 8-element group's index in the rounding counter
  int32_t is_signed; // quantise / dequantise
  int32_t qblock;    // INT8 states: elements per absmax block (32, 64, 128 or 256)
};

// tc_fused.cu: the FORGE step (mode kModeFusedOpt) for one (W dtype, state dtype).
// s1, s2: tensor maps of the state tiles the bf16-weight epilogue stages
// through shared memory (unused, any valid map, for fp32 weights or for
// states the rule does not keep); w: bf16 W in 64-column x 128-row boxes
// (128-byte swizzle), staged when sdt is kSInt8W (else any valid map); bh:
// the B operand in 64-column boxes for half units (GemmParams::split_from;
// any valid map when nothing is split).
// With `after_dx` the launch may start while the fp32-weight dX kernel before
// it on the stream still runs (programmatic dependent launch); its epilogue
// waits for that grid before writing weights or states.
cudaError_t launch_tc_fused(int wdt, int sdt, const CUtensorMap& a, const CUtensorMap& b,
                            const CUtensorMap& bh, const CUtensorMap& s1, const CUtensorMap& s2,
                            const CUtensorMap& w, const GemmParams& p, int grid, cudaStream_t s,
                            bool after_dx = false);
// tc_step.cu: dX and the FORGE step in one launch (mode kModeStep, bf16
// weights): a, b the dW operands, da, db the dX operands (dY K-major, W),
// dx the dX output (bf16, 64-column x 128-row boxes, 128-byte swizzle).
cudaError_t launch_tc_step(int sdt, const CUtensorMap& a, const CUtensorMap& b,
                           const CUtensorMap& da, const CUtensorMap& db, const CUtensorMap& s1,
                           const CUtensorMap& s2, const CUtensorMap& dx, const CUtensorMap& w,
                           const GemmParams& p, int grid, cudaStream_t s);
// CTA pairs of the one-launch step that can be resident at once (its dW tiles
// wait for dX tiles of other pairs, so its grid must not exceed this); 0 if
// the query fails.
int step_max_pairs(int sdt);
// tc_fp8.cu: the FORGE step from E4M3 operands (mode kModeFusedFp8, bf16
// weights): a = dY^T codes [N x T], b = X^T codes [K x T], 128 x 128-byte
// boxes with the 128-byte swizzle; p.gscale the product of the scales.
cudaError_t launch_tc_fp8(int sdt, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& bh,
                          const CUtensorMap& s1, const CUtensorMap& s2, const CUtensorMap& w,
                          const GemmParams& p, int grid, cudaStream_t s);
// tc_plain.cu: unfused pass 1 (kModeWgradStore) or dX (kModeDgrad).
cudaError_t launch_tc_plain(int mode, const CUtensorMap& a, const CUtensorMap& b,
                            const GemmParams& p, int grid, cudaStream_t s);
// elementwise.cu
cudaError_t launch_opt_step(int wdt, int sdt, const ElemParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_quantize(const ElemParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_dequantize(const ElemParams& p, int num_sms, cudaStream_t s);
// dX = dY * bf16(W) for fp32 master weights (CUDA cores); its blocks let the
// next launch on the stream start early (programmatic dependent launch).
cudaError_t launch_dgrad_fp32w(const void* dY, const float* W, void* dX, int64_t T, int64_t N,
                               int64_t K, int num_sms, cudaStream_t s);


// The grouped step's mode for T tokens over `groups` experts.  An expert's
// length is known on the device only, so the rule goes by their mean.  Step
// kernels, us, fp32 and bf16 moments, in the order short, middle, long
// (16384 tokens):
//   mean 16384 (1 of 4096 x 4096)   526 408   420 362   363 354
//   mean  4096 (4 of 4096 x 4096)   562 428   468 395   425 390
//   mean  2048 (8 of 4096 x 4096)   681 492   577 468   686 527
//   mean  1024 (16 of 2048 x 4096)  493 367   577 434   661 504
inline int group_mode(int64_t T, int64_t groups, int sdt) {
  if (sdt != kSFp32 && sdt != kSBf16) return kModeGroupedLong;
  return T < 1536 * groups ? kModeGrouped : (T < 3584 * groups ? kModeGroupedMid : kModeGroupedLong);
}
// tc_grouped.cu, tc_grouped_long.cu: the FORGE step of every expert (modes
// kModeGrouped*, bf16 weights): a, b the operands with a stage's rows as a
// dimension (see producer_role), s1, s2, w with the experts as a third.  With
// `after_dx` the launch may start while the grouped dX kernel before it on the
// stream still runs; it writes nothing before that grid has ended.
cudaError_t launch_tc_grouped(int mode, int sdt, const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& s1,
                              const CUtensorMap& s2, const CUtensorMap& w, const GemmParams& p, int grid,
                              cudaStream_t s, bool after_dx);
cudaError_t launch_tc_grouped_long(int mode, int sdt, const CUtensorMap& a, const CUtensorMap& b,
                                   const CUtensorMap& s1, const CUtensorMap& s2, const CUtensorMap& w,
                                   const GemmParams& p, int grid, cudaStream_t s, bool after_dx);
// grouped.cu: the grouped forward product (dgrad false) or dX (true).  w: the
// weights' map; tok[i]: the token operand in boxes of 64 columns x (16 << i)
// rows.
cudaError_t launch_grouped(bool dgrad, const CUtensorMap& w, const CUtensorMap (&tok)[4],
                           const GroupedParams& p, int grid, cudaStream_t s);
// grouped.cu: the forward product of at most kFewMaxT token rows (K: reduction
// length).  Against the tensor-core tiles, us in a graph for experts of 2048 x
// 4096: one row 7 and 21; 32 rows of one expert 24 to 26 and 22, over 16 experts
// 43 and 48; 64 rows of one expert (read twice here) 37 and 22, over 16 experts 46
// and 48.
constexpr int64_t kFewMaxT = 32;
cudaError_t launch_grouped_few(const void* W, const void* X, const GroupedParams& p, int K, int num_sms,
                               cudaStream_t s);

// One tensor of a many-tensor optimizer step.
struct MultiItem {
  const void* g;     // gradient (nullptr = zero)
  void* W;
  void* s1;
  void* s2;
  float* s1_scale;
  float* s2_scale;
  int64_t n;         // elements
  uint32_t first;    // its first tile in the launch
  uint32_t index;    // its place in the caller's list: added to the rounding seed
};
// Tensors a launch carries in its parameters (64 bytes each, 32 KB at most).
constexpr int kMultiShort = 56, kMultiMiddle = 140, kMultiLong = 480;
constexpr int kMultiTile = 2048;  // elements per block
template <int CAP>
struct MultiParams {
  OptScalars sc;
  uint64_t seed, step;
  int32_t count;     // tensors
  int32_t qblock;    // INT8 states: elements per absmax block
  MultiItem items[CAP];
};
// multi.cu: the rule over `tiles` tiles of p.count tensors, one block a tile.
cudaError_t launch_multi(int wdt, int sdt, int gdt, const MultiParams<kMultiLong>& p, uint32_t tiles,
                         cudaStream_t s);

// Root-mean-square norm (norm.cu).
struct NormParams {
  const void* x;         // [T x K] bf16 input (bwd: the stream h the norm read)
  const void* res;       // [T x K] bf16 residual, or nullptr
  const void* w;         // [K] bf16
  void* h;               // [T x K] bf16: x + residual, or nullptr
  float* rstd;           // [T] (bwd: input), or nullptr
  void* y;               // [T x K] bf16, or nullptr (bwd: dx)
  void* q;               // [T x K] E4M3, or nullptr
  float* q_scale;        // [T]
  void* qt;              // [K x T] E4M3, or nullptr
  float* amax;           // [1], or nullptr
  const void* dy;        // bwd: [T x K] bf16
  const void* dh;        // bwd: [T x K] bf16, or nullptr
  float* dw;             // bwd: [K]
  float* partial;        // bwd: [blocks x K]
  int64_t T;
  int32_t K;
  float eps;
  float inv_scale;       // qt: 1 / its scale
  uint64_t wait_limit_ns;  // qt: how long a block waits for its cluster's
  uint32_t* status;      // device status word
  int32_t skip_sends;    // qt: the test hook of the failure path
};
cudaError_t launch_norm_fwd(const NormParams& p, int num_sms, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormParams& p, int num_sms, cudaStream_t s);
// Rows of p.partial that launch_norm_bwd uses.
int64_t norm_bwd_blocks(int64_t T, int K, int num_sms);

}  // namespace forge
