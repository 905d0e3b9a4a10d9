// C ABI of the gated feed-forward block, the E4M3 codes in blocks of 128 and
// their product (declared in include/forge.h).  Argument checks and launches;
// nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "forge.h"
#include "host.h"
#include "launch.h"
#include "widths.h"

using namespace forge;

namespace {

constexpr int64_t kBlock = 128;
// row and column indices, with a tile's overhang, stay within 31 bits
constexpr int64_t kMost = (int64_t{1} << 31) - 1024;
constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// A pointer that must be there, aligned to `to` bytes.
forge_status_t need(const void* p, const char* name, uintptr_t to = 16) {
  if (p == nullptr) return fail(FORGE_ERR_INVALID_ARG, "%s is NULL", name);
  if ((reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0)
    return fail(FORGE_ERR_INVALID_ARG, "%s must be %d-byte aligned", name, static_cast<int>(to));
  return FORGE_OK;
}

forge_status_t ready(DeviceInfo* d) {
  const forge_status_t st = device_info(d);
  return st != FORGE_OK ? st : check_device(*d);
}

forge_status_t zero(void* p, int64_t bytes, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(bytes), s);
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "cudaMemsetAsync");
}

// The tiles of `rows` token rows x `cols` output columns, `wide` of them a tile.
void set_tiles(PairParams* p, int64_t rows, int64_t cols, int64_t wide, int64_t stages, const DeviceInfo& d) {
  const int64_t tm = ceil_div(rows, 2 * kTileM), tn = ceil_div(cols, wide);
  p->T = static_cast<int32_t>(rows);
  p->tiles_m = static_cast<int32_t>(tm);
  p->tiles_n = static_cast<int32_t>(tn);
  p->num_tiles = static_cast<int32_t>(tm * tn);
  p->num_kb = static_cast<int32_t>(stages);
  p->skip_loads = skip_loads();
  p->wait_limit_ns = wait_limit_ns();
  p->status = d.status;
}
// Their count, at the narrowest, has to fit an int.
forge_status_t check_tiles(int64_t rows, int64_t cols, int64_t narrowest) {
  if (ceil_div(rows, 2 * kTileM) * ceil_div(cols, narrowest) > (int64_t{1} << 30))
    return fail(FORGE_ERR_UNSUPPORTED, "too many output tiles (%lld x %lld)", (long long)rows, (long long)cols);
  return FORGE_OK;
}
// Token rows of a copy of the A operand.
uint32_t box_rows(int64_t T) { return T <= kShortRows ? kShortRows : kTileM; }
int pairs_of(const PairParams& p, const DeviceInfo& d) { return p.num_tiles < d.num_sms / 2 ? p.num_tiles : d.num_sms / 2; }

// The checks that both directions of the gated product share: shapes, the
// activation and what is kept.  R: the reduction's length.
forge_status_t check_gated(int64_t T, int64_t F, int64_t R, const char* r_name, int32_t act, const void* gu,
                           const void* codes, const float* scale) {
  if (T < 0 || F < 0 || R < 0)
    return fail(FORGE_ERR_INVALID_ARG, "negative shape T=%lld F=%lld %s=%lld", (long long)T, (long long)F, r_name, (long long)R);
  if (F % 8 != 0 || R % 8 != 0)
    return fail(FORGE_ERR_INVALID_ARG, "F and %s must be multiples of 8 (F=%lld %s=%lld)", r_name, (long long)F, r_name,
                (long long)R);
  if (T > kMost || 2 * F > kMost || R > kMost) return fail(FORGE_ERR_UNSUPPORTED, "T, 2 F and %s must fit in 31 bits", r_name);
  if (act != FORGE_ACT_SILU && act != FORGE_ACT_GELU_TANH) return fail(FORGE_ERR_INVALID_ARG, "act %d", act);
  if (gu != nullptr && codes != nullptr) return fail(FORGE_ERR_INVALID_ARG, "gu and gu_codes: one of them");
  if ((codes == nullptr) != (scale == nullptr)) return fail(FORGE_ERR_INVALID_ARG, "gu_codes and gu_scale go together");
  return check_tiles(T, F, kLeastWidth);
}

forge_status_t check_codes(int64_t rows, int64_t cols, int32_t x_dtype, int32_t block_rows) {
  if (rows < 0 || cols < 0)
    return fail(FORGE_ERR_INVALID_ARG, "negative shape rows=%lld cols=%lld", (long long)rows, (long long)cols);
  if (cols % 8 != 0) return fail(FORGE_ERR_INVALID_ARG, "cols must be a multiple of 8 (cols=%lld)", (long long)cols);
  if (x_dtype != FORGE_G_FP32 && x_dtype != FORGE_G_BF16) return fail(FORGE_ERR_INVALID_ARG, "x_dtype %d", x_dtype);
  if (block_rows != 1 && block_rows != kBlock) return fail(FORGE_ERR_INVALID_ARG, "block_rows must be 1 or 128 (got %d)", block_rows);
  if (rows > kMost || cols > kMost || ceil_div(rows, kBlock) * ceil_div(cols, kBlock) > kMost ||
      (rows > 0 && cols > (int64_t{1} << 40) / rows))
    return fail(FORGE_ERR_UNSUPPORTED, "rows, cols and the 128 x 128 blocks must fit in 31 bits, rows * cols in 40");
  return FORGE_OK;
}

}  // namespace

extern "C" {

forge_status_t forge_gated_linear(const forge_gated_t* g, void* stream) {
  clear_message();
  forge_status_t st;
  if (g == nullptr) return fail(FORGE_ERR_INVALID_ARG, "gated is NULL");
  const int64_t T = g->T, F = g->F, K = g->K;
  if ((st = check_gated(T, F, K, "K", g->act, g->gu, g->gu_codes, g->gu_scale)) != FORGE_OK) return st;
  if (T == 0 || F == 0) return FORGE_OK;
  if ((st = need(g->Y, "Y")) != FORGE_OK) return st;
  if (K > 0 && ((st = need(g->X, "X")) != FORGE_OK || (st = need(g->W, "W")) != FORGE_OK)) return st;
  if (g->gu != nullptr && (st = need(g->gu, "gu")) != FORGE_OK) return st;
  if (g->gu_codes != nullptr && ((st = need(g->gu_codes, "gu_codes")) != FORGE_OK || (st = need(g->gu_scale, "gu_scale", 4)) != FORGE_OK))
    return st;
  DeviceInfo d;
  if ((st = ready(&d)) != FORGE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t NB = ceil_div(F, kBlock);
  if (K == 0) {  // empty sums: zero projections
    if ((st = zero(g->Y, T * F * 2, s)) != FORGE_OK) return st;
    if (g->gu != nullptr && (st = zero(g->gu, T * F * 4, s)) != FORGE_OK) return st;
    if (g->gu_codes != nullptr && ((st = zero(g->gu_codes, T * F * 2, s)) != FORGE_OK || (st = zero(g->gu_scale, T * NB * 8, s)) != FORGE_OK))
      return st;
    return FORGE_OK;
  }
  const int width = g->gu_codes != nullptr ? 128 : pick_width(T, F, 1, kLeastWidth, d.num_sms / 2);
  GatedParams p;
  std::memset(&p, 0, sizeof(p));
  set_tiles(&p, T, F, width, ceil_div(K, kBlockK), d);
  p.F = static_cast<int32_t>(F);
  p.act = g->act;
  p.Y = g->Y;
  p.gu = g->gu;
  p.codes = g->gu_codes;
  p.scale = g->gu_scale;
  if (T <= kFewGated && g->gu_codes == nullptr && p.skip_loads == 0) {  // (that hook is for the pipelined kernels' waits)
    const cudaError_t e = launch_gated_few(g->W, g->X, p, static_cast<int>(K), s);
    return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "gated product launch");
  }
  CUtensorMap mx, mw;
  if ((st = tensor_map(&mx, g->X, kBf16, 2, K, T, kBlockK, g->gu_codes != nullptr ? kTileM : box_rows(T), CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK ||
      (st = tensor_map(&mw, g->W, kBf16, 2, K, 2 * F, kBlockK, static_cast<uint32_t>(width), CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK)
    return st;
  const cudaError_t e = launch_gated(width, mx, mw, p, pairs_of(p, d), s);
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "gated product launch");
}

forge_status_t forge_gated_dgrad(const forge_gated_grad_t* g, void* stream) {
  clear_message();
  forge_status_t st;
  if (g == nullptr) return fail(FORGE_ERR_INVALID_ARG, "grad is NULL");
  const int64_t T = g->T, F = g->F, N = g->N;
  if ((st = check_gated(T, F, N, "N", g->act, g->gu, g->gu_codes, g->gu_scale)) != FORGE_OK) return st;
  if (T == 0 || F == 0) return FORGE_OK;
  if (g->gu == nullptr && g->gu_codes == nullptr) return fail(FORGE_ERR_INVALID_ARG, "gu or gu_codes is needed");
  if ((st = need(g->dGU, "dGU")) != FORGE_OK) return st;
  if (N > 0 && ((st = need(g->dY, "dY")) != FORGE_OK || (st = need(g->Wd, "Wd")) != FORGE_OK)) return st;
  if (N == 0) return fail(FORGE_ERR_UNSUPPORTED, "the gradient needs N > 0");
  if (g->gu != nullptr && (st = need(g->gu, "gu")) != FORGE_OK) return st;
  if (g->gu_codes != nullptr && ((st = need(g->gu_codes, "gu_codes")) != FORGE_OK || (st = need(g->gu_scale, "gu_scale", 4)) != FORGE_OK))
    return st;
  if (g->Y != nullptr && (st = need(g->Y, "Y")) != FORGE_OK) return st;
  DeviceInfo d;
  if ((st = ready(&d)) != FORGE_OK) return st;
  const int width = pick_width(T, F, 2, 64, d.num_sms / 2);
  GatedParams p;
  std::memset(&p, 0, sizeof(p));
  set_tiles(&p, T, F, 2 * width, ceil_div(N, kBlockK), d);
  p.F = static_cast<int32_t>(F);
  p.act = g->act;
  p.Y = g->Y;
  p.gu = const_cast<void*>(g->gu);
  p.codes = const_cast<void*>(g->gu_codes);
  p.scale = const_cast<float*>(g->gu_scale);
  p.dGU = g->dGU;
  p.op3d = F % 64 == 0;
  CUtensorMap my, mw;
  if ((st = tensor_map(&my, g->dY, kBf16, 2, N, T, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK) return st;
  if (p.op3d) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(F) / 64};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(F) * 2, 128};
    const cuuint32_t box[3] = {64, kBlockK, static_cast<cuuint32_t>(width) / 64};
    st = tensor_map_nd(&mw, g->Wd, kBf16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    st = tensor_map(&mw, g->Wd, kBf16, 2, F, N, 64, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (st != FORGE_OK) return st;
  const cudaError_t e = launch_gated_grad(width, my, mw, p, pairs_of(p, d), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "gated gradient launch");
}

forge_status_t forge_quantize_e4m3(const void* x, int32_t x_dtype, void* codes, float* scale, int64_t rows, int64_t cols,
                                   int32_t block_rows, void* stream) {
  clear_message();
  forge_status_t st;
  if ((st = check_codes(rows, cols, x_dtype, block_rows)) != FORGE_OK) return st;
  if (rows == 0 || cols == 0) return FORGE_OK;
  if ((st = need(x, "x")) != FORGE_OK || (st = need(codes, "codes")) != FORGE_OK || (st = need(scale, "scale", 4)) != FORGE_OK)
    return st;
  DeviceInfo d;
  if ((st = ready(&d)) != FORGE_OK) return st;
  const CodesParams p = {x, static_cast<uint8_t*>(codes), scale, rows, cols, block_rows != 1};
  const cudaError_t e = launch_quantize_e4m3(x_dtype == FORGE_G_FP32, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "quantise launch");
}

forge_status_t forge_dequantize_e4m3(const void* codes, const float* scale, void* x, int32_t x_dtype, int64_t rows,
                                     int64_t cols, int32_t block_rows, void* stream) {
  clear_message();
  forge_status_t st;
  if ((st = check_codes(rows, cols, x_dtype, block_rows)) != FORGE_OK) return st;
  if (rows == 0 || cols == 0) return FORGE_OK;
  if ((st = need(x, "x")) != FORGE_OK || (st = need(codes, "codes")) != FORGE_OK || (st = need(scale, "scale", 4)) != FORGE_OK)
    return st;
  DeviceInfo d;
  if ((st = ready(&d)) != FORGE_OK) return st;
  const CodesParams p = {x, static_cast<uint8_t*>(const_cast<void*>(codes)), const_cast<float*>(scale), rows, cols, block_rows != 1};
  const cudaError_t e = launch_dequantize_e4m3(x_dtype == FORGE_G_FP32, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "dequantise launch");
}

forge_status_t forge_linear_e4m3(const forge_linear_e4m3_t* lin, void* stream) {
  clear_message();
  forge_status_t st;
  if (lin == nullptr) return fail(FORGE_ERR_INVALID_ARG, "linear is NULL");
  const int64_t T = lin->T, N = lin->N, K = lin->K;
  if (T < 0 || N < 0 || K < 0)
    return fail(FORGE_ERR_INVALID_ARG, "negative shape T=%lld N=%lld K=%lld", (long long)T, (long long)N, (long long)K);
  if (N % 8 != 0 || K % 16 != 0)
    return fail(FORGE_ERR_INVALID_ARG, "N must be a multiple of 8 and K of 16 (N=%lld K=%lld)", (long long)N, (long long)K);
  if (T > kMost || N > kMost || K > kMost) return fail(FORGE_ERR_UNSUPPORTED, "T, N and K must fit in 31 bits");
  if ((st = check_tiles(T, N, 2 * kLeastWidth)) != FORGE_OK) return st;
  if (T == 0 || N == 0) return FORGE_OK;
  if ((st = need(lin->Y, "Y")) != FORGE_OK) return st;
  if (K > 0 && ((st = need(lin->Xq, "Xq")) != FORGE_OK || (st = need(lin->Wq, "Wq")) != FORGE_OK ||
                (st = need(lin->x_scale, "x_scale", 4)) != FORGE_OK || (st = need(lin->w_scale, "w_scale", 4)) != FORGE_OK))
    return st;
  DeviceInfo d;
  if ((st = ready(&d)) != FORGE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return zero(lin->Y, T * N * 2, s);  // empty sums
  const int width = pick_width(T, N, 2, kLeastWidth, d.num_sms / 2);
  ProductParams p;
  std::memset(&p, 0, sizeof(p));
  set_tiles(&p, T, N, 2 * width, ceil_div(K, kBlock), d);
  p.N = static_cast<int32_t>(N);
  p.x_scale = lin->x_scale;
  p.w_scale = lin->w_scale;
  p.Y = lin->Y;
  if (T <= kFewProduct && p.skip_loads == 0) {
    const cudaError_t e = launch_product_few(lin->Wq, lin->Xq, p, static_cast<int>(K), d.num_sms, s);
    return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "block-scaled product launch");
  }
  CUtensorMap mx, mw;
  if ((st = tensor_map(&mx, lin->Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, T, kBlock, box_rows(T), CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK ||
      (st = tensor_map(&mw, lin->Wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, N, kBlock, static_cast<uint32_t>(width),
                       CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK)
    return st;
  CUtensorMap my = mx;
  if (width == 128 && (st = tensor_map(&my, lin->Y, kBf16, 2, N, T, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B)) != FORGE_OK) return st;
  const cudaError_t e = launch_product(width, mx, mw, my, p, pairs_of(p, d), s);
  return e == cudaSuccess ? FORGE_OK : cuda_fail(e, "block-scaled product launch");
}

}  // extern "C"
