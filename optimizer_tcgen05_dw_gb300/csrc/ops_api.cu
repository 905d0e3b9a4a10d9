// C ABI of the operators around the linear step (declared in include/forge.h):
// the grouped linears, the many-tensor optimizer step and the norm.  Argument checks and launches;
// nothing here allocates device memory.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "forge.h"
#include "host.h"
#include "launch.h"

using namespace forge;

namespace {

constexpr int64_t kMaxNormCols = 16384;  // four vectors a thread, 512 threads
constexpr uint32_t kMaxMultiTiles = 1u << 30;

forge_status_t check_norm_shape(int64_t T, int64_t K) {
  if (T < 0) return fail(FORGE_ERR_INVALID_ARG, "negative T=%lld", (long long)T);
  if (K < 8 || K % 8 != 0) return fail(FORGE_ERR_INVALID_ARG, "K must be a positive multiple of 8 (K=%lld)", (long long)K);
  if (K > kMaxNormCols || T > (int64_t{1} << 31) - 1)
    return fail(FORGE_ERR_UNSUPPORTED, "the norm takes K <= %lld and T below 2^31 (T=%lld K=%lld)",
                (long long)kMaxNormCols, (long long)T, (long long)K);
  return FORGE_OK;
}

// A pointer that must be there (or may be NULL when `optional`), 16-byte aligned.
forge_status_t check_ptr(const void* p, const char* name, bool optional = false) {
  if (p == nullptr) return optional ? FORGE_OK : fail(FORGE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned16(p)) return fail(FORGE_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return FORGE_OK;
}

// ---------------------------------------------------------------- grouped linears

forge_status_t check_grouped(const forge_grouped_t* g) {
  if (g == nullptr) return fail(FORGE_ERR_INVALID_ARG, "grouped is NULL");
  if (g->T < 0 || g->N < 0 || g->K < 0 || g->groups < 0)
    return fail(FORGE_ERR_INVALID_ARG, "negative shape T=%lld N=%lld K=%lld groups=%d", (long long)g->T,
                (long long)g->N, (long long)g->K, g->groups);
  if (g->N % 8 != 0 || g->K % 8 != 0)
    return fail(FORGE_ERR_INVALID_ARG, "N and K must be multiples of 8 (N=%lld K=%lld)", (long long)g->N,
                (long long)g->K);
  // row indices, with the tile's overhang, stay within 31 bits
  constexpr int64_t kMost = (int64_t{1} << 31) - 1024;
  if (g->T > kMost || g->K > kMost || g->N > kMost || static_cast<int64_t>(g->groups) * g->N > kMost)
    return fail(FORGE_ERR_UNSUPPORTED, "T, K and groups * N must fit in 31 bits");
  if (g->groups > kMaxGroups) return fail(FORGE_ERR_UNSUPPORTED, "at most %d groups (got %d)", kMaxGroups, g->groups);
  if (g->groups > 0 && (g->offsets == nullptr || (reinterpret_cast<uintptr_t>(g->offsets) & 3u) != 0))
    return fail(FORGE_ERR_INVALID_ARG, "offsets must be a non-NULL 4-byte aligned device pointer");
  return FORGE_OK;
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// out[t, :] = W_e tok[t, :] (dgrad false: tok = X, out = Y) or W_e^T tok[t, :]
// (tok = dY, out = dX).
forge_status_t grouped_product(const forge_grouped_t* g, const void* W, bool dgrad, const DeviceInfo& d, cudaStream_t s) {
  const int64_t F = dgrad ? g->K : g->N, R = dgrad ? g->N : g->K;
  const void* tok = dgrad ? g->dY : g->X;
  void* out = dgrad ? g->dX : g->Y;
  if (g->T == 0 || F == 0) return FORGE_OK;
  forge_status_t st;
  cudaError_t e;
  if ((st = check_ptr(out, dgrad ? "dX" : "Y")) != FORGE_OK) return st;
  if (R == 0 || g->groups == 0) {  // an empty sum, or rows of no group
    if ((e = cudaMemsetAsync(out, 0, static_cast<size_t>(g->T * F * 2), s)) != cudaSuccess)
      return cuda_fail(e, "cudaMemsetAsync");
    return FORGE_OK;
  }
  if ((st = check_ptr(tok, dgrad ? "dY" : "X")) != FORGE_OK || (st = check_ptr(W, "W")) != FORGE_OK) return st;
  GroupedParams p;
  std::memset(&p, 0, sizeof(p));
  p.offsets = g->offsets;
  p.groups = g->groups;
  p.T = static_cast<int32_t>(g->T);
  p.F = static_cast<int32_t>(F);
  p.w_rows = static_cast<int32_t>(g->N);
  p.num_kb = static_cast<int32_t>((R + kBlockK - 1) / kBlockK);
  p.tiles_f = static_cast<int32_t>((F + 2 * kTileM - 1) / (2 * kTileM));
  p.out = out;
  p.wait_limit_ns = wait_limit_ns();
  p.status = d.status;
  p.skip_loads = skip_loads() ? 1 : 0;
  if (!dgrad && g->T <= kFewMaxT && p.skip_loads == 0) {  // (that hook is for the pipelined kernels' waits)
    if ((e = launch_grouped_few(W, tok, p, static_cast<int>(R), d.num_sms, s)) != cudaSuccess)
      return cuda_fail(e, "grouped product launch");
    return FORGE_OK;
  }
  const cuuint64_t N = static_cast<cuuint64_t>(g->N), K = static_cast<cuuint64_t>(g->K),
                   E = static_cast<cuuint64_t>(g->groups);
  CUtensorMap mw, mt[4];
  if (!dgrad) {
    st = tensor_map(&mw, W, kBf16, 2, g->K, g->N * g->groups, kBlockK, kTileM, CU_TENSOR_MAP_SWIZZLE_128B);
  } else if (K % 64 == 0) {
    p.w3d = 1;
    const cuuint64_t dims[4] = {64, N, K / 64, E}, strides[3] = {K * 2, 128, N * K * 2};
    const cuuint32_t box[4] = {64, kBlockK, 2, 1};
    st = tensor_map_nd(&mw, W, kBf16, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  } else {
    const cuuint64_t dims[3] = {K, N, E}, strides[2] = {K * 2, N * K * 2};
    const cuuint32_t box[3] = {64, kBlockK, 1};
    st = tensor_map_nd(&mw, W, kBf16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (st != FORGE_OK) return st;
  for (int i = 0; i < 4; ++i)
    if ((st = tensor_map(&mt[i], tok, kBf16, 2, R, g->T, kBlockK, 16u << i, CU_TENSOR_MAP_SWIZZLE_128B)) != FORGE_OK)
      return st;
  // at most one column tile per 256 tokens and one more for each group that has any
  const int64_t tiles = g->T / kTileN + (g->groups < g->T ? g->groups : g->T);
  const int64_t pairs = tiles * p.tiles_f < d.num_sms / 2 ? tiles * p.tiles_f : d.num_sms / 2;
  if ((e = launch_grouped(dgrad, mw, mt, p, static_cast<int>(2 * pairs), s)) != cudaSuccess)
    return cuda_fail(e, dgrad ? "grouped dX launch" : "grouped product launch");
  return FORGE_OK;
}

// The weight-gradient operand [T x cols] of the grouped step, 64 columns x 64
// rows a box: the rows of a stage are dimension 1 (of extent 64, so that a box
// may start before it and read zeros), the row a stage starts from the last.
forge_status_t ragged_map(CUtensorMap* m, const void* base, int64_t cols, int64_t T, bool blocks) {
  const cuuint64_t ld = static_cast<cuuint64_t>(cols) * 2;
  if (blocks) {
    const cuuint64_t dims[4] = {64, kFusedBlockK, static_cast<cuuint64_t>(cols) / 64, static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[3] = {ld, 128, ld};
    const cuuint32_t box[4] = {64, kFusedBlockK, 2, 1};
    return tensor_map_nd(m, base, kBf16, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), kFusedBlockK, static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {ld, ld};
  const cuuint32_t box[3] = {64, kFusedBlockK, 1};
  return tensor_map_nd(m, base, kBf16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// A tensor [groups x N x K] in boxes of box_cols x 128 rows of one expert.
forge_status_t expert_map(CUtensorMap* m, const void* base, CUtensorMapDataType dtype, int esize, const forge_grouped_t* g,
                          uint32_t box_cols, CUtensorMapSwizzle swizzle) {
  const cuuint64_t N = static_cast<cuuint64_t>(g->N), K = static_cast<cuuint64_t>(g->K);
  const cuuint64_t dims[3] = {K, N, static_cast<cuuint64_t>(g->groups)};
  const cuuint64_t strides[2] = {K * esize, N * K * esize};
  const cuuint32_t box[3] = {box_cols, kTileM, 1};
  return tensor_map_nd(m, base, dtype, 3, dims, strides, box, swizzle);
}

}  // namespace

extern "C" {

forge_status_t forge_grouped_linear(const forge_grouped_t* g, const void* W, void* stream) {
  clear_message();
  forge_status_t st;
  if ((st = check_grouped(g)) != FORGE_OK) return st;
  if (g->T == 0 || g->N == 0) return FORGE_OK;
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  return grouped_product(g, W, false, d, static_cast<cudaStream_t>(stream));
}

forge_status_t forge_grouped_dgrad(const forge_grouped_t* g, const void* W, void* stream) {
  clear_message();
  forge_status_t st;
  if ((st = check_grouped(g)) != FORGE_OK) return st;
  if (g->T == 0 || g->K == 0) return FORGE_OK;
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  return grouped_product(g, W, true, d, static_cast<cudaStream_t>(stream));
}

forge_status_t forge_grouped_bwd_step(const forge_grouped_t* g, const forge_state_t* state, int32_t opt_kind,
                                      const forge_hparams_t* hp, int64_t step, uint64_t seed, void* stream) {
  clear_message();
  forge_status_t st;
  if ((st = check_grouped(g)) != FORGE_OK) return st;
  if ((st = check_hp(opt_kind, hp, step)) != FORGE_OK) return st;
  const int64_t T = g->T, N = g->N, K = g->K;
  if ((st = check_state(state, opt_kind, N * g->groups, K)) != FORGE_OK) return st;
  if (state->w_dtype != FORGE_W_BF16_SR)
    return fail(FORGE_ERR_UNSUPPORTED, "the grouped step takes bf16 weights (w_dtype must be FORGE_W_BF16_SR)");
  const bool any = g->groups > 0 && N > 0 && K > 0;
  if (T > 0 && any && ((st = check_ptr(g->X, "X")) != FORGE_OK || (st = check_ptr(g->dY, "dY")) != FORGE_OK)) return st;
  if (g->dX != nullptr && (st = check_ptr(g->dX, "dX")) != FORGE_OK) return st;
  if (!any && (g->dX == nullptr || T == 0 || K == 0)) return FORGE_OK;
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // 1. dX from the weights before the update, first on the stream
  if (g->dX != nullptr && (st = grouped_product(g, state->W, true, d, s)) != FORGE_OK) return st;
  if (!any) return FORGE_OK;
  const OptScalars sc = make_scalars(opt_kind, *hp, step);
  const int qb = qblock_of(state->s_dtype);
  cudaError_t e;
  if (T == 0) {  // no token: the rule on a zero gradient
    ElemParams ep;
    std::memset(&ep, 0, sizeof(ep));
    ep.W = state->W; ep.s1 = state->s1; ep.s2 = state->s2;
    ep.s1_scale = state->s1_scale; ep.s2_scale = state->s2_scale;
    ep.N = N * g->groups; ep.K = K; ep.sc = sc; ep.seed = seed; ep.step = static_cast<uint64_t>(step);
    ep.qblock = qb;
    if ((e = launch_opt_step(state->w_dtype, base_sdt(state->s_dtype), ep, d.num_sms, s)) != cudaSuccess)
      return cuda_fail(e, "optimizer launch (T = 0)");
    return FORGE_OK;
  }
  // 2. every expert's weight gradient and optimizer step
  const int sdt = qb == 64 ? kSInt8W : (qb != 0 ? kSInt8WX : base_sdt(state->s_dtype));
  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  p.M = static_cast<int32_t>(N);
  p.Ncols = static_cast<int32_t>(K);
  p.tiles_m = static_cast<int32_t>((N + 2 * kTileM - 1) / (2 * kTileM));
  p.tiles_n = static_cast<int32_t>((K + kTileN - 1) / kTileN);
  const int64_t per = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (per * g->groups > (int64_t{1} << 30)) return fail(FORGE_ERR_UNSUPPORTED, "too many weight tiles");
  p.group_tiles = static_cast<int32_t>(per);
  p.num_tiles = p.num_units = p.split_from = static_cast<int32_t>(per * g->groups);
  p.op3d = N % 64 == 0 && K % 64 == 0;
  p.W = state->W; p.s1 = state->s1; p.s2 = state->s2;
  p.s1_scale = state->s1_scale; p.s2_scale = state->s2_scale;
  p.sc = sc;
  p.qblock = qb;
  for (p.qshift = 0; (1 << p.qshift) < qb; ++p.qshift) {}
  p.seed = seed;
  philox_round_keys(seed, p.round_keys);
  p.step = static_cast<uint64_t>(step);
  p.status = d.status;
  p.wait_limit_ns = wait_limit_ns();
  p.skip_loads = skip_loads() ? 1 : 0;
  p.offsets = g->offsets;
  p.groups = g->groups;
  p.tokens = static_cast<int32_t>(T);
  CUtensorMap ma, mb;
  if ((st = ragged_map(&ma, g->dY, N, T, p.op3d != 0)) != FORGE_OK) return st;
  if ((st = ragged_map(&mb, g->X, K, T, p.op3d != 0)) != FORGE_OK) return st;
  CUtensorMap m1 = ma, m2 = ma, mw = ma;
  const CUtensorMapDataType sd = qb != 0 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : sdt == kSBf16 ? kBf16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  const int esize = qb != 0 ? 1 : (sdt == kSBf16 ? 2 : 4);
  const uint32_t cols = qb != 0 ? 64 : 32;
  const CUtensorMapSwizzle sw = esize == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (uses_s1(opt_kind) && (st = expert_map(&m1, state->s1, sd, esize, g, cols, sw)) != FORGE_OK) return st;
  if (uses_s2(opt_kind) && (st = expert_map(&m2, state->s2, sd, esize, g, cols, sw)) != FORGE_OK) return st;
  // weights in the columns of a chunk: 64 (INT8) or 32
  if ((st = expert_map(&mw, state->W, kBf16, 2, g, cols, qb != 0 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B)) != FORGE_OK)
    return st;
  const int pairs = p.num_units < d.num_sms / 2 ? p.num_units : d.num_sms / 2;
  // after dX's kernel (N > 0, T > 0: it was launched) the step may start at once
  if ((e = launch_tc_grouped(group_mode(T, g->groups, sdt), sdt, ma, mb, m1, m2, mw, p, 2 * pairs, s, g->dX != nullptr)) != cudaSuccess)
    return cuda_fail(e, "grouped step launch");
  return FORGE_OK;
}

forge_status_t forge_multi_opt_step(const forge_tensor_t* tensors, int32_t count, int32_t w_dtype,
                                    int32_t g_dtype, int32_t s_dtype, int32_t opt_kind,
                                    const forge_hparams_t* hp, int64_t step, uint64_t seed, void* stream) {
  clear_message();
  forge_status_t st;
  if (count < 0 || (count > 0 && tensors == nullptr))
    return fail(FORGE_ERR_INVALID_ARG, "need count >= 0 and a tensor table (count=%d)", count);
  if (w_dtype != FORGE_W_FP32 && w_dtype != FORGE_W_BF16_SR) return fail(FORGE_ERR_INVALID_ARG, "w_dtype %d", w_dtype);
  if (g_dtype != FORGE_G_FP32 && g_dtype != FORGE_G_BF16) return fail(FORGE_ERR_INVALID_ARG, "g_dtype %d", g_dtype);
  const int qb = qblock_of(s_dtype);
  if (s_dtype != FORGE_STATE_FP32 && s_dtype != FORGE_STATE_BF16 && qb == 0)
    return fail(FORGE_ERR_INVALID_ARG, "s_dtype %d", s_dtype);
  if ((st = check_hp(opt_kind, hp, step)) != FORGE_OK) return st;
  bool any = false;
  for (int32_t i = 0; i < count; ++i) {
    const forge_tensor_t& t = tensors[i];
    if (t.n < 0) return fail(FORGE_ERR_INVALID_ARG, "tensor %d: n = %lld", i, (long long)t.n);
    if (t.n == 0) continue;
    any = true;
    if (t.n > int64_t{kMaxMultiTiles} * kMultiTile)
      return fail(FORGE_ERR_UNSUPPORTED, "tensor %d: n = %lld is past 2^41", i, (long long)t.n);
    if (t.W == nullptr || !aligned16(t.W))
      return fail(FORGE_ERR_INVALID_ARG, "tensor %d: W must be a non-NULL 16-byte aligned device pointer", i);
    if (t.grad != nullptr && !aligned16(t.grad))
      return fail(FORGE_ERR_INVALID_ARG, "tensor %d: grad must be 16-byte aligned", i);
    if (uses_s1(opt_kind) && (t.s1 == nullptr || !aligned16(t.s1) || (qb != 0 && t.s1_scale == nullptr)))
      return fail(FORGE_ERR_INVALID_ARG, "tensor %d: rule %d needs s1 (16-byte aligned; INT8: with s1_scale)", i, opt_kind);
    if (uses_s2(opt_kind) && (t.s2 == nullptr || !aligned16(t.s2) || (qb != 0 && t.s2_scale == nullptr)))
      return fail(FORGE_ERR_INVALID_ARG, "tensor %d: rule %d needs s2 (16-byte aligned; INT8: with s2_scale)", i, opt_kind);
  }
  if (!any) return FORGE_OK;
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  MultiParams<kMultiLong> p;
  p.sc = make_scalars(opt_kind, *hp, step);
  p.seed = seed;
  p.step = static_cast<uint64_t>(step);
  p.qblock = qb;
  p.count = 0;
  uint32_t tiles = 0;
  auto flush = [&]() -> cudaError_t {
    if (p.count == 0) return cudaSuccess;
    const cudaError_t e = launch_multi(w_dtype, base_sdt(s_dtype), g_dtype, p, tiles, static_cast<cudaStream_t>(stream));
    p.count = 0;
    tiles = 0;
    return e;
  };
  cudaError_t e;
  for (int32_t i = 0; i < count; ++i) {
    const forge_tensor_t& t = tensors[i];
    if (t.n == 0) continue;
    const uint32_t mine = static_cast<uint32_t>((t.n + kMultiTile - 1) / kMultiTile);
    if ((p.count == kMultiLong || tiles + mine > kMaxMultiTiles) && (e = flush()) != cudaSuccess)
      return cuda_fail(e, "many-tensor step launch");
    p.items[p.count++] = MultiItem{t.grad, t.W, t.s1, t.s2, t.s1_scale, t.s2_scale, t.n, tiles, static_cast<uint32_t>(i)};
    tiles += mine;
  }
  if ((e = flush()) != cudaSuccess) return cuda_fail(e, "many-tensor step launch");
  return FORGE_OK;
}

forge_status_t forge_rmsnorm_fwd(const forge_rmsnorm_t* n, void* stream) {
  clear_message();
  forge_status_t st;
  if (n == nullptr) return fail(FORGE_ERR_INVALID_ARG, "norm is NULL");
  if ((st = check_norm_shape(n->T, n->K)) != FORGE_OK) return st;
  if (!(n->eps >= 0.f) || !std::isfinite(n->eps)) return fail(FORGE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (n->yt != nullptr) {
    if (n->T % 16 != 0) return fail(FORGE_ERR_INVALID_ARG, "yt needs T %% 16 == 0 (T=%lld)", (long long)n->T);
    if (!(n->yt_scale > 0.f) || !std::isfinite(n->yt_scale) || !std::isfinite(1.f / n->yt_scale))
      return fail(FORGE_ERR_INVALID_ARG, "yt_scale and its reciprocal must be finite and positive");
  }
  if ((n->yq == nullptr) != (n->yq_scale == nullptr))
    return fail(FORGE_ERR_INVALID_ARG, "yq and yq_scale go together");
  if (n->amax != nullptr && n->yt == nullptr && n->T > 0)  // (an empty tensor has no address)
    return fail(FORGE_ERR_INVALID_ARG, "amax is an output of yt");
  if (n->residual != nullptr && n->h == nullptr) return fail(FORGE_ERR_INVALID_ARG, "a residual needs h");
  if (n->T == 0 && n->amax == nullptr) return FORGE_OK;
  if (n->T > 0 && ((st = check_ptr(n->x, "x")) != FORGE_OK || (st = check_ptr(n->w, "w")) != FORGE_OK ||
                   (st = check_ptr(n->residual, "residual", true)) != FORGE_OK ||
                   (st = check_ptr(n->h, "h", true)) != FORGE_OK || (st = check_ptr(n->y, "y", true)) != FORGE_OK ||
                   (st = check_ptr(n->yq, "yq", true)) != FORGE_OK || (st = check_ptr(n->yt, "yt", true)) != FORGE_OK))
    return st;
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n->T == 0) {  // no token: the maximum over nothing
    if ((e = cudaMemsetAsync(n->amax, 0, sizeof(float), s)) != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(amax)");
    return FORGE_OK;
  }
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.x = n->x; p.res = n->residual; p.w = n->w; p.h = n->h; p.rstd = n->rstd; p.y = n->y;
  p.q = n->yq; p.q_scale = n->yq_scale; p.qt = n->yt; p.amax = n->amax;
  p.T = n->T; p.K = static_cast<int32_t>(n->K); p.eps = n->eps;
  p.inv_scale = n->yt != nullptr ? 1.f / n->yt_scale : 1.f;
  p.wait_limit_ns = wait_limit_ns();
  p.status = d.status;
  p.skip_sends = skip_loads() ? 1 : 0;
  // without a residual h is x itself (copied first: y may lie over x)
  if (n->residual == nullptr && n->h != nullptr && n->h != n->x &&
      (e = cudaMemcpyAsync(n->h, n->x, static_cast<size_t>(n->T * n->K * 2), cudaMemcpyDeviceToDevice, s)) != cudaSuccess)
    return cuda_fail(e, "cudaMemcpyAsync(h)");
  if ((e = launch_norm_fwd(p, d.num_sms, s)) != cudaSuccess) return cuda_fail(e, "norm launch");
  return FORGE_OK;
}

int64_t forge_rmsnorm_bwd_workspace(int64_t T, int64_t K) {
  clear_message();
  if (check_norm_shape(T, K) != FORGE_OK) return -1;
  DeviceInfo d;
  if (device_info(&d) != FORGE_OK) return -1;
  return norm_bwd_blocks(T, static_cast<int>(K), d.num_sms) * K;
}

forge_status_t forge_rmsnorm_bwd(const forge_rmsnorm_grad_t* g, void* stream) {
  clear_message();
  forge_status_t st;
  if (g == nullptr) return fail(FORGE_ERR_INVALID_ARG, "grad is NULL");
  if ((st = check_norm_shape(g->T, g->K)) != FORGE_OK) return st;
  if ((st = check_ptr(g->dw, "dw")) != FORGE_OK) return st;
  if (g->T > 0 && ((st = check_ptr(g->dy, "dy")) != FORGE_OK || (st = check_ptr(g->h, "h")) != FORGE_OK ||
                   (st = check_ptr(g->w, "w")) != FORGE_OK || (st = check_ptr(g->dh, "dh", true)) != FORGE_OK ||
                   (st = check_ptr(g->dx, "dx")) != FORGE_OK || (st = check_ptr(g->workspace, "workspace")) != FORGE_OK))
    return st;
  if (g->T > 0 && g->rstd == nullptr) return fail(FORGE_ERR_INVALID_ARG, "rstd is NULL");
  DeviceInfo d;
  if ((st = device_info(&d)) != FORGE_OK) return st;
  if ((st = check_device(d)) != FORGE_OK) return st;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.dy = g->dy; p.x = g->h; p.w = g->w; p.rstd = const_cast<float*>(g->rstd); p.dh = g->dh;
  p.y = g->dx; p.dw = g->dw; p.partial = g->workspace;
  p.T = g->T; p.K = static_cast<int32_t>(g->K);
  const cudaError_t e = launch_norm_bwd(p, d.num_sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "norm gradient launch");
  return FORGE_OK;
}

}  // extern "C"
