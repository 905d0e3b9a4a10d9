// C ABI of the operators around the linear step (declared in include/forge.h):
// the many-tensor optimizer step and the norm.  Argument checks and launches;
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

}  // namespace

extern "C" {

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
  if ((e = launch_norm_fwd(p, d.num_sms, s)) != cudaSuccess) return cuda_fail(e, "norm launch");
  // without a residual h is x itself
  if (n->residual == nullptr && n->h != nullptr && n->h != n->x &&
      (e = cudaMemcpyAsync(n->h, n->x, static_cast<size_t>(n->T * n->K * 2), cudaMemcpyDeviceToDevice, s)) != cudaSuccess)
    return cuda_fail(e, "cudaMemcpyAsync(h)");
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
