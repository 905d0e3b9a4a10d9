// Host-side helpers shared by the translation units that hold the C ABI
// (api.cu, ops_api.cu): error reporting, per-device facts, tensor maps and the
// argument checks every optimizer entry point makes.  Defined in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "common.h"
#include "forge.h"

namespace forge {

// The calling thread's message (forge_last_error_message): cleared at the
// start of every entry point, set by fail, which returns `st`.
void clear_message();
forge_status_t fail(forge_status_t st, const char* fmt, ...);
forge_status_t cuda_fail(cudaError_t e, const char* what);

struct DeviceInfo {
  int num_sms = 0;
  uint32_t* status = nullptr;
  uint32_t* dx_done = nullptr;
  uint32_t* static_scratch = nullptr;  // g_static_scratch on this device
  int step_pairs[kNumKernelSdt] = {};  // resident one-launch-step pairs, by kernel state dtype
  int cc_major = 0, cc_minor = 0;
};
forge_status_t device_info(DeviceInfo* out);
forge_status_t check_device(const DeviceInfo& d);

uint64_t wait_limit_ns();
int skip_loads();

forge_status_t tensor_map(CUtensorMap* m, const void* base, CUtensorMapDataType dtype, int esize,
                          int64_t inner, int64_t outer, uint32_t box_inner, uint32_t box_outer,
                          CUtensorMapSwizzle swizzle);
forge_status_t tensor_map_nd(CUtensorMap* m, const void* base, CUtensorMapDataType dtype, int rank,
                             const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                             CUtensorMapSwizzle swizzle);

int qblock_of(int32_t s_dtype);
int base_sdt(int32_t s_dtype);
void philox_round_keys(uint64_t seed, uint32_t* rk);
OptScalars make_scalars(int kind, const forge_hparams_t& hp, int64_t step);
bool aligned16(const void* p);
forge_status_t check_state(const forge_state_t* st, int kind, int64_t N, int64_t K);
forge_status_t check_hp(int32_t kind, const forge_hparams_t* hp, int64_t step);

}  // namespace forge
