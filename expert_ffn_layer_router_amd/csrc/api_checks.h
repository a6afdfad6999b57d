// Argument checks shared by the operators' C entry points.
#pragma once

#include <hip/hip_runtime.h>

#include "products.h"

#define MOE_EXPORT extern "C" __attribute__((visibility("default")))

#define MOE_TRY(call)                       \
  do {                                      \
    const moe_status st_ = (call);          \
    if (st_ != MOE_OK) return st_;          \
  } while (0)

namespace moe {

moe_status api_fail(moe_status st, const char* fmt, ...);

constexpr int kMaxRows = 1 << 22, kMaxWidth = 65536, kMaxGroups = 256;
constexpr int64_t kMaxStride = 1 << 20;

// A row matrix: null allowed only without rows.
inline moe_status check_rows(const char* name, const void* m, int64_t ld, int rows, int width, int unit) {
  if (!m && rows > 0) return api_fail(MOE_ERR_INVALID_ARG, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(m) % 16) return api_fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (ld < width || ld > kMaxStride || ld % unit)
    return api_fail(MOE_ERR_INVALID_ARG, "row stride %lld of %s must be a multiple of %d in [%d, %lld]", (long long)ld,
                    name, unit, width, (long long)kMaxStride);
  return MOE_OK;
}

inline moe_status check_plain(const char* name, const void* m) {
  if (!m) return api_fail(MOE_ERR_INVALID_ARG, "%s is null", name);
  if (reinterpret_cast<uintptr_t>(m) % 16) return api_fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return MOE_OK;
}

inline moe_status check_offsets(const moe_product* p, const int32_t* offsets) {
  if (!offsets && p->groups != 1) return api_fail(MOE_ERR_INVALID_ARG, "offsets is null with %d groups", p->groups);
  if (reinterpret_cast<uintptr_t>(offsets) % 4) return api_fail(MOE_ERR_INVALID_ARG, "offsets is not 4-byte aligned");
  return MOE_OK;
}

inline moe_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (have < need) return api_fail(MOE_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, the call needs %zu", have, need);
  return check_plain("workspace", ws);
}

inline moe_status check_launch() {
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return api_fail(MOE_ERR_HIP, "kernel launch failed: %s", hipGetErrorString(err));
  return MOE_OK;
}

}  // namespace moe
