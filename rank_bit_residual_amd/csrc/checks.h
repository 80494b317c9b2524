// Argument checks shared by the C ABI of the tensor calls (svdq_mx_*, svdq_i8_*, svdq_layer_norm*).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "svdq_internal.h"

namespace svdq {

constexpr int64_t kMaxMxDim = (int64_t)1 << 30;

inline int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return SVDQ_OK;
  if (e == hipErrorInvalidConfiguration) return set_error(SVDQ_EINVAL, std::string(what) + ": more threads than a launch holds");
  return set_error(SVDQ_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }
inline int64_t size_of(int dtype) { return dtype == SVDQ_F32 ? 4 : 2; }

inline int check_mx_dtype(int dtype) {
  if (dtype != SVDQ_F32 && dtype != SVDQ_BF16 && dtype != SVDQ_F16)
    return set_error(SVDQ_EDTYPE, "dtype must be SVDQ_F32, SVDQ_BF16 or SVDQ_F16");
  return SVDQ_OK;
}

// Common start of a device call: a clean error state and a dtype these calls take.
inline int begin(int dtype) {
  clear_error();
  (void)hipGetLastError();  // an error that an earlier, unrelated HIP call left
  return check_mx_dtype(dtype);
}

inline int check_dim(int64_t v, const char* name) {
  if (v < 1 || v > kMaxMxDim) return set_error(SVDQ_EINVAL, std::string(name) + " must be in [1, 2^30]");
  return SVDQ_OK;
}

inline int check_tensor(const void* codes, const void* scales, const char* name) {
  if (!codes || !scales) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (!aligned(codes, kAlign) || !aligned(scales, kAlign))
    return set_error(SVDQ_EINVAL, std::string(name) + ": codes and scales must be 256-byte aligned");
  return SVDQ_OK;
}

// An output pair that may be left out as a whole.
inline int check_out(const void* codes, const void* scales, const char* name) {
  if (!codes && !scales) return SVDQ_OK;
  return check_tensor(codes, scales, name);
}

inline int check_matrix(const void* p, int64_t ld, int64_t cols, int dtype, const char* name) {
  if (!p) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (ld < cols) return set_error(SVDQ_EINVAL, std::string(name) + ": row stride smaller than the row");
  if (!aligned(p, size_of(dtype))) return set_error(SVDQ_EINVAL, std::string(name) + " misaligned");
  return SVDQ_OK;
}

inline int check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need || !aligned(ws, kAlign)))
    return set_error(SVDQ_EINVAL, "workspace too small or not 256-byte aligned");
  return SVDQ_OK;
}

inline int check_strided(const void* x, int64_t sr, int64_t sc, int dtype, const char* name) {
  if (!x) return set_error(SVDQ_EINVAL, std::string(name) + ": NULL buffer");
  if (!aligned(x, size_of(dtype))) return set_error(SVDQ_EINVAL, std::string(name) + " misaligned");
  if (sr < 0 || sc < 0) return set_error(SVDQ_EINVAL, "strides must not be negative");
  return SVDQ_OK;
}

// For calls of several launches, before the first.
inline int check_grid(bool fits, const char* what) {
  return fits ? SVDQ_OK : hip_status(hipErrorInvalidConfiguration, what);
}

}  // namespace svdq
