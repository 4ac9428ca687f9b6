// Checks of arguments shared by the C entry points of the products and the operators beside
// them (host).
#pragma once

#include "common.h"

namespace exmoe {

inline int check_matrix(const char* name, const void* p, size_t ld, int cols, int bytes) {
  if (!p) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if ((uintptr_t)p % (unsigned)bytes) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", name, bytes);
  if (ld < (size_t)cols) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: row stride %zu smaller than its %d columns", name, ld, cols);
  return EXMOE_OK;
}

// (the stride of a single expert means nothing)
inline int check_experts(const char* name, size_t ld, size_t stride, int N, int K, int E) {
  if (E > 1 && stride < (size_t)(N - 1) * ld + K)
    return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s: expert stride %zu smaller than a matrix", name, stride);
  return EXMOE_OK;
}

inline int check_int32(const char* name, const void* p, bool may_be_null) {
  if (!p && !may_be_null) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must not be NULL", name);
  if ((uintptr_t)p % 4) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "%s must be 4-byte aligned", name);
  return EXMOE_OK;
}

inline int check_ws(size_t need, const void* ws, size_t ws_bytes) {
  if (!need) return EXMOE_OK;
  if (!ws || ws_bytes < need)
    return set_error(EXMOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, ws ? ws_bytes : 0);
  if (!aligned16(ws)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "workspace must be 16-byte aligned");
  return EXMOE_OK;
}

inline int launched(hipError_t e, const char* what) { return e == hipSuccess ? EXMOE_OK : hip_error(e, what); }

// Whether rows of outputs can be stored 16 bytes at a time.
inline int vec_store(const void* p, size_t ld, size_t stride, int out_f32) {
  const size_t n = out_f32 ? 4 : 8;
  return aligned16(p) && ld % n == 0 && stride % n == 0;
}

}  // namespace exmoe

#define EXMOE_TRY(call)        \
  do {                         \
    const int st_ = (call);    \
    if (st_) return st_;       \
  } while (0)

#define EXMOE_CALL(call)                                                                    \
  do {                                                                                     \
    if (!(call)) return set_error(EXMOE_ERR_INVALID_ARGUMENT, "call must not be NULL");     \
  } while (0)
