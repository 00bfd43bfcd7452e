// What the entry points share: statuses with a message, and the checks of pointers and workspaces.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "sbp.h"
#include "sbp_internal.cuh"

namespace sbp {

inline sbp_status fail(sbp_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

// returns from an entry point where a CUDA call failed
#define SBP_CK(expr)                                                                 \
  do {                                                                               \
    cudaError_t e_ = (expr);                                                         \
    if (e_ != cudaSuccess)                                                           \
      return fail(SBP_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString(e_));     \
  } while (0)

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

inline sbp_status check_ws(void* ws, size_t have, size_t need) {
  if (!ws) return fail(SBP_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SBP_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  if (have < need)
    return fail(SBP_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
  return SBP_OK;
}

}  // namespace sbp
