// api_checks.h -- argument checks that the operators' entry points share.
#pragma once
#include <hip/hip_runtime_api.h>

#include "internal.h"

namespace sshdp {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? SSHDP_OK : SSHDP_ERR_HIP; }

// Whether a kernel on the current device may be given `p`: the device's own
// memory, or host memory the runtime allocated (NULL passes: optional tensors).
inline bool on_device(int cur, const void *p) {
  if (!p) return true;
  hipPointerAttribute_t a{};
  if (hipPointerGetAttributes(&a, p) != hipSuccess) {
    (void)hipGetLastError();                         // an address the runtime does not know
    return false;
  }
  if (a.type == hipMemoryTypeDevice) return a.device == cur;
  return a.type == hipMemoryTypeHost || a.type == hipMemoryTypeManaged;
}

template <class... P>
int check_device(const P *...p) {
  int cur = -1;
  if (hipGetDevice(&cur) != hipSuccess) return SSHDP_ERR_HIP;
  return (on_device(cur, p) && ...) ? SSHDP_OK : SSHDP_ERR_ARG;
}

inline bool dtype_ok(int32_t d) { return d == SSHDP_DTYPE_FP32 || d == SSHDP_DTYPE_BF16; }

inline int64_t dtype_size(int32_t d) { return d == SSHDP_DTYPE_BF16 ? 2 : 4; }

// A norm's weight, or its gradient: at any element of its array.
inline bool aligned_element(const void *p, int32_t d) { return reinterpret_cast<uintptr_t>(p) % dtype_size(d) == 0; }

inline int check_ws(const void *ws, size_t bytes, int64_t need) {
  if (need == 0) return SSHDP_OK;
  if (!ws || bytes < (size_t)need) return SSHDP_ERR_WORKSPACE;
  if (!aligned16(ws)) return SSHDP_ERR_ALIGN;
  return check_device(ws);
}

constexpr int64_t kMaxEdge = 1ll << 30;              // rows and columns of a matrix
// Region rules of a matrix (those of a plan's MXFP8 region at offset 0), codes and
// scales present unless it is empty.
inline int check_matrix(const sshdp_mx_matrix *m) {
  if (!m || m->rows < 0 || m->cols < 0) return SSHDP_ERR_ARG;
  if (m->layout != SSHDP_SCALE_ROWMAJOR && m->layout != SSHDP_SCALE_TILE32X4 && m->layout != SSHDP_SCALE_BLOCK32X32)
    return SSHDP_ERR_ARG;
  if (m->rows && m->cols && (!m->codes || !m->scales)) return SSHDP_ERR_ARG;
  if (m->cols % 32 || m->rows > kMaxEdge || m->cols > kMaxEdge) return SSHDP_ERR_SCHEMA;
  if (m->layout == SSHDP_SCALE_TILE32X4 && (m->rows % 32 || m->cols % 128)) return SSHDP_ERR_SCHEMA;
  if (m->layout == SSHDP_SCALE_BLOCK32X32 && m->rows % 32) return SSHDP_ERR_SCHEMA;
  return SSHDP_OK;
}

}  // namespace sshdp
