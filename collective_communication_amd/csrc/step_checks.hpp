// step_checks.hpp -- argument checks that the C ABI's files of the operators
// around the gradient exchange share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hc.h"
#include "launch.hpp"

namespace hc {

constexpr size_t kMax31 = ((size_t)1 << 31) - 1;

inline size_t esize(hc_dtype_t d) { return d == HC_F32 ? 4 : 2; }

inline hc_status_t check_dtype(hc_dtype_t d, const char* name) {
  if (d == HC_F32 || d == HC_BF16) return HC_SUCCESS;
  return fail(HC_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", name, (int)d);
}

inline hc_status_t check_ptr(const void* p, size_t align, const char* name) {
  if (!p) return fail(HC_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if ((uintptr_t)p % align) return fail(HC_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", name, align);
  return HC_SUCCESS;
}

inline hc_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (have < need) return fail(HC_ERR_INSUFFICIENT_CAPACITY, "workspace holds %zu bytes, needs %zu", have, need);
  return need ? check_ptr(ws, 16, "ws") : HC_SUCCESS;
}

// A matrix of `rows` rows; `dtype` is checked first.
inline hc_status_t check_rows(const void* p, hc_dtype_t dtype, size_t rows, size_t dim, size_t stride, const char* name) {
  if (hc_status_t st = check_dtype(dtype, name)) return st;
  if (stride < dim) return fail(HC_ERR_INVALID_ARGUMENT, "%s: stride %zu < width %zu", name, stride, dim);
  if (stride > ((size_t)1 << 40)) return fail(HC_ERR_INVALID_ARGUMENT, "%s: stride %zu", name, stride);
  return rows && dim ? check_ptr(p, esize(dtype), name) : HC_SUCCESS;
}

inline hc_status_t check_ids(const void* ids, int id_bytes, size_t n, const char* name) {
  if (id_bytes != 4 && id_bytes != 8)
    return fail(HC_ERR_INVALID_ARGUMENT, "%s: id_bytes %d is neither 4 nor 8", name, id_bytes);
  return n ? check_ptr(ids, (size_t)id_bytes, name) : HC_SUCCESS;
}

inline hc_status_t check_size(size_t v, const char* name) {
  if (v > kMax31) return fail(HC_ERR_INVALID_ARGUMENT, "%s %zu is 2^31 or more", name, v);
  return HC_SUCCESS;
}

#define HC_TRY(expr) \
  do { \
    if (hc_status_t st_ = (expr)) return st_; \
  } while (0)

inline hc_status_t no_memory() { return fail(HC_ERR_DEVICE, "out of host memory"); }

inline hc_status_t done(hipError_t e, const char* where) {
  return e == hipSuccess ? HC_SUCCESS : device_fail(e, where);
}

}  // namespace hc
