// step_launch.hpp -- internal launch interface of the operators around the
// gradient exchange: gradient norm and clipping, embedding lookup and
// gradient, tokens sorted by expert and back.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hc.h"

namespace hc {

// Enqueues a kernel and returns that launch's own status: not whatever error
// an earlier call of the process may have left behind.  The arguments are
// converted to the kernel's parameter types.
template <typename... P, typename... A>
inline hipError_t enqueue(void (*kernel)(P...), uint32_t grid, uint32_t block, hipStream_t stream, const A&... args) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument per parameter");
  return [&](const P&... p) {
    const void* at[] = {static_cast<const void*>(&p)...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(block),
                                         const_cast<void**>(at), 0, stream);
    if (e != hipSuccess) (void)hipGetLastError();   // reported here, so not once more by the next reader
    return e;
  }(args...);
}
#define HC_ENQUEUE(kernel, ...) \
  do { \
    if (hipError_t e_ = ::hc::enqueue(kernel, __VA_ARGS__); e_ != hipSuccess) return e_; \
  } while (0)

// ---- gradient norm and clipping (grad_kernels.hip)
size_t grad_norm_ws_bytes(size_t ntensors);
// norm of all tensors into *d_norm; when outs is not NULL, also outs[i] =
// coef * grads[i] with coef = min(1, max_norm / (norm + 1e-6)).
hipError_t launch_grad_norm(const void* const* grads, void* const* outs, const size_t* counts,
                            const hc_dtype_t* dtypes, size_t ntensors, hc_norm_t kind, float max_norm, float* d_norm,
                            void* ws, hipStream_t stream);
// The scaling alone, by the norm in *d_norm.
hipError_t launch_grad_clip(const void* const* grads, void* const* outs, const size_t* counts,
                            const hc_dtype_t* dtypes, size_t ntensors, float max_norm, const float* d_norm, void* ws,
                            hipStream_t stream);

// ---- keys (key_sort.hpp)
// Small integer keys made from 32- or 64-bit ids: id - start where that lies
// in [0, nkeys) and the id is not `skip`; any other id has no key.
struct KeySource {
  const void* ids;
  int id_bytes;
  int64_t start;
  uint32_t nkeys;
  int64_t skip;     // an id without a key, where use_skip is set
  int use_skip;
};
constexpr uint32_t kNoKey = 0xFFFFFFFFu;

// ---- embedding (embed_kernels.hip)
hipError_t launch_embedding(const KeySource& src, size_t ntokens, const void* weight, hc_dtype_t dtype, size_t dim,
                            size_t wstride, float scale, void* out, size_t ostride, hipStream_t stream);
size_t embedding_grad_ws_bytes(size_t ntokens, size_t dim);   // of any number of table rows
hipError_t launch_embedding_grad(const KeySource& src, size_t ntokens, const void* dout, hc_dtype_t dtype, size_t dim,
                                 size_t dstride, float scale, void* dweight, hc_dtype_t dwtype, size_t wstride,
                                 bool accumulate, void* ws, hipStream_t stream);

// ---- experts (expert_kernels.hip)
size_t expert_sort_ws_bytes(size_t nslots, size_t nexperts);
hipError_t launch_expert_sort(const KeySource& src, const hc_expert_plan_t& plan, void* ws, hipStream_t stream);
hipError_t launch_expert_dispatch(const void* x, hc_dtype_t dtype, size_t dim, size_t xstride,
                                  const hc_expert_plan_t& plan, void* rows, size_t rstride, hipStream_t stream);
hipError_t launch_expert_combine(const void* rows, hc_dtype_t dtype, size_t dim, size_t rstride,
                                 const hc_expert_plan_t& plan, const float* weights, void* out, size_t ostride,
                                 hipStream_t stream);
hipError_t launch_expert_combine_grad(const void* dout, hc_dtype_t dtype, size_t dim, size_t dstride,
                                      const void* rows, size_t rstride, const hc_expert_plan_t& plan,
                                      const float* weights, void* drows, size_t drstride, float* dweights,
                                      hipStream_t stream);

}  // namespace hc
