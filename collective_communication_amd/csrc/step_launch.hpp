// step_launch.hpp -- internal launch interface of the operators around the
// gradient exchange: gradient norm and clipping, embedding lookup and
// gradient, the norm of rows, routing, tokens sorted by expert and back, and
// the optimizer's step.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "hc.h"

namespace hc {

// Enqueues a kernel and returns that launch's own status: not whatever error
// an earlier call of the process may have left behind.  The arguments are
// converted to the kernel's parameter types.
// lds: bytes of shared memory beside the kernel's own.
template <typename... P, typename... A>
inline hipError_t enqueue_lds(uint32_t lds, void (*kernel)(P...), uint32_t grid, uint32_t block, hipStream_t stream,
                              const A&... args) {
  static_assert(sizeof...(P) == sizeof...(A), "one argument per parameter");
  return [&](const P&... p) {
    const void* at[] = {static_cast<const void*>(&p)...};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(block),
                                         const_cast<void**>(at), lds, stream);
    if (e != hipSuccess) (void)hipGetLastError();   // reported here, so not once more by the next reader
    return e;
  }(args...);
}
template <typename... P, typename... A>
inline hipError_t enqueue(void (*kernel)(P...), uint32_t grid, uint32_t block, hipStream_t stream, const A&... args) {
  return enqueue_lds(0, kernel, grid, block, stream, args...);
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

// ---- norm of rows (norm_kernels.hip)
// Pointers with their strides; residual is the gradient that arrives at h, x is
// h and out is dx for the gradient.
struct NormRows {
  const void* x;
  size_t xstride;
  const void* residual;
  size_t rstride;
  const void* weight;
  hc_dtype_t wtype;
  void* sum;
  size_t sstride;
  void* out;
  size_t ostride;
  hc_dtype_t dtype;
  size_t ntokens, dim;
  float eps;
};
// group: columns per scale, 0 for the whole row.
hipError_t launch_rms_norm(const NormRows& a, bool q8, uint32_t group, float* scales, size_t cstride,
                           hipStream_t stream);
size_t rms_norm_grad_ws_bytes(size_t ntokens, size_t dim);
hipError_t launch_rms_norm_grad(const NormRows& a, const void* dout, size_t dstride, void* dweight, hc_dtype_t dwtype,
                                bool accumulate, void* ws, hipStream_t stream);

// ---- routing (route_kernels.hip)
hipError_t launch_route(const void* logits, hc_dtype_t dtype, size_t ntokens, uint32_t nexperts, size_t lstride,
                        const hc_route_opts_t& o, int32_t* experts, float* weights, hipStream_t stream);
hipError_t launch_route_grad(const void* logits, hc_dtype_t dtype, size_t ntokens, uint32_t nexperts, size_t lstride,
                             const hc_route_opts_t& o, const int32_t* experts, const float* dweights, void* dlogits,
                             size_t dstride, hipStream_t stream);

// ---- AdamW (adamw_kernels.hip)
struct AdamWTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;         // NULL: states of 32 bits
  float* vs;
  void* copy;
  size_t count, index;
  float decay;
  hc_dtype_t p_dtype, g_dtype;
};
size_t adamw_table_bytes(size_t ntensors);
// Writes the table and all of *plan but state_bits.
hipError_t launch_adamw_plan(hc_adamw_plan_t* plan, const AdamWTensor* tensors, size_t n, void* table,
                             hipStream_t stream);
hipError_t launch_adamw(const hc_adamw_plan_t& plan, const hc_adamw_opts_t& o, hipStream_t stream);

}  // namespace hc
