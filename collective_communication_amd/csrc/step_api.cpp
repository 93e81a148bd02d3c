// step_api.cpp -- the C ABI of the operators around the gradient exchange:
// argument checks, then the launches.  Every check runs on the host before
// anything is enqueued; nothing here synchronises or allocates device memory.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "hc.h"
#include "launch.hpp"
#include "step_launch.hpp"

namespace {

using hc::device_fail;
using hc::fail;

constexpr size_t kMax31 = ((size_t)1 << 31) - 1;

size_t esize(hc_dtype_t d) { return d == HC_F32 ? 4 : 2; }

hc_status_t check_dtype(hc_dtype_t d, const char* name) {
  if (d == HC_F32 || d == HC_BF16) return HC_SUCCESS;
  return fail(HC_ERR_INVALID_ARGUMENT, "%s: unknown dtype %d", name, (int)d);
}

hc_status_t check_ptr(const void* p, size_t align, const char* name) {
  if (!p) return fail(HC_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if ((uintptr_t)p % align) return fail(HC_ERR_INVALID_ARGUMENT, "%s is not %zu-byte aligned", name, align);
  return HC_SUCCESS;
}

hc_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (have < need) return fail(HC_ERR_INSUFFICIENT_CAPACITY, "workspace holds %zu bytes, needs %zu", have, need);
  return need ? check_ptr(ws, 16, "ws") : HC_SUCCESS;
}

// A matrix of `rows` rows; `dtype` is checked first.
hc_status_t check_rows(const void* p, hc_dtype_t dtype, size_t rows, size_t dim, size_t stride, const char* name) {
  if (hc_status_t st = check_dtype(dtype, name)) return st;
  if (stride < dim) return fail(HC_ERR_INVALID_ARGUMENT, "%s: stride %zu < width %zu", name, stride, dim);
  if (stride > ((size_t)1 << 40)) return fail(HC_ERR_INVALID_ARGUMENT, "%s: stride %zu", name, stride);
  return rows && dim ? check_ptr(p, esize(dtype), name) : HC_SUCCESS;
}

hc_status_t check_ids(const void* ids, int id_bytes, size_t n, const char* name) {
  if (id_bytes != 4 && id_bytes != 8)
    return fail(HC_ERR_INVALID_ARGUMENT, "%s: id_bytes %d is neither 4 nor 8", name, id_bytes);
  return n ? check_ptr(ids, (size_t)id_bytes, name) : HC_SUCCESS;
}

hc_status_t check_size(size_t v, const char* name) {
  if (v > kMax31) return fail(HC_ERR_INVALID_ARGUMENT, "%s %zu is 2^31 or more", name, v);
  return HC_SUCCESS;
}

#define HC_TRY(expr) \
  do { \
    if (hc_status_t st_ = (expr)) return st_; \
  } while (0)

// ---------------------------------------------------------------- gradients

hc_status_t check_tensors(const void* const* grads, const size_t* counts, const hc_dtype_t* dtypes, size_t n) {
  if (n > ((size_t)1 << 24)) return fail(HC_ERR_INVALID_ARGUMENT, "ntensors %zu", n);
  if (!n) return HC_SUCCESS;
  if (!grads || !counts || !dtypes) return fail(HC_ERR_INVALID_ARGUMENT, "grads, counts or dtypes is NULL");
  for (size_t i = 0; i < n; ++i) {
    if (dtypes[i] != HC_F32 && dtypes[i] != HC_BF16)
      return fail(HC_ERR_INVALID_ARGUMENT, "dtypes[%zu]: unknown dtype %d", i, (int)dtypes[i]);
    if (counts[i] >= ((size_t)1 << 47)) return fail(HC_ERR_INVALID_ARGUMENT, "counts[%zu] = %zu", i, counts[i]);
    if (!counts[i]) continue;
    if (!grads[i]) return fail(HC_ERR_INVALID_ARGUMENT, "grads[%zu] is NULL", i);
    if ((uintptr_t)grads[i] % esize(dtypes[i]))
      return fail(HC_ERR_INVALID_ARGUMENT, "grads[%zu] is not %zu-byte aligned", i, esize(dtypes[i]));
  }
  return HC_SUCCESS;
}

struct Range {
  uintptr_t lo, hi;
  size_t i;
  bool out;
};

// Whether the outputs, in their order, ascend without touching (the views of
// one bucket do), with every gradient but an output's own outside their span:
// then nothing overlaps, found without sorting.
bool plainly_disjoint(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                      size_t n) {
  uintptr_t first = 0, end = 0;
  for (size_t i = 0; i < n; ++i) {
    if (!counts[i]) continue;
    const uintptr_t o = (uintptr_t)outs[i];
    if (o < end) return false;
    if (!first) first = o;
    end = o + counts[i] * esize(dtypes[i]);
  }
  for (size_t i = 0; i < n; ++i) {
    const uintptr_t g = (uintptr_t)grads[i];
    if (counts[i] && grads[i] != outs[i] && g < end && g + counts[i] * esize(dtypes[i]) > first) return false;
  }
  return true;
}

// Outputs must be disjoint from one another and from every gradient but their
// own.  Else one sort by address: an output overlaps something when it begins
// before the furthest end so far, or when something begins before its end.
hc_status_t check_outs(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                       size_t n) {
  if (!n) return HC_SUCCESS;
  if (!outs) return fail(HC_ERR_INVALID_ARGUMENT, "outs is NULL");
  for (size_t i = 0; i < n; ++i) {
    if (!counts[i]) continue;
    if (!outs[i]) return fail(HC_ERR_INVALID_ARGUMENT, "outs[%zu] is NULL", i);
    if ((uintptr_t)outs[i] % esize(dtypes[i]))
      return fail(HC_ERR_INVALID_ARGUMENT, "outs[%zu] is not %zu-byte aligned", i, esize(dtypes[i]));
  }
  if (plainly_disjoint(grads, outs, counts, dtypes, n)) return HC_SUCCESS;
  std::vector<Range> r;
  r.reserve(2 * n);
  for (size_t i = 0; i < n; ++i) {
    if (!counts[i]) continue;
    const size_t bytes = counts[i] * esize(dtypes[i]);
    const uintptr_t o = (uintptr_t)outs[i], g = (uintptr_t)grads[i];
    r.push_back({o, o + bytes, i, true});
    if (o != g) r.push_back({g, g + bytes, i, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  // the furthest ends of the outputs and of all ranges that began so far
  uintptr_t out_end = 0, any_end = 0;
  size_t out_i = 0, any_i = 0;
  for (const Range& x : r) {
    if (x.lo < out_end)
      return fail(HC_ERR_INVALID_ARGUMENT, "outs[%zu] overlaps %s[%zu]", out_i, x.out ? "outs" : "grads", x.i);
    if (x.out && x.lo < any_end)
      return fail(HC_ERR_INVALID_ARGUMENT, "outs[%zu] overlaps grads[%zu]", x.i, any_i);
    if (x.out && x.hi > out_end) out_end = x.hi, out_i = x.i;
    if (x.hi > any_end) any_end = x.hi, any_i = x.i;
  }
  return HC_SUCCESS;
}

hc_status_t check_max_norm(float m) {
  if (m >= 0.0f) return HC_SUCCESS;
  return fail(HC_ERR_INVALID_ARGUMENT, "max_norm %g is negative or no number", (double)m);
}

hc_status_t check_norm_kind(hc_norm_t k) {
  if (k == HC_NORM_L2 || k == HC_NORM_INF) return HC_SUCCESS;
  return fail(HC_ERR_INVALID_ARGUMENT, "unknown norm %d", (int)k);
}

hc_status_t no_memory() { return fail(HC_ERR_DEVICE, "out of host memory"); }

// ---------------------------------------------------------------- experts

hc_status_t check_plan_sizes(size_t ntokens, int k, int nexperts, int row_align) {
  if (k < 1 || k > HC_MAX_TOPK) return fail(HC_ERR_INVALID_ARGUMENT, "k %d outside 1..%d", k, HC_MAX_TOPK);
  if (nexperts < 1 || nexperts > HC_MAX_EXPERTS)
    return fail(HC_ERR_INVALID_ARGUMENT, "nexperts %d outside 1..%d", nexperts, HC_MAX_EXPERTS);
  if (row_align < 1) return fail(HC_ERR_INVALID_ARGUMENT, "row_align %d < 1", row_align);
  if (ntokens > kMax31 / (size_t)k) return fail(HC_ERR_INVALID_ARGUMENT, "ntokens * k is 2^31 or more");
  const size_t n = ntokens * (size_t)k;
  if (n + std::min<size_t>(nexperts, n) * (size_t)(row_align - 1) > kMax31)
    return fail(HC_ERR_INVALID_ARGUMENT, "the rows of all experts are 2^31 or more");
  return HC_SUCCESS;
}

hc_status_t check_plan(const hc_expert_plan_t* p) {
  if (!p) return fail(HC_ERR_INVALID_ARGUMENT, "plan is NULL");
  HC_TRY(check_plan_sizes(p->ntokens, p->k, p->nexperts, p->row_align));
  HC_TRY(check_size(p->rows, "plan: rows"));
  const size_t need = hc_expert_rows_bound(p->ntokens, p->k, p->nexperts, p->row_align);
  if (p->rows < need)
    return fail(HC_ERR_INSUFFICIENT_CAPACITY, "plan: room for %zu rows, needs %zu", p->rows, need);
  if (p->ntokens) HC_TRY(check_ptr(p->row_of_slot, 4, "plan: row_of_slot"));
  if (p->rows) HC_TRY(check_ptr(p->slot_of_row, 4, "plan: slot_of_row"));
  HC_TRY(check_ptr(p->expert_offsets, 4, "plan: expert_offsets"));
  return check_ptr(p->expert_counts, 4, "plan: expert_counts");
}

void log_plan(const char* op, const hc_expert_plan_t* p, size_t dim, hc_dtype_t dtype) {
  if (!hc::log_enabled()) return;
  hc::log_line("%s: tokens=%zu k=%d experts=%d align=%d rows=%zu dim=%zu dtype=%s", op, p->ntokens, p->k, p->nexperts,
               p->row_align, p->rows, dim, dtype == HC_F32 ? "f32" : "bf16");
}

hc_status_t done(hipError_t e, const char* where) {
  return e == hipSuccess ? HC_SUCCESS : device_fail(e, where);
}

}  // namespace

extern "C" {

size_t hc_grad_norm_workspace_bytes(size_t ntensors) { return hc::grad_norm_ws_bytes(ntensors); }

hc_status_t hc_grad_norm(const void* const* grads, const size_t* counts, const hc_dtype_t* dtypes, size_t ntensors,
                         hc_norm_t norm, float* d_norm, void* ws, size_t ws_bytes, hipStream_t stream) try {
  hc::clear_error();
  HC_TRY(check_norm_kind(norm));
  HC_TRY(check_tensors(grads, counts, dtypes, ntensors));
  HC_TRY(check_ptr(d_norm, 4, "d_norm"));
  HC_TRY(check_ws(ws, ws_bytes, hc::grad_norm_ws_bytes(ntensors)));
  if (hc::log_enabled()) hc::log_line("hc_grad_norm: tensors=%zu", ntensors);
  return done(hc::launch_grad_norm(grads, nullptr, counts, dtypes, ntensors, norm, 0.0f, d_norm, ws, stream),
              "gradient norm launch");
} catch (const std::bad_alloc&) {
  return no_memory();
}

hc_status_t hc_clip_grads(const void* const* grads, void* const* outs, const size_t* counts, const hc_dtype_t* dtypes,
                          size_t ntensors, const float* d_norm, float max_norm, void* ws, size_t ws_bytes,
                          hipStream_t stream) try {
  hc::clear_error();
  HC_TRY(check_tensors(grads, counts, dtypes, ntensors));
  HC_TRY(check_outs(grads, outs, counts, dtypes, ntensors));
  HC_TRY(check_max_norm(max_norm));
  HC_TRY(check_ptr(d_norm, 4, "d_norm"));
  HC_TRY(check_ws(ws, ws_bytes, hc::grad_norm_ws_bytes(ntensors)));
  if (hc::log_enabled()) hc::log_line("hc_clip_grads: tensors=%zu max_norm=%g", ntensors, (double)max_norm);
  return done(hc::launch_grad_clip(grads, outs, counts, dtypes, ntensors, max_norm, d_norm, ws, stream),
              "gradient clipping launch");
} catch (const std::bad_alloc&) {
  return no_memory();
}

hc_status_t hc_clip_grad_norm(const void* const* grads, void* const* outs, const size_t* counts,
                              const hc_dtype_t* dtypes, size_t ntensors, hc_norm_t norm, float max_norm, float* d_norm,
                              void* ws, size_t ws_bytes, hipStream_t stream) try {
  hc::clear_error();
  HC_TRY(check_norm_kind(norm));
  HC_TRY(check_tensors(grads, counts, dtypes, ntensors));
  HC_TRY(check_outs(grads, outs, counts, dtypes, ntensors));
  HC_TRY(check_max_norm(max_norm));
  HC_TRY(check_ptr(d_norm, 4, "d_norm"));
  HC_TRY(check_ws(ws, ws_bytes, hc::grad_norm_ws_bytes(ntensors)));
  if (hc::log_enabled()) hc::log_line("hc_clip_grad_norm: tensors=%zu max_norm=%g", ntensors, (double)max_norm);
  return done(hc::launch_grad_norm(grads, outs, counts, dtypes, ntensors, norm, max_norm, d_norm, ws, stream),
              "gradient clipping launch");
} catch (const std::bad_alloc&) {
  return no_memory();
}

hc_status_t hc_embedding(const void* ids, int id_bytes, size_t ntokens, const void* weight, hc_dtype_t dtype,
                         size_t vocab, size_t dim, size_t weight_stride, int64_t vocab_start, float scale, void* out,
                         size_t out_stride, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_size(ntokens, "ntokens"));
  HC_TRY(check_size(vocab, "vocab"));
  HC_TRY(check_size(dim, "dim"));
  HC_TRY(check_ids(ids, id_bytes, ntokens, "ids"));
  HC_TRY(check_rows(weight, dtype, vocab, dim, weight_stride, "weight"));
  HC_TRY(check_rows(out, dtype, ntokens, dim, out_stride, "out"));
  if (hc::log_enabled())
    hc::log_line("hc_embedding: tokens=%zu vocab=%zu dim=%zu dtype=%s", ntokens, vocab, dim,
                 dtype == HC_F32 ? "f32" : "bf16");
  if (!ntokens || !dim) return HC_SUCCESS;
  const hc::KeySource src = {ids, id_bytes, vocab_start, (uint32_t)vocab, 0, 0};
  return done(hc::launch_embedding(src, ntokens, weight, dtype, dim, weight_stride, scale, out, out_stride, stream),
              "embedding launch");
}

size_t hc_embedding_grad_workspace_bytes(size_t ntokens, size_t vocab, size_t dim) {
  if (ntokens > kMax31 || vocab > kMax31 || dim > kMax31) return 0;
  return hc::embedding_grad_ws_bytes(ntokens, dim);
}

hc_status_t hc_embedding_grad(const void* ids, int id_bytes, size_t ntokens, const void* dout, hc_dtype_t dout_dtype,
                              size_t dout_stride, size_t vocab, size_t dim, int64_t vocab_start, int64_t padding_id,
                              float scale, void* dweight, hc_dtype_t dweight_dtype, size_t dweight_stride,
                              int accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_size(ntokens, "ntokens"));
  HC_TRY(check_size(vocab, "vocab"));
  HC_TRY(check_size(dim, "dim"));
  HC_TRY(check_ids(ids, id_bytes, ntokens, "ids"));
  HC_TRY(check_rows(dout, dout_dtype, ntokens, dim, dout_stride, "dout"));
  HC_TRY(check_rows(dweight, dweight_dtype, vocab, dim, dweight_stride, "dweight"));
  HC_TRY(check_ws(ws, ws_bytes, hc::embedding_grad_ws_bytes(ntokens, dim)));
  if (hc::log_enabled())
    hc::log_line("hc_embedding_grad: tokens=%zu vocab=%zu dim=%zu dtypes=%s,%s accumulate=%d", ntokens, vocab, dim,
                 dout_dtype == HC_F32 ? "f32" : "bf16", dweight_dtype == HC_F32 ? "f32" : "bf16", accumulate != 0);
  if (!vocab || !dim || (accumulate && !ntokens)) return HC_SUCCESS;
  const hc::KeySource src = {ids, id_bytes, vocab_start, (uint32_t)vocab, padding_id, padding_id >= 0};
  return done(hc::launch_embedding_grad(src, ntokens, dout, dout_dtype, dim, dout_stride, scale, dweight,
                                        dweight_dtype, dweight_stride, accumulate != 0, ws, stream),
              "embedding gradient launch");
}

size_t hc_expert_rows_bound(size_t ntokens, int k, int nexperts, int row_align) {
  if (k < 1 || k > HC_MAX_TOPK || nexperts < 1 || nexperts > HC_MAX_EXPERTS || row_align < 1 ||
      ntokens > kMax31 / (size_t)k)
    return 0;
  const size_t n = ntokens * (size_t)k;
  return n + std::min<size_t>(nexperts, n) * (size_t)(row_align - 1);
}

size_t hc_expert_sort_workspace_bytes(size_t nslots, int nexperts) {
  if (nslots > kMax31 || nexperts < 1 || nexperts > HC_MAX_EXPERTS) return 0;
  return hc::expert_sort_ws_bytes(nslots, (size_t)nexperts);
}

hc_status_t hc_expert_sort(const void* experts, int id_bytes, int64_t expert_start, const hc_expert_plan_t* plan,
                           void* ws, size_t ws_bytes, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_plan(plan));
  const size_t n = plan->ntokens * (size_t)plan->k;
  HC_TRY(check_ids(experts, id_bytes, n, "experts"));
  HC_TRY(check_ws(ws, ws_bytes, hc::expert_sort_ws_bytes(n, (size_t)plan->nexperts)));
  log_plan("hc_expert_sort", plan, 0, HC_F32);
  const hc::KeySource src = {experts, id_bytes, expert_start, (uint32_t)plan->nexperts, 0, 0};
  return done(hc::launch_expert_sort(src, *plan, ws, stream), "expert sort launch");
}

hc_status_t hc_expert_dispatch(const void* x, hc_dtype_t dtype, size_t dim, size_t x_stride,
                               const hc_expert_plan_t* plan, void* rows, size_t rows_stride, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_plan(plan));
  HC_TRY(check_size(dim, "dim"));
  HC_TRY(check_rows(x, dtype, plan->ntokens, dim, x_stride, "x"));
  HC_TRY(check_rows(rows, dtype, plan->rows, dim, rows_stride, "rows"));
  log_plan("hc_expert_dispatch", plan, dim, dtype);
  if (!dim) return HC_SUCCESS;
  return done(hc::launch_expert_dispatch(x, dtype, dim, x_stride, *plan, rows, rows_stride, stream),
              "expert dispatch launch");
}

hc_status_t hc_expert_combine(const void* rows, hc_dtype_t dtype, size_t dim, size_t rows_stride,
                              const hc_expert_plan_t* plan, const float* weights, void* out, size_t out_stride,
                              hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_plan(plan));
  HC_TRY(check_size(dim, "dim"));
  HC_TRY(check_rows(rows, dtype, plan->rows, dim, rows_stride, "rows"));
  HC_TRY(check_rows(out, dtype, plan->ntokens, dim, out_stride, "out"));
  if (weights) HC_TRY(check_ptr(weights, 4, "weights"));
  log_plan("hc_expert_combine", plan, dim, dtype);
  if (!dim) return HC_SUCCESS;
  return done(hc::launch_expert_combine(rows, dtype, dim, rows_stride, *plan, weights, out, out_stride, stream),
              "expert combine launch");
}

hc_status_t hc_expert_combine_grad(const void* dout, hc_dtype_t dtype, size_t dim, size_t dout_stride,
                                   const void* rows, size_t rows_stride, const hc_expert_plan_t* plan,
                                   const float* weights, void* drows, size_t drows_stride, float* dweights,
                                   hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_plan(plan));
  HC_TRY(check_size(dim, "dim"));
  HC_TRY(check_rows(dout, dtype, plan->ntokens, dim, dout_stride, "dout"));
  HC_TRY(check_rows(rows, dtype, plan->rows, dim, rows_stride, "rows"));
  HC_TRY(check_rows(drows, dtype, plan->rows, dim, drows_stride, "drows"));
  if (plan->ntokens) {
    HC_TRY(check_ptr(weights, 4, "weights"));
    HC_TRY(check_ptr(dweights, 4, "dweights"));
  }
  log_plan("hc_expert_combine_grad", plan, dim, dtype);
  return done(hc::launch_expert_combine_grad(dout, dtype, dim, dout_stride, rows, rows_stride, *plan, weights, drows,
                                             drows_stride, dweights, stream),
              "expert combine gradient launch");
}

}  // extern "C"
