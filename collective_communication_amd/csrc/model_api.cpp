// model_api.cpp -- the C ABI of the norm of rows, the routing to experts and
// the optimizer's step: argument checks, then the launches.  Every check runs
// on the host before anything is enqueued; nothing here synchronises or
// allocates device memory.
#include <hip/hip_runtime.h>
#include <math.h>

#include <algorithm>
#include <new>
#include <vector>

#include "hc.h"
#include "launch.hpp"
#include "step_checks.hpp"
#include "step_launch.hpp"

using namespace hc;

namespace {

const char* type_name(hc_dtype_t d) { return d == HC_F32 ? "f32" : "bf16"; }

// ---------------------------------------------------------------- norm of rows

hc_status_t check_norm_sizes(size_t ntokens, size_t dim, float eps) {
  HC_TRY(check_size(ntokens, "ntokens"));
  if (dim < 1 || dim > HC_MAX_NORM_DIM)
    return fail(HC_ERR_INVALID_ARGUMENT, "dim %zu outside 1..%d", dim, HC_MAX_NORM_DIM);
  if (!(eps >= 0.0f) || isinf(eps)) return fail(HC_ERR_INVALID_ARGUMENT, "eps %g", (double)eps);
  return HC_SUCCESS;
}

// Rows that are written where others are read: the same rows, or apart.
hc_status_t check_onto(const void* to, size_t tstride, const void* from, size_t fstride, size_t ntokens,
                       const char* name) {
  if (to == from && to && ntokens > 1 && tstride != fstride)
    return fail(HC_ERR_INVALID_ARGUMENT, "%s: stride %zu on rows of stride %zu", name, tstride, fstride);
  return HC_SUCCESS;
}

hc_status_t check_weight(const void* weight, hc_dtype_t type, const char* name) {
  HC_TRY(check_dtype(type, name));
  return check_ptr(weight, esize(type), name);
}

// What hc_rms_norm and hc_rms_norm_8bit share; out8: rows of bytes.
hc_status_t check_norm(const NormRows& a, bool out8) {
  HC_TRY(check_norm_sizes(a.ntokens, a.dim, a.eps));
  HC_TRY(check_rows(a.x, a.dtype, a.ntokens, a.dim, a.xstride, "x"));
  if (a.residual) HC_TRY(check_rows(a.residual, a.dtype, a.ntokens, a.dim, a.rstride, "residual"));
  if (a.sum) {
    if (!a.residual) return fail(HC_ERR_INVALID_ARGUMENT, "sum_out without a residual");
    HC_TRY(check_rows(a.sum, a.dtype, a.ntokens, a.dim, a.sstride, "sum_out"));
    if (a.ntokens && a.sum == a.out) return fail(HC_ERR_INVALID_ARGUMENT, "sum_out is out");
    HC_TRY(check_onto(a.sum, a.sstride, a.x, a.xstride, a.ntokens, "sum_out"));
    HC_TRY(check_onto(a.sum, a.sstride, a.residual, a.rstride, a.ntokens, "sum_out"));
  }
  HC_TRY(check_weight(a.weight, a.wtype, "weight"));
  if (!out8) {
    HC_TRY(check_rows(a.out, a.dtype, a.ntokens, a.dim, a.ostride, "out"));
    HC_TRY(check_onto(a.out, a.ostride, a.x, a.xstride, a.ntokens, "out"));
    return check_onto(a.out, a.ostride, a.residual, a.rstride, a.ntokens, "out");
  }
  if (a.ntokens && (a.out == a.x || a.out == a.residual || a.out == a.sum))
    return fail(HC_ERR_INVALID_ARGUMENT, "out: rows of 8 bits where other rows are");
  if (a.ostride < a.dim || a.ostride > ((size_t)1 << 40))
    return fail(HC_ERR_INVALID_ARGUMENT, "out: stride %zu, width %zu", a.ostride, a.dim);
  return a.ntokens ? check_ptr(a.out, 1, "out") : HC_SUCCESS;
}

void log_norm(const char* op, const NormRows& a) {
  if (hc::log_enabled())
    hc::log_line("%s: tokens=%zu dim=%zu dtype=%s weight=%s residual=%d", op, a.ntokens, a.dim, type_name(a.dtype),
                 type_name(a.wtype), a.residual != nullptr);
}

// ---------------------------------------------------------------- routing

hc_status_t check_route(size_t ntokens, int nexperts, const hc_route_opts_t* o) {
  if (!o) return fail(HC_ERR_INVALID_ARGUMENT, "opts is NULL");
  if (nexperts < 1 || nexperts > HC_MAX_EXPERTS)
    return fail(HC_ERR_INVALID_ARGUMENT, "nexperts %d outside 1..%d", nexperts, HC_MAX_EXPERTS);
  if (o->k < 1 || o->k > HC_MAX_TOPK) return fail(HC_ERR_INVALID_ARGUMENT, "k %d outside 1..%d", o->k, HC_MAX_TOPK);
  if (ntokens > kMax31 / (size_t)o->k) return fail(HC_ERR_INVALID_ARGUMENT, "ntokens * k is 2^31 or more");
  if (o->scores != HC_SCORES_SOFTMAX && o->scores != HC_SCORES_SIGMOID)
    return fail(HC_ERR_INVALID_ARGUMENT, "unknown scores %d", (int)o->scores);
  if (!isfinite(o->scale)) return fail(HC_ERR_INVALID_ARGUMENT, "scale %g", (double)o->scale);
  return HC_SUCCESS;
}

hc_status_t check_groups(int nexperts, const hc_route_opts_t* o) {
  if (o->ngroups < 1 || o->ngroups > HC_MAX_GROUPS || nexperts % o->ngroups)
    return fail(HC_ERR_INVALID_ARGUMENT, "ngroups %d for %d experts (1..%d, a divisor)", o->ngroups, nexperts,
                HC_MAX_GROUPS);
  if (o->top_groups < 1 || o->top_groups > o->ngroups)
    return fail(HC_ERR_INVALID_ARGUMENT, "top_groups %d outside 1..%d", o->top_groups, o->ngroups);
  if (o->group_best != 1 && o->group_best != 2)
    return fail(HC_ERR_INVALID_ARGUMENT, "group_best %d is neither 1 nor 2", o->group_best);
  if (o->k > o->top_groups * (nexperts / o->ngroups))
    return fail(HC_ERR_INVALID_ARGUMENT, "k %d of %d experts in %d groups", o->k,
                o->top_groups * (nexperts / o->ngroups), o->top_groups);
  if (o->bias) return check_ptr(o->bias, 4, "bias");
  return HC_SUCCESS;
}

void log_route(const char* op, size_t ntokens, int nexperts, const hc_route_opts_t* o, hc_dtype_t dtype) {
  if (hc::log_enabled())
    hc::log_line("%s: tokens=%zu experts=%d k=%d groups=%d of %d scores=%s dtype=%s", op, ntokens, nexperts, o->k,
                 o->top_groups, o->ngroups, o->scores == HC_SCORES_SIGMOID ? "sigmoid" : "softmax", type_name(dtype));
}

// ---------------------------------------------------------------- AdamW

struct Span {
  uintptr_t lo, hi;
  const char* what;
  size_t i;
  bool written;
};

// Whether nothing written overlaps anything else: the spans by address, against
// the furthest ends of the written ones and of all before.
hc_status_t check_spans(std::vector<Span>& s) {
  std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  const Span *written = nullptr, *any = nullptr;
  for (const Span& x : s) {
    const Span* y = written && x.lo < written->hi ? written : x.written && any && x.lo < any->hi ? any : nullptr;
    if (y)
      return fail(HC_ERR_INVALID_ARGUMENT, "%s[%zu] overlaps %s[%zu]", x.what, x.i, y->what, y->i);
    if (x.written && (!written || x.hi > written->hi)) written = &x;
    if (!any || x.hi > any->hi) any = &x;
  }
  return HC_SUCCESS;
}

bool fraction(double b) { return b >= 0.0 && b < 1.0; }

}  // namespace

extern "C" {

hc_status_t hc_rms_norm(const void* x, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t x_stride,
                        const void* residual, size_t residual_stride, const void* weight, hc_dtype_t weight_dtype,
                        float eps, void* sum_out, size_t sum_stride, void* out, size_t out_stride,
                        hipStream_t stream) {
  hc::clear_error();
  const NormRows a = {x,       x_stride,   residual, residual_stride, weight, weight_dtype, sum_out,
                      sum_stride, out, out_stride, dtype, ntokens, dim, eps};
  HC_TRY(check_norm(a, false));
  log_norm("hc_rms_norm", a);
  if (!ntokens) return HC_SUCCESS;
  return done(hc::launch_rms_norm(a, false, 0, nullptr, 0, stream), "norm launch");
}

hc_status_t hc_rms_norm_8bit(const void* x, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t x_stride,
                             const void* residual, size_t residual_stride, const void* weight,
                             hc_dtype_t weight_dtype, float eps, void* sum_out, size_t sum_stride, void* out,
                             size_t out_stride, int group, float* scales, size_t scales_stride, hipStream_t stream) {
  hc::clear_error();
  const NormRows a = {x,       x_stride,   residual, residual_stride, weight, weight_dtype, sum_out,
                      sum_stride, out, out_stride, dtype, ntokens, dim, eps};
  HC_TRY(check_norm(a, true));
  if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
    return fail(HC_ERR_INVALID_ARGUMENT, "group %d is none of 0, 32, 64, 128, 256", group);
  HC_TRY(check_rows(scales, HC_F32, ntokens, group ? (dim + group - 1) / group : 1, scales_stride, "scales"));
  log_norm("hc_rms_norm_8bit", a);
  if (!ntokens) return HC_SUCCESS;
  return done(hc::launch_rms_norm(a, true, (uint32_t)group, scales, scales_stride, stream), "norm launch");
}

size_t hc_rms_norm_grad_workspace_bytes(size_t ntokens, size_t dim) {
  if (ntokens > kMax31 || dim < 1 || dim > HC_MAX_NORM_DIM) return 0;
  return hc::rms_norm_grad_ws_bytes(ntokens, dim);
}

hc_status_t hc_rms_norm_grad(const void* dout, hc_dtype_t dtype, size_t ntokens, size_t dim, size_t dout_stride,
                             const void* h, size_t h_stride, const void* weight, hc_dtype_t weight_dtype, float eps,
                             const void* dsum, size_t dsum_stride, void* dx, size_t dx_stride, void* dweight,
                             hc_dtype_t dweight_dtype, int accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_norm_sizes(ntokens, dim, eps));
  HC_TRY(check_rows(dout, dtype, ntokens, dim, dout_stride, "dout"));
  HC_TRY(check_rows(h, dtype, ntokens, dim, h_stride, "h"));
  HC_TRY(check_weight(weight, weight_dtype, "weight"));
  if (dsum) HC_TRY(check_rows(dsum, dtype, ntokens, dim, dsum_stride, "dsum"));
  HC_TRY(check_rows(dx, dtype, ntokens, dim, dx_stride, "dx"));
  HC_TRY(check_onto(dx, dx_stride, dout, dout_stride, ntokens, "dx"));
  HC_TRY(check_onto(dx, dx_stride, h, h_stride, ntokens, "dx"));
  HC_TRY(check_onto(dx, dx_stride, dsum, dsum_stride, ntokens, "dx"));
  if (dweight) {
    HC_TRY(check_weight(dweight, dweight_dtype, "dweight"));
    HC_TRY(check_ws(ws, ws_bytes, hc::rms_norm_grad_ws_bytes(ntokens, dim)));
  }
  const NormRows a = {h,       h_stride,   dsum, dsum_stride, weight, weight_dtype, nullptr,
                      0, dx, dx_stride, dtype, ntokens, dim, eps};
  log_norm("hc_rms_norm_grad", a);
  if (!ntokens && (!dweight || accumulate)) return HC_SUCCESS;
  return done(hc::launch_rms_norm_grad(a, dout, dout_stride, dweight, dweight_dtype, accumulate != 0, ws, stream),
              "norm gradient launch");
}

hc_status_t hc_route(const void* logits, hc_dtype_t dtype, size_t ntokens, int nexperts, size_t logits_stride,
                     const hc_route_opts_t* opts, int32_t* experts, float* weights, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_route(ntokens, nexperts, opts));
  HC_TRY(check_groups(nexperts, opts));
  HC_TRY(check_rows(logits, dtype, ntokens, (size_t)nexperts, logits_stride, "logits"));
  if (ntokens) {
    HC_TRY(check_ptr(experts, 4, "experts"));
    HC_TRY(check_ptr(weights, 4, "weights"));
  }
  log_route("hc_route", ntokens, nexperts, opts, dtype);
  if (!ntokens) return HC_SUCCESS;
  return done(hc::launch_route(logits, dtype, ntokens, (uint32_t)nexperts, logits_stride, *opts, experts, weights,
                               stream),
              "route launch");
}

hc_status_t hc_route_grad(const void* logits, hc_dtype_t dtype, size_t ntokens, int nexperts, size_t logits_stride,
                          const hc_route_opts_t* opts, const int32_t* experts, const float* dweights, void* dlogits,
                          size_t dlogits_stride, hipStream_t stream) {
  hc::clear_error();
  HC_TRY(check_route(ntokens, nexperts, opts));
  HC_TRY(check_rows(logits, dtype, ntokens, (size_t)nexperts, logits_stride, "logits"));
  HC_TRY(check_rows(dlogits, dtype, ntokens, (size_t)nexperts, dlogits_stride, "dlogits"));
  HC_TRY(check_onto(dlogits, dlogits_stride, logits, logits_stride, ntokens, "dlogits"));
  if (ntokens) {
    HC_TRY(check_ptr(experts, 4, "experts"));
    HC_TRY(check_ptr(dweights, 4, "dweights"));
  }
  hc_route_opts_t o = *opts;
  o.ngroups = o.top_groups = o.group_best = 1;
  o.bias = nullptr;
  log_route("hc_route_grad", ntokens, nexperts, &o, dtype);
  if (!ntokens) return HC_SUCCESS;
  return done(hc::launch_route_grad(logits, dtype, ntokens, (uint32_t)nexperts, logits_stride, o, experts, dweights,
                                    dlogits, dlogits_stride, stream),
              "route gradient launch");
}

size_t hc_adamw_table_bytes(size_t ntensors) {
  return ntensors > ((size_t)1 << 24) ? 0 : std::max<size_t>(16, hc::adamw_table_bytes(ntensors));
}

hc_status_t hc_adamw_plan(hc_adamw_plan_t* plan, void* const* params, const void* const* grads, void* const* exp_avgs,
                          void* const* exp_avg_sqs, float* const* m_scales, float* const* v_scales,
                          void* const* copies, const float* decays, const size_t* counts,
                          const hc_dtype_t* param_dtypes, const hc_dtype_t* grad_dtypes, size_t ntensors,
                          void* d_table, size_t table_bytes, hipStream_t stream) try {
  hc::clear_error();
  if (!plan) return fail(HC_ERR_INVALID_ARGUMENT, "plan is NULL");
  if (ntensors > ((size_t)1 << 24)) return fail(HC_ERR_INVALID_ARGUMENT, "ntensors %zu", ntensors);
  if (ntensors && (!params || !grads || !exp_avgs || !exp_avg_sqs || !counts || !param_dtypes || !grad_dtypes))
    return fail(HC_ERR_INVALID_ARGUMENT, "params, grads, exp_avgs, exp_avg_sqs, counts or a list of dtypes is NULL");
  if (!m_scales != !v_scales) return fail(HC_ERR_INVALID_ARGUMENT, "m_scales and v_scales go together");
  const bool eight = m_scales != nullptr;
  std::vector<AdamWTensor> all;
  std::vector<Span> spans;
  all.reserve(ntensors);
  spans.reserve(ntensors * 7);
  for (size_t i = 0; i < ntensors; ++i) {
    HC_TRY(check_dtype(param_dtypes[i], "params"));
    HC_TRY(check_dtype(grad_dtypes[i], "grads"));
    const size_t n = counts[i];
    if (n >= ((size_t)1 << 44)) return fail(HC_ERR_INVALID_ARGUMENT, "counts[%zu] = %zu", i, n);
    if (decays && !isfinite(decays[i])) return fail(HC_ERR_INVALID_ARGUMENT, "decays[%zu] = %g", i, (double)decays[i]);
    if (!n) continue;
    const AdamWTensor t = {params[i],
                           grads[i],
                           exp_avgs[i],
                           exp_avg_sqs[i],
                           eight ? m_scales[i] : nullptr,
                           eight ? v_scales[i] : nullptr,
                           copies ? copies[i] : nullptr,
                           n,
                           i,
                           decays ? decays[i] : 1.0f,
                           param_dtypes[i],
                           grad_dtypes[i]};
    if (t.copy && t.p_dtype != HC_F32)
      return fail(HC_ERR_INVALID_ARGUMENT, "copies[%zu]: params[%zu] is not fp32", i, i);
    const size_t state = eight ? 1 : 4, scales = (n + HC_STATE_BLOCK - 1) / HC_STATE_BLOCK * 4;
    const struct {
      const void* p;
      size_t bytes, align;
      const char* what;
      bool needed, written;
    } parts[] = {{t.p, n * esize(t.p_dtype), esize(t.p_dtype), "params", true, true},
                 {t.g, n * esize(t.g_dtype), esize(t.g_dtype), "grads", true, false},
                 {t.m, n * state, state, "exp_avgs", true, true},
                 {t.v, n * state, state, "exp_avg_sqs", true, true},
                 {t.ms, scales, 4, "m_scales", eight, true},
                 {t.vs, scales, 4, "v_scales", eight, true},
                 {t.copy, n * 2, 2, "copies", false, true}};
    for (const auto& x : parts) {
      if (!x.p && x.needed) return fail(HC_ERR_INVALID_ARGUMENT, "%s[%zu] is NULL", x.what, i);
      if (!x.p) continue;
      if ((uintptr_t)x.p % x.align)
        return fail(HC_ERR_INVALID_ARGUMENT, "%s[%zu] is not %zu-byte aligned", x.what, i, x.align);
      spans.push_back({(uintptr_t)x.p, (uintptr_t)x.p + x.bytes, x.what, i, x.written});
    }
    all.push_back(t);
  }
  HC_TRY(check_spans(spans));
  HC_TRY(check_ws(d_table, table_bytes, hc_adamw_table_bytes(ntensors)));
  if (hc::log_enabled()) hc::log_line("hc_adamw_plan: tensors=%zu states=%d", ntensors, eight ? 8 : 32);
  plan->state_bits = eight ? 8 : 32;
  return done(hc::launch_adamw_plan(plan, all.data(), all.size(), d_table, stream), "AdamW table launch");
} catch (const std::bad_alloc&) {
  return no_memory();
}

hc_status_t hc_adamw(const hc_adamw_plan_t* plan, const hc_adamw_opts_t* o, hipStream_t stream) {
  hc::clear_error();
  if (!plan) return fail(HC_ERR_INVALID_ARGUMENT, "plan is NULL");
  if (!o) return fail(HC_ERR_INVALID_ARGUMENT, "opts is NULL");
  HC_TRY(check_ptr(plan->d_table, 16, "plan: d_table"));
  if ((plan->state_bits != 8 && plan->state_bits != 32) || plan->chunks > 0xFFFFFFFFull ||
      plan->ntensors > ((size_t)1 << 24) || (plan->chunks != 0) != (plan->ntensors != 0))
    return fail(HC_ERR_INVALID_ARGUMENT, "plan: not one that hc_adamw_plan filled in");
  if (!o->d_step && o->step < 1) return fail(HC_ERR_INVALID_ARGUMENT, "step %lld < 1", (long long)o->step);
  if (!fraction(o->beta1) || !fraction(o->beta2))
    return fail(HC_ERR_INVALID_ARGUMENT, "betas %g, %g outside [0, 1)", o->beta1, o->beta2);
  if (!(o->eps >= 0.0) || !isfinite((float)o->eps)) return fail(HC_ERR_INVALID_ARGUMENT, "eps %g", o->eps);
  if (!isfinite((float)o->lr) || !isfinite((float)o->weight_decay) || !isfinite(o->grad_scale))
    return fail(HC_ERR_INVALID_ARGUMENT, "lr %g, weight_decay %g or grad_scale %g", o->lr, o->weight_decay,
                (double)o->grad_scale);
  if (o->d_norm) {
    HC_TRY(check_ptr(o->d_norm, 4, "d_norm"));
    if (!(o->max_norm >= 0.0f))
      return fail(HC_ERR_INVALID_ARGUMENT, "max_norm %g is negative or no number", (double)o->max_norm);
  }
  if (o->d_lr) HC_TRY(check_ptr(o->d_lr, 4, "d_lr"));
  if (o->d_step) HC_TRY(check_ptr(o->d_step, 8, "d_step"));
  if (hc::log_enabled())
    hc::log_line("hc_adamw: tensors=%zu chunks=%llu states=%d step=%lld", plan->ntensors,
                 (unsigned long long)plan->chunks, plan->state_bits, (long long)o->step);
  return done(hc::launch_adamw(*plan, *o, stream), "AdamW launch");
}

}  // extern "C"
