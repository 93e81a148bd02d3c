// native_binding.cpp -- the module `_native`: torch tensors marshalled to the
// C ABI for the operators around the gradient exchange.
//
// These calls take hundreds of small tensors (a model's gradients) or run for
// a few microseconds (a decoding step's tokens), where reading tensors'
// attributes from Python costs more than the kernels: 290 gradients and their
// outputs took 240 us from Python and take 8 us here.  Each function checks
// the tensors, calls the C function of the same name and returns its status;
// binding.py turns a status into HcError.  A wrong type is TypeError, any
// other unfit tensor ValueError, as in the rest of the binding.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cstdarg>
#include <stdexcept>
#include <string>
#include <vector>

#include "hc.h"

namespace {

struct PyError {};    // a Python exception is set

[[noreturn]] void raise(PyObject* type, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(type, fmt, ap);
  va_end(ap);
  throw PyError{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

hc_dtype_t dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return HC_F32;
  if (t.scalar_type() == at::kBFloat16) return HC_BF16;
  raise(PyExc_TypeError, "unsupported dtype %s (float32 or bfloat16)", c10::toString(t.scalar_type()));
}

// A contiguous device tensor of at least `need` elements.
void* flat(PyObject* o, size_t need, const char* name, size_t* bytes = nullptr) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda() || !t.is_contiguous()) raise(PyExc_ValueError, "%s must be a contiguous device tensor", name);
  if ((size_t)t.numel() < need)
    raise(PyExc_ValueError, "%s holds %zd elements, needs %zu", name, (Py_ssize_t)t.numel(), need);
  if (bytes) *bytes = t.nbytes();
  return t.data_ptr();
}

float* flat_f32(PyObject* o, size_t need, const char* name) {
  if (tensor(o, name).scalar_type() != at::kFloat) raise(PyExc_TypeError, "%s must be float32", name);
  return static_cast<float*>(flat(o, need, name));
}

struct Ids {
  const void* p;
  int bytes;
  size_t n;
};
Ids ids_of(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != at::kInt && t.scalar_type() != at::kLong)
    raise(PyExc_TypeError, "%s must be int32 or int64", name);
  return Ids{flat(o, 0, name), t.scalar_type() == at::kInt ? 4 : 8, (size_t)t.numel()};
}

// A 2-D device tensor whose rows are dense and do not overlap.
struct Matrix {
  void* p;
  size_t rows, dim, stride;
  hc_dtype_t dtype;
};
Matrix matrix(PyObject* o, const char* name) {
  const at::Tensor& t = tensor(o, name);
  const hc_dtype_t dt = dtype_of(t);
  if (t.dim() != 2 || !t.is_cuda()) raise(PyExc_ValueError, "%s must be a 2-D device tensor", name);
  const int64_t rows = t.size(0), dim = t.size(1);
  const int64_t stride = rows > 1 ? t.stride(0) : dim;
  if ((dim > 1 && t.stride(1) != 1) || stride < dim)
    raise(PyExc_ValueError, "%s needs dense rows that do not overlap (strides %zd, %zd)", name, (Py_ssize_t)t.stride(0),
          (Py_ssize_t)t.stride(1));
  return Matrix{t.data_ptr(), (size_t)rows, (size_t)dim, (size_t)stride, dt};
}
void fits(const Matrix& m, size_t rows, size_t dim, const char* name) {
  if (m.rows < rows || m.dim != dim)
    raise(PyExc_ValueError, "%s is (%zu, %zu), needs (%zu, %zu)", name, m.rows, m.dim, rows, dim);
}
void same_dtype(PyObject* a, PyObject* b) {
  if (dtype_of(tensor(a, "rows")) != dtype_of(tensor(b, "rows"))) raise(PyExc_TypeError, "all rows need one dtype");
}

hipStream_t stream_of(PyObject* o) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream().stream();
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw PyError{};
  return static_cast<hipStream_t>(p);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return v;
}
const hc_expert_plan_t* plan_of(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "plan is NULL");
    throw PyError{};
  }
  return static_cast<const hc_expert_plan_t*>(p);
}

// Many tensors' addresses, counts and dtypes.  A norm and a scaling go over a
// tensor's storage, so any order of dimensions will do, but no gaps.
struct Tensors {
  std::vector<const void*> p;
  std::vector<size_t> counts;
  std::vector<hc_dtype_t> dtypes;
};
struct Sequence {
  PyObject* o;
  explicit Sequence(PyObject* x, const char* name) : o(PySequence_Fast(x, name)) {
    if (!o) throw PyError{};
  }
  ~Sequence() { Py_DECREF(o); }
  size_t size() const { return (size_t)PySequence_Fast_GET_SIZE(o); }
  PyObject* operator[](size_t i) const { return PySequence_Fast_GET_ITEM(o, (Py_ssize_t)i); }
};

// Whether the elements fill their storage, once each, in any order.
bool dense(const at::Tensor& t) { return t.is_non_overlapping_and_dense(); }

Tensors tensors(const Sequence& s) {
  Tensors r;
  const size_t n = s.size();
  r.p.reserve(n);
  r.counts.reserve(n);
  r.dtypes.reserve(n);
  for (size_t i = 0; i < n; ++i) {
    const at::Tensor& t = tensor(s[i], "a gradient");
    r.dtypes.push_back(dtype_of(t));
    if (!dense(t)) raise(PyExc_ValueError, "grads[%zu] is not dense: its storage has gaps", i);
    if (!t.is_cuda()) raise(PyExc_ValueError, "grads[%zu] is not a device tensor", i);
    r.p.push_back(t.data_ptr());
    r.counts.push_back((size_t)t.numel());
  }
  return r;
}

// The outputs' addresses; None: the gradients themselves.
std::vector<void*> outputs(PyObject* o, const Sequence& grads, const Tensors& g) {
  std::vector<void*> p;
  const size_t n = grads.size();
  p.reserve(n);
  if (o == Py_None) {
    for (const void* x : g.p) p.push_back(const_cast<void*>(x));
    return p;
  }
  const Sequence outs(o, "outs must be a sequence of tensors");
  if (outs.size() != n) raise(PyExc_ValueError, "one output per gradient");
  for (size_t i = 0; i < n; ++i) {
    const at::Tensor &x = tensor(grads[i], "a gradient"), &y = tensor(outs[i], "an output");
    if (!y.is_cuda() || y.scalar_type() != x.scalar_type() || y.sizes() != x.sizes() || y.strides() != x.strides())
      raise(PyExc_ValueError, "outs[%zu] must have the device, dtype, shape and strides of grads[%zu]", i, i);
    p.push_back(y.data_ptr());
  }
  return p;
}

typedef PyObject* const* Args;

hc_status_t grad_norm(Args a) {   // grads, d_norm, ws, kind, stream
  const Sequence s(a[0], "grads must be a sequence of tensors");
  const Tensors g = tensors(s);
  size_t room;
  void* ws = flat(a[2], 0, "ws", &room);
  return hc_grad_norm(g.p.data(), g.counts.data(), g.dtypes.data(), s.size(), (hc_norm_t)integer(a[3]),
                      flat_f32(a[1], 1, "d_norm"), ws, room, stream_of(a[4]));
}

hc_status_t clip_grads(Args a) {  // grads, outs, d_norm, max_norm, ws, stream
  const Sequence s(a[0], "grads must be a sequence of tensors");
  const Tensors g = tensors(s);
  const std::vector<void*> o = outputs(a[1], s, g);
  size_t room;
  void* ws = flat(a[4], 0, "ws", &room);
  return hc_clip_grads(g.p.data(), o.data(), g.counts.data(), g.dtypes.data(), s.size(), flat_f32(a[2], 1, "d_norm"),
                       (float)number(a[3]), ws, room, stream_of(a[5]));
}

hc_status_t clip_grad_norm(Args a) {  // grads, outs, kind, max_norm, d_norm, ws, stream
  const Sequence s(a[0], "grads must be a sequence of tensors");
  const Tensors g = tensors(s);
  const std::vector<void*> o = outputs(a[1], s, g);
  size_t room;
  void* ws = flat(a[5], 0, "ws", &room);
  return hc_clip_grad_norm(g.p.data(), o.data(), g.counts.data(), g.dtypes.data(), s.size(),
                           (hc_norm_t)integer(a[2]), (float)number(a[3]), flat_f32(a[4], 1, "d_norm"), ws, room,
                           stream_of(a[6]));
}

hc_status_t embedding(Args a) {   // ids, weight, out, vocab_start, scale, stream
  same_dtype(a[1], a[2]);
  const Ids i = ids_of(a[0], "ids");
  const Matrix w = matrix(a[1], "weight"), o = matrix(a[2], "out");
  fits(o, i.n, w.dim, "out");
  return hc_embedding(i.p, i.bytes, i.n, w.p, w.dtype, w.rows, w.dim, w.stride, integer(a[3]), (float)number(a[4]),
                      o.p, o.stride, stream_of(a[5]));
}

hc_status_t embedding_grad(Args a) {  // ids, dout, dweight, ws, vocab_start, padding_id, scale, accumulate, stream
  const Ids i = ids_of(a[0], "ids");
  const Matrix d = matrix(a[1], "dout"), w = matrix(a[2], "dweight");
  fits(d, i.n, w.dim, "dout");
  size_t room;
  void* ws = flat(a[3], 0, "ws", &room);
  return hc_embedding_grad(i.p, i.bytes, i.n, d.p, d.dtype, d.stride, w.rows, w.dim, integer(a[4]), integer(a[5]),
                           (float)number(a[6]), w.p, w.dtype, w.stride, (int)integer(a[7]), ws, room, stream_of(a[8]));
}

hc_status_t expert_sort(Args a) {     // experts, plan, ws, expert_start, stream
  const Ids i = ids_of(a[0], "experts");
  const hc_expert_plan_t* p = plan_of(a[1]);
  if (i.n != p->ntokens * (size_t)p->k)
    raise(PyExc_ValueError, "experts holds %zu ids, the plan %zu x %d", i.n, p->ntokens, (int)p->k);
  size_t room = 0;
  void* ws = a[2] == Py_None ? nullptr : flat(a[2], 0, "ws", &room);
  return hc_expert_sort(i.p, i.bytes, integer(a[3]), p, ws, room, stream_of(a[4]));
}

hc_status_t expert_dispatch(Args a) {  // x, plan, rows, stream
  const hc_expert_plan_t* p = plan_of(a[1]);
  same_dtype(a[0], a[2]);
  const Matrix x = matrix(a[0], "x"), r = matrix(a[2], "rows");
  fits(x, p->ntokens, x.dim, "x");
  fits(r, p->rows, x.dim, "rows");
  return hc_expert_dispatch(x.p, x.dtype, x.dim, x.stride, p, r.p, r.stride, stream_of(a[3]));
}

hc_status_t expert_combine(Args a) {   // rows, plan, weights, out, stream
  const hc_expert_plan_t* p = plan_of(a[1]);
  same_dtype(a[0], a[3]);
  const Matrix r = matrix(a[0], "rows"), o = matrix(a[3], "out");
  fits(r, p->rows, r.dim, "rows");
  fits(o, p->ntokens, r.dim, "out");
  const float* w = a[2] == Py_None ? nullptr : flat_f32(a[2], p->ntokens * (size_t)p->k, "weights");
  return hc_expert_combine(r.p, r.dtype, r.dim, r.stride, p, w, o.p, o.stride, stream_of(a[4]));
}

hc_status_t expert_combine_grad(Args a) {  // dout, rows, plan, weights, drows, dweights, stream
  const hc_expert_plan_t* p = plan_of(a[2]);
  same_dtype(a[0], a[1]);
  same_dtype(a[0], a[4]);
  const Matrix d = matrix(a[0], "dout"), r = matrix(a[1], "rows"), g = matrix(a[4], "drows");
  fits(d, p->ntokens, r.dim, "dout");
  fits(r, p->rows, r.dim, "rows");
  fits(g, p->rows, r.dim, "drows");
  const size_t n = p->ntokens * (size_t)p->k;
  const float* w = flat_f32(a[3], n, "weights");
  return hc_expert_combine_grad(d.p, d.dtype, d.dim, d.stride, r.p, r.stride, p, w, g.p, g.stride,
                                flat_f32(a[5], n, "dweights"), stream_of(a[6]));
}

// The device that a call's tensors have to be on: the current one, which its
// launches go to.
void here(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be a device tensor", name);
  if (t.get_device() != c10::hip::current_device())
    raise(PyExc_ValueError, "%s is on device %d, the current one is %d", name, (int)t.get_device(),
          (int)c10::hip::current_device());
}
Matrix matrix_here(PyObject* o, const char* name) {
  const Matrix m = matrix(o, name);
  here(tensor(o, name), name);
  return m;
}
// None: none, as rows of width dim.
Matrix maybe_matrix(PyObject* o, const Matrix& like, const char* name) {
  if (o == Py_None) return Matrix{nullptr, 0, like.dim, like.dim, like.dtype};
  const Matrix m = matrix_here(o, name);
  if (m.dtype != like.dtype) raise(PyExc_TypeError, "%s must have the rows' dtype", name);
  fits(m, like.rows, like.dim, name);
  return m;
}
// Rows of the first one's number and width, and dtype.
Matrix same_rows(PyObject* o, const Matrix& like, const char* name) {
  if (o == Py_None) raise(PyExc_TypeError, "%s must be a tensor", name);
  return maybe_matrix(o, like, name);
}

struct Vector {
  void* p;
  hc_dtype_t dtype;
};
Vector vector_here(PyObject* o, size_t need, const char* name) {
  const at::Tensor& t = tensor(o, name);
  const Vector v = {flat(o, need, name), dtype_of(t)};
  here(t, name);
  return v;
}
float* f32_here(PyObject* o, size_t need, const char* name) {
  float* p = flat_f32(o, need, name);
  here(tensor(o, name), name);
  return p;
}
bool is_codes(const at::Tensor& t) { return t.scalar_type() == at::kFloat8_e4m3fn || t.scalar_type() == at::kByte; }

hc_status_t rms_norm(Args a) {  // x, weight, out, residual, sum_out, eps, stream
  const Matrix x = matrix_here(a[0], "x"), o = same_rows(a[2], x, "out");
  const Matrix r = maybe_matrix(a[3], x, "residual"), s = maybe_matrix(a[4], x, "sum_out");
  const Vector w = vector_here(a[1], x.dim, "weight");
  return hc_rms_norm(x.p, x.dtype, x.rows, x.dim, x.stride, r.p, r.stride, w.p, w.dtype, (float)number(a[5]), s.p,
                     s.stride, o.p, o.stride, stream_of(a[6]));
}

hc_status_t rms_norm_8bit(Args a) {  // x, weight, out, scales, group, residual, sum_out, eps, stream
  const Matrix x = matrix_here(a[0], "x");
  const at::Tensor& o = tensor(a[2], "out");
  if (!is_codes(o)) raise(PyExc_TypeError, "out must be float8_e4m3fn or uint8");
  here(o, "out");
  const size_t ostride = o.dim() == 2 && o.size(0) > 1 ? (size_t)o.stride(0) : x.dim;
  if (o.dim() != 2 || (size_t)o.size(0) < x.rows || (size_t)o.size(1) != x.dim || (x.dim > 1 && o.stride(1) != 1) ||
      ostride < x.dim)
    raise(PyExc_ValueError, "out must be (%zu, %zu) with dense rows that do not overlap", x.rows, x.dim);
  const Matrix r = maybe_matrix(a[5], x, "residual"), s = maybe_matrix(a[6], x, "sum_out");
  const Vector w = vector_here(a[1], x.dim, "weight");
  const int64_t group = integer(a[4]);
  if (group < 0 || group > 1 << 20) raise(PyExc_ValueError, "group %zd", (Py_ssize_t)group);
  const Matrix c = matrix_here(a[3], "scales");
  if (c.dtype != HC_F32) raise(PyExc_TypeError, "scales must be float32");
  fits(c, x.rows, group ? (x.dim + group - 1) / group : 1, "scales");
  return hc_rms_norm_8bit(x.p, x.dtype, x.rows, x.dim, x.stride, r.p, r.stride, w.p, w.dtype, (float)number(a[7]),
                          s.p, s.stride, o.data_ptr(), ostride, (int)group, static_cast<float*>(c.p), c.stride,
                          stream_of(a[8]));
}

hc_status_t rms_norm_grad(Args a) {  // dout, h, weight, dx, dweight, ws, dsum, eps, accumulate, stream
  const Matrix h = matrix_here(a[1], "h"), d = same_rows(a[0], h, "dout"), x = same_rows(a[3], h, "dx");
  const Matrix s = maybe_matrix(a[6], h, "dsum");
  const Vector w = vector_here(a[2], h.dim, "weight");
  Vector dw = {nullptr, HC_F32};
  size_t room = 0;
  void* ws = nullptr;
  if (a[4] != Py_None) dw = vector_here(a[4], h.dim, "dweight");
  if (a[5] != Py_None) {
    ws = flat(a[5], 0, "ws", &room);
    here(tensor(a[5], "ws"), "ws");
  }
  return hc_rms_norm_grad(d.p, d.dtype, h.rows, h.dim, d.stride, h.p, h.stride, w.p, w.dtype, (float)number(a[7]),
                          s.p, s.stride, x.p, x.stride, dw.p, dw.dtype, (int)integer(a[8]), ws, room,
                          stream_of(a[9]));
}

// (rows, k) contiguous, of int32 (experts) or fp32 (weights).
void* choices(PyObject* o, const Matrix& logits, bool ids, int32_t* k, const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != (ids ? at::kInt : at::kFloat))
    raise(PyExc_TypeError, "%s must be %s", name, ids ? "int32" : "float32");
  if (t.dim() != 2 || (size_t)t.size(0) != logits.rows || !t.is_contiguous() || (!ids && t.size(1) != *k))
    raise(PyExc_ValueError, "%s must be a contiguous (%zu, k) tensor", name, logits.rows);
  here(t, name);
  if (t.size(1) > HC_MAX_TOPK) raise(PyExc_ValueError, "%s: k %zd is more than %d", name, (Py_ssize_t)t.size(1), HC_MAX_TOPK);
  *k = (int32_t)t.size(1);
  return t.data_ptr();
}
int experts_of(const Matrix& logits) {
  if (logits.dim > HC_MAX_EXPERTS) raise(PyExc_ValueError, "%zu experts are more than %d", logits.dim, HC_MAX_EXPERTS);
  return (int)logits.dim;
}
int32_t small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int32_t)v) raise(PyExc_ValueError, "%s %zd", name, (Py_ssize_t)v);
  return (int32_t)v;
}

hc_status_t route(Args a) {  // logits, experts, weights, scores, bias, groups, top, best, renormalise, scale, stream
  const Matrix x = matrix_here(a[0], "logits");
  const int n = experts_of(x);
  hc_route_opts_t o = {};
  void* experts = choices(a[1], x, true, &o.k, "experts");
  void* weights = choices(a[2], x, false, &o.k, "weights");
  o.scores = (hc_scores_t)small(a[3], "scores");
  o.bias = a[4] == Py_None ? nullptr : f32_here(a[4], x.dim, "bias");
  o.ngroups = small(a[5], "groups");
  o.top_groups = small(a[6], "top_groups");
  o.group_best = small(a[7], "group_best");
  o.renormalise = (int32_t)integer(a[8]);
  o.scale = (float)number(a[9]);
  return hc_route(x.p, x.dtype, x.rows, n, x.stride, &o, static_cast<int32_t*>(experts), static_cast<float*>(weights),
                  stream_of(a[10]));
}

hc_status_t route_grad(Args a) {  // logits, experts, dweights, dlogits, scores, renormalise, scale, stream
  const Matrix x = matrix_here(a[0], "logits"), d = same_rows(a[3], x, "dlogits");
  const int n = experts_of(x);
  hc_route_opts_t o = {};
  const void* experts = choices(a[1], x, true, &o.k, "experts");
  const void* dweights = choices(a[2], x, false, &o.k, "dweights");
  o.scores = (hc_scores_t)small(a[4], "scores");
  o.renormalise = (int32_t)integer(a[5]);
  o.scale = (float)number(a[6]);
  return hc_route_grad(x.p, x.dtype, x.rows, n, x.stride, &o, static_cast<const int32_t*>(experts),
                       static_cast<const float*>(dweights), d.p, d.stride, stream_of(a[7]));
}

// Whether two tensors' elements lie in the same order.
bool same_layout(const at::Tensor& a, const at::Tensor& b) {
  if (a.sizes() != b.sizes()) return false;
  for (int64_t d = 0; d < a.dim(); ++d)
    if (a.size(d) > 1 && a.stride(d) != b.stride(d)) return false;
  return true;
}

// A list of tensors with a parameter's layout each; None entries are NULL where
// `optional`.
template <typename Fits>
std::vector<void*> list_like(const Sequence& params, PyObject* o, const char* name, bool optional, Fits type_fits) {
  const Sequence s(o, name);
  if (s.size() != params.size()) raise(PyExc_ValueError, "%s: one per parameter", name);
  std::vector<void*> p;
  p.reserve(s.size());
  for (size_t i = 0; i < s.size(); ++i) {
    if (optional && s[i] == Py_None) {
      p.push_back(nullptr);
      continue;
    }
    const at::Tensor& t = tensor(s[i], name);
    if (!type_fits(t)) raise(PyExc_TypeError, "%s[%zu]: unsupported dtype %s", name, i, c10::toString(t.scalar_type()));
    if (!same_layout(tensor(params[i], "a parameter"), t))
      raise(PyExc_ValueError, "%s[%zu] must have the shape and strides of params[%zu]", name, i, i);
    here(t, name);
    p.push_back(t.data_ptr());
  }
  return p;
}

std::vector<float*> scales_list(PyObject* o, const std::vector<size_t>& counts, const char* name) {
  const Sequence s(o, name);
  if (s.size() != counts.size()) raise(PyExc_ValueError, "%s: one per parameter", name);
  std::vector<float*> p;
  p.reserve(counts.size());
  for (size_t i = 0; i < counts.size(); ++i)
    p.push_back(f32_here(s[i], (counts[i] + HC_STATE_BLOCK - 1) / HC_STATE_BLOCK, name));
  return p;
}

// plan, params, grads, exp_avgs, exp_avg_sqs, m_scales, v_scales, copies, decays, table, stream
hc_status_t adamw_plan(Args a) {
  hc_adamw_plan_t* plan = static_cast<hc_adamw_plan_t*>(PyLong_AsVoidPtr(a[0]));
  if (!plan) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "plan is NULL");
    throw PyError{};
  }
  const Sequence ps(a[1], "params must be a sequence of tensors");
  const size_t n = ps.size();
  std::vector<void*> params;
  std::vector<size_t> counts;
  std::vector<hc_dtype_t> ptypes, gtypes;
  for (size_t i = 0; i < n; ++i) {
    const at::Tensor& t = tensor(ps[i], "a parameter");
    ptypes.push_back(dtype_of(t));
    if (!dense(t)) raise(PyExc_ValueError, "params[%zu] is not dense: its storage has gaps", i);
    here(t, "params");
    params.push_back(t.data_ptr());
    counts.push_back((size_t)t.numel());
  }
  const std::vector<void*> grads = list_like(ps, a[2], "grads", false, [&](const at::Tensor& t) {
    gtypes.push_back(dtype_of(t));
    return true;
  });
  if ((a[5] == Py_None) != (a[6] == Py_None)) raise(PyExc_ValueError, "m_scales and v_scales go together");
  const bool eight = a[5] != Py_None;
  auto state = [&](const at::Tensor& t) { return eight ? is_codes(t) : t.scalar_type() == at::kFloat; };
  const std::vector<void*> m = list_like(ps, a[3], "exp_avgs", false, state);
  const std::vector<void*> v = list_like(ps, a[4], "exp_avg_sqs", false, state);
  std::vector<float*> ms, vs;
  if (eight) {
    ms = scales_list(a[5], counts, "m_scales");
    vs = scales_list(a[6], counts, "v_scales");
    if (ms.empty()) ms.push_back(nullptr), vs.push_back(nullptr);    // a list all the same
  }
  std::vector<void*> copies;
  if (a[7] != Py_None)
    copies = list_like(ps, a[7], "copies", true, [](const at::Tensor& t) { return t.scalar_type() == at::kBFloat16; });
  std::vector<float> decays;
  if (a[8] != Py_None) {
    const Sequence d(a[8], "decays must be a sequence of numbers");
    if (d.size() != n) raise(PyExc_ValueError, "decays: one per parameter");
    for (size_t i = 0; i < n; ++i) decays.push_back((float)number(d[i]));
  }
  size_t room;
  void* table = flat(a[9], 0, "table", &room);
  here(tensor(a[9], "table"), "table");
  std::vector<const void*> g(grads.begin(), grads.end());
  return hc_adamw_plan(plan, params.data(), g.data(), m.data(), v.data(), eight ? ms.data() : nullptr,
                       eight ? vs.data() : nullptr, copies.empty() ? nullptr : copies.data(),
                       decays.empty() ? nullptr : decays.data(), counts.data(), ptypes.data(), gtypes.data(), n, table,
                       room, stream_of(a[10]));
}

// A scalar on the device, or NULL for None.
const void* scalar(PyObject* o, at::ScalarType type, const char* name) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type) raise(PyExc_TypeError, "%s must be %s", name, c10::toString(type));
  here(t, name);
  return flat(o, 1, name);
}

// plan, table, step, lr, beta1, beta2, eps, weight_decay, grad_scale, d_norm, max_norm, seed, skip_nonfinite, stream
// (step and lr: numbers or device scalars)
hc_status_t adamw(Args a) {
  const hc_adamw_plan_t* plan = static_cast<const hc_adamw_plan_t*>(PyLong_AsVoidPtr(a[0]));
  if (!plan && PyErr_Occurred()) throw PyError{};
  here(tensor(a[1], "table"), "the plan");
  hc_adamw_opts_t o = {};
  if (THPVariable_Check(a[2]))
    o.d_step = static_cast<const int64_t*>(scalar(a[2], at::kLong, "step"));
  else
    o.step = integer(a[2]);
  if (THPVariable_Check(a[3]))
    o.d_lr = static_cast<const float*>(scalar(a[3], at::kFloat, "lr"));
  else
    o.lr = number(a[3]);
  o.beta1 = number(a[4]);
  o.beta2 = number(a[5]);
  o.eps = number(a[6]);
  o.weight_decay = number(a[7]);
  o.grad_scale = (float)number(a[8]);
  o.d_norm = static_cast<const float*>(scalar(a[9], at::kFloat, "d_norm"));
  o.max_norm = (float)number(a[10]);
  o.seed = PyLong_AsUnsignedLongLong(a[11]);
  if (o.seed == ~0ull && PyErr_Occurred()) throw PyError{};
  o.skip_nonfinite = integer(a[12]) != 0;
  return hc_adamw(plan, &o, stream_of(a[13]));
}

// Runs one of the functions above: its status as an int, or a Python error.
template <hc_status_t (*Fn)(Args), Py_ssize_t N>
PyObject* call(PyObject*, Args args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", n, N);
    return nullptr;
  }
  try {
    return PyLong_FromLong((long)Fn(args));
  } catch (const PyError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

PyObject* is_dense(PyObject*, PyObject* o) {
  if (!THPVariable_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "not a tensor");
    return nullptr;
  }
  return PyBool_FromLong(dense(THPVariable_Unpack(o)));
}

#define HC_METHOD(name, n) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<name, n>)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {
    HC_METHOD(grad_norm, 5),       HC_METHOD(clip_grads, 6),     HC_METHOD(clip_grad_norm, 7),
    HC_METHOD(embedding, 6),       HC_METHOD(embedding_grad, 9), HC_METHOD(expert_sort, 5),
    HC_METHOD(expert_dispatch, 4), HC_METHOD(expert_combine, 5), HC_METHOD(expert_combine_grad, 7),
    HC_METHOD(rms_norm, 7),        HC_METHOD(rms_norm_8bit, 9),  HC_METHOD(rms_norm_grad, 10),
    HC_METHOD(route, 11),          HC_METHOD(route_grad, 8),     HC_METHOD(adamw_plan, 11),
    HC_METHOD(adamw, 14),
    {"is_dense", is_dense, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Tensors marshalled to the C ABI of libhc.", -1, methods,
                      nullptr,               nullptr,   nullptr,                                     nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
