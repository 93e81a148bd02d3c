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
    {"is_dense", is_dense, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Tensors marshalled to the C ABI of libhc.", -1, methods,
                      nullptr,               nullptr,   nullptr,                                     nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
