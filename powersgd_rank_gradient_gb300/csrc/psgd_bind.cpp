// Python binding of the training operators' calls (include/psgd.h): argument
// checks, outputs and the current stream for training.py.  A call of one token
// or one row takes the GPU two or three microseconds, less than the same checks
// take in Python, so they are compiled; nothing is computed here.  Autograd does
// not see these calls: while it records, operands that require a gradient are
// refused, and what a call writes advances its tensor's version, so that a value
// saved before is known to be overwritten.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>
#include <vector>

#include "../../include/psgd.h"

#ifndef PSGD_BIND_HASH
#define PSGD_BIND_HASH "unknown"
#endif
#ifndef PSGD_SOURCE_HASH
#define PSGD_SOURCE_HASH "unknown"
#endif
#ifndef PSGD_BIND_TORCH
#define PSGD_BIND_TORCH "unknown"
#endif

namespace {

struct ValueError {
  std::string message;
};
struct PythonError {};  // already set

// What a handle's Python object keeps for its calls.
struct Spec {
  void* handle;
  int64_t rows;  // of the table
  int64_t dim;
  double value;  // scale, eps
  int64_t padding;
  int index;     // CUDA device
};

Spec* spec_of(PyObject* o) {
  auto* s = static_cast<Spec*>(PyCapsule_GetPointer(o, "psgd.spec"));
  if (!s) throw PythonError();
  return s;
}

std::string str(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw ValueError{std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

// A tensor whose values (not indices) a call reads or writes.
const at::Tensor& values(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.requires_grad() && at::GradMode::is_enabled())
    throw ValueError{std::string(what) + " requires a gradient, which this call does not record: use torch.no_grad(), and "
                     "the operator's own gradient"};
  return t;
}

void on_device(const at::Tensor& t, int index, const char* what) {
  if (!t.is_cuda() || t.get_device() != index)
    throw ValueError{std::string(what) + " must be on cuda:" + std::to_string(index) + ", got " + t.device().str()};
}

int dtype_code(at::ScalarType t) {
  return t == at::kFloat ? PSGD_F32 : t == at::kHalf ? PSGD_F16 : t == at::kBFloat16 ? PSGD_BF16 : -1;
}

// The library's name of the type of `t`, which must be on CUDA device `index`.
psgd_dtype dtype_of(const at::Tensor& t, int index, const char* what) {
  const int d = dtype_code(t.scalar_type());
  if (d < 0)
    throw ValueError{std::string(what) + " must be float32, float16 or bfloat16, got " + c10::toString(t.scalar_type())};
  on_device(t, index, what);
  return static_cast<psgd_dtype>(d);
}

int id_bits_of(const at::Tensor& t, int index, const char* what) {
  const int bits = t.scalar_type() == at::kLong ? 64 : t.scalar_type() == at::kInt ? 32 : 0;
  if (!bits)
    throw ValueError{std::string(what) + " must be int32 or int64, got " + c10::toString(t.scalar_type())};
  on_device(t, index, what);
  return bits;
}

// The first `lead` dimensions as (outer, inner) with a stride each.
struct Layout {
  int64_t outer, inner, os, is;
};
Layout layout_of(at::IntArrayRef shape, at::IntArrayRef stride, size_t lead, const char* what) {
  if (lead == 2) return {shape[0], shape[1], stride[0], stride[1]};
  if (lead == 1) return {1, shape[0], 0, stride[0]};
  if (lead == 0) return {1, 1, 0, 0};
  // more than two: all but the last must collapse into one
  int64_t outer = 1;
  for (size_t d = 0; d + 1 < lead; ++d) outer *= shape[d];
  if (outer == 0 || shape[lead - 1] == 0) return {0, 0, 0, 0};
  int64_t step = 0, run = 1;
  bool have = false;
  for (size_t d = lead - 1; d-- > 0;) {
    if (shape[d] == 1) continue;
    if (!have) {
      step = stride[d];
      have = true;
    }
    if (stride[d] != step * run)
      throw ValueError{std::string(what) + ": its leading dimensions must be contiguous among themselves"};
    run *= shape[d];
  }
  return {outer, shape[lead - 1], step, stride[lead - 1]};
}

// (rows, row stride) of a tensor of rows of `dim` elements.
struct Rows {
  int64_t rows, stride;
};
Rows rows_of(const at::Tensor& t, int64_t dim, const char* what) {
  const auto shape = t.sizes();
  if (dim < 1 || shape.empty() || shape.back() != dim)
    throw ValueError{std::string(what) + " must have a last dimension of " + std::to_string(dim < 1 ? 1 : dim) + ", got " +
                     str(shape)};
  if (t.is_contiguous()) return {t.numel() / dim, dim};
  const auto stride = t.strides();
  if (dim > 1 && stride.back() != 1)
    throw ValueError{std::string(what) + " must be contiguous in its last dimension"};
  if (shape.size() == 2) return {shape[0], stride[0]};
  const Layout l = layout_of(shape, stride, shape.size() - 1, what);
  if (l.outer > 1 && l.inner > 1 && l.os != l.inner * l.is)
    throw ValueError{std::string(what) + ": its rows must be one stride apart"};
  return {l.outer * l.inner, l.inner > 1 ? l.is : l.os};
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int index) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(index)));
}

// A contiguous tensor of `shape` in the memory of `t`, `offset` elements in.
at::Tensor part_of(const at::Tensor& t, at::IntArrayRef shape, int64_t offset) {
  at::Tensor p = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.storage()), t.key_set(), t.dtype());
  p.unsafeGetTensorImpl()->set_storage_offset(offset);
  p.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return p;
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream(); }

// Raises the library's error of a failed call, as every other binding does.
void check(int rc) {
  if (rc >= 0) return;
  PyObject* lib = PyImport_ImportModule("powersgd_rank_gradient_gb300._lib");
  PyObject* r = lib ? PyObject_CallMethod(lib, "check", "i", rc) : nullptr;
  Py_XDECREF(r);
  Py_XDECREF(lib);
  throw PythonError();
}

template <typename F> int call(F&& f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

// The written tensor as Python's object: the caller's, or a new one.
PyObject* given_or_new(PyObject* given, at::Tensor made) {
  if (given != Py_None) {
    if (!made.is_inference()) made.unsafeGetTensorImpl()->bump_version();
    Py_INCREF(given);
    return given;
  }
  PyObject* o = THPVariable_Wrap(std::move(made));
  if (!o) throw PythonError();
  return o;
}

struct Object {  // an owned reference
  PyObject* p;
  explicit Object(PyObject* o) : p(o) {}
  Object(const Object&) = delete;
  ~Object() { Py_XDECREF(p); }
};

PyObject* pack(std::initializer_list<Object*> items) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
  if (!t) throw PythonError();
  Py_ssize_t i = 0;
  for (Object* o : items) {
    PyTuple_SET_ITEM(t, i++, o->p);
    o->p = nullptr;
  }
  return t;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PythonError();
  return v != 0;
}

// C++ exceptions end here.
template <typename F> PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.message.c_str());
  } catch (const PythonError&) {
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void free_spec(PyObject* o) { delete static_cast<Spec*>(PyCapsule_GetPointer(o, "psgd.spec")); }

// spec(handle, rows, dim, value, padding, index)
PyObject* py_spec(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Spec v{reinterpret_cast<void*>(integer(a[0])), integer(a[1]), integer(a[2]), number(a[3]), integer(a[4]),
           static_cast<int>(integer(a[5]))};
    return PyCapsule_New(new Spec(v), "psgd.spec", free_spec);
  });
}

// closed(spec): the handle is gone
PyObject* py_closed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    spec_of(a[0])->handle = nullptr;
    Py_RETURN_NONE;
  });
}

// -- embedding ---------------------------------------------------------------------

struct Table {
  psgd_dtype dtype;
  int64_t stride;
};
Table table_of(const Spec& s, const at::Tensor& t, const char* what) {
  if (t.dim() != 2 || t.size(0) != s.rows || t.size(1) != s.dim)
    throw ValueError{std::string(what) + " must be " + str({s.rows, s.dim}) + ", got " + str(t.sizes())};
  if (t.stride(1) != 1 && s.dim > 1) throw ValueError{std::string(what) + " must be contiguous in its last dimension"};
  return {dtype_of(t, s.index, what), s.rows > 1 ? t.stride(0) : s.dim};
}

struct TokenRows {
  psgd_dtype dtype;
  int64_t os, is;
};
TokenRows token_rows_of(const Spec& s, const at::Tensor& t, at::IntArrayRef ids, const char* what) {
  const auto shape = t.sizes();
  const size_t lead = ids.size();
  bool same = shape.size() == lead + 1 && shape[lead] == s.dim;
  for (size_t i = 0; same && i < lead; ++i) same = shape[i] == ids[i];
  if (!same) {
    std::vector<int64_t> want(ids.begin(), ids.end());
    want.push_back(s.dim);
    throw ValueError{std::string(what) + " must be " + str(want) + ", got " + str(shape)};
  }
  const auto stride = t.strides();
  if (stride[lead] != 1 && s.dim > 1) throw ValueError{std::string(what) + " must be contiguous in its last dimension"};
  const psgd_dtype d = dtype_of(t, s.index, what);
  const Layout l = layout_of(shape, stride, lead, what);
  return {d, l.os, l.is};
}

// embedding_forward(spec, weight, ids, out, out_dtype)
PyObject* py_embedding_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Spec& s = *spec_of(a[0]);
    const at::Tensor &weight = values(a[1], "weight"), &ids = tensor(a[2], "ids");
    const Table w = table_of(s, weight, "weight");
    const int bits = id_bits_of(ids, s.index, "ids");
    const Layout l = layout_of(ids.sizes(), ids.strides(), ids.sizes().size(), "ids");
    at::Tensor out;
    TokenRows o;
    if (a[3] == Py_None) {
      at::ScalarType type = weight.scalar_type();
      if (a[4] != Py_None) {
        if (!THPDtype_Check(a[4])) throw ValueError{"out_dtype must be a torch.dtype"};
        type = reinterpret_cast<THPDtype*>(a[4])->scalar_type;
      }
      const int d = dtype_code(type);
      if (d < 0)
        throw ValueError{std::string("out_dtype must be float32, float16 or bfloat16, got ") + c10::toString(type)};
      c10::SmallVector<int64_t, 8> shape(ids.sizes().begin(), ids.sizes().end());
      shape.push_back(s.dim);
      out = fresh(shape, type, s.index);
      o = {static_cast<psgd_dtype>(d), l.inner * s.dim, s.dim};
    } else {
      out = values(a[3], "out");
      o = token_rows_of(s, out, ids.sizes(), "out");
    }
    void* stream = stream_of(s.index);
    check(call([&] {
      return psgd_embedding_forward(static_cast<psgd_embedding*>(s.handle), weight.const_data_ptr(), w.dtype, w.stride,
                                    ids.const_data_ptr(), bits, l.outer, l.inner, l.os, l.is,
                                    static_cast<float>(s.value), out.mutable_data_ptr(), o.dtype, o.os, o.is, stream);
    }));
    return given_or_new(a[3], std::move(out));
  });
}

// embedding_backward(spec, ids, grad, out, accumulate)
PyObject* py_embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Spec& s = *spec_of(a[0]);
    const at::Tensor &ids = tensor(a[1], "ids"), &grad = values(a[2], "grad");
    const int bits = id_bits_of(ids, s.index, "ids");
    const Layout l = layout_of(ids.sizes(), ids.strides(), ids.sizes().size(), "ids");
    const TokenRows g = token_rows_of(s, grad, ids.sizes(), "grad");
    const bool accumulate = truth(a[4]);
    if (a[3] == Py_None && accumulate) throw ValueError{"accumulate needs an out to add to"};
    at::Tensor out = a[3] == Py_None ? fresh({s.rows, s.dim}, at::kFloat, s.index) : values(a[3], "out");
    const Table w = table_of(s, out, "out");
    void* stream = stream_of(s.index);
    check(call([&] {
      return psgd_embedding_backward(static_cast<psgd_embedding*>(s.handle), ids.const_data_ptr(), bits, l.outer, l.inner,
                                     l.os, l.is, grad.const_data_ptr(), g.dtype, g.os, g.is,
                                     static_cast<float>(s.value), s.padding, accumulate, out.mutable_data_ptr(), w.dtype,
                                     w.stride, stream);
    }));
    return given_or_new(a[3], std::move(out));
  });
}

// -- layer norm --------------------------------------------------------------------

// Type and addresses of two optional vectors of one type.
struct Pair {
  psgd_dtype dtype;
  const at::Tensor *a, *b;
  const void* pa() const { return a ? a->const_data_ptr() : nullptr; }
  const void* pb() const { return b ? b->const_data_ptr() : nullptr; }
};
const at::Tensor* vector_of(const Spec& s, PyObject* o, const char* what) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = values(o, what);
  if (t.dim() != 1 || t.size(0) != s.dim || !t.is_contiguous())
    throw ValueError{std::string(what) + " must be a contiguous vector of " + std::to_string(s.dim) + " elements"};
  return &t;
}
Pair pair_of(const Spec& s, const at::Tensor* a, const at::Tensor* b, const char* name_a, const char* name_b) {
  Pair p{PSGD_F32, a, b};
  if (a) p.dtype = dtype_of(*a, s.index, name_a);
  if (b) {
    const psgd_dtype d = dtype_of(*b, s.index, name_b);
    if (a && d != p.dtype) throw ValueError{std::string(name_a) + " and " + name_b + " must have one type"};
    p.dtype = d;
  }
  return p;
}

// The row stride of a tensor that must match x.
int64_t stride_like(const Spec& s, const at::Tensor& t, const at::Tensor& x, const char* what) {
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type())
    throw ValueError{std::string(what) + " must have x's shape and type"};
  on_device(t, s.index, what);
  return rows_of(t, s.dim, what).stride;
}

// layernorm_forward(spec, x, weight, bias, out)
PyObject* py_layernorm_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const Spec& s = *spec_of(a[0]);
    const at::Tensor& x = values(a[1], "x");
    const psgd_dtype d = dtype_of(x, s.index, "x");
    const Rows r = rows_of(x, s.dim, "x");
    const Pair p = pair_of(s, vector_of(s, a[2], "weight"), vector_of(s, a[3], "bias"), "weight", "bias");
    at::Tensor out;
    int64_t ys = s.dim;
    if (a[4] == Py_None) {
      out = fresh(x.sizes(), x.scalar_type(), s.index);
    } else {
      out = values(a[4], "out");
      ys = stride_like(s, out, x, "out");
    }
    const auto lead = x.sizes().slice(0, x.sizes().size() - 1);
    // one allocation for both statistics
    const at::Tensor stats = fresh({2 * r.rows}, at::kFloat, s.index);
    at::Tensor mean = part_of(stats, lead, 0), rstd = part_of(stats, lead, r.rows);
    void* stream = stream_of(s.index);
    check(call([&] {
      return psgd_layernorm_forward(static_cast<psgd_layernorm*>(s.handle), x.const_data_ptr(), d, r.stride, r.rows,
                                    p.pa(), p.pb(), p.dtype, static_cast<float>(s.value), out.mutable_data_ptr(), ys,
                                    static_cast<float*>(mean.mutable_data_ptr()),
                                    static_cast<float*>(rstd.mutable_data_ptr()), stream);
    }));
    Object y(given_or_new(a[4], std::move(out))), m(given_or_new(Py_None, std::move(mean))),
        v(given_or_new(Py_None, std::move(rstd)));
    return pack({&y, &m, &v});
  });
}

const float* stat_of(const Spec& s, PyObject* o, int64_t rows, const char* what) {
  const at::Tensor& t = values(o, what);
  if (t.scalar_type() != at::kFloat || t.numel() != rows || !t.is_contiguous())
    throw ValueError{std::string(what) + " must be a contiguous float32 tensor of " + std::to_string(rows) + " elements"};
  on_device(t, s.index, what);
  return static_cast<const float*>(t.const_data_ptr());
}

// layernorm_backward(spec, grad, x, mean, rstd, weight, dx, dweight, dbias, accumulate)
PyObject* py_layernorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Spec& s = *spec_of(a[0]);
    const at::Tensor &grad = values(a[1], "grad"), &x = values(a[2], "x");
    const psgd_dtype d = dtype_of(x, s.index, "x");
    const Rows r = rows_of(x, s.dim, "x");
    const int64_t gs = stride_like(s, grad, x, "grad");
    const float *mean = stat_of(s, a[3], r.rows, "mean"), *rstd = stat_of(s, a[4], r.rows, "rstd");
    const Pair p = pair_of(s, vector_of(s, a[5], "weight"), nullptr, "weight", "");
    at::Tensor dx;
    int64_t ds = s.dim;
    if (a[6] == Py_None) {
      dx = fresh(x.sizes(), x.scalar_type(), s.index);
    } else {
      dx = values(a[6], "dx");
      ds = stride_like(s, dx, x, "dx");
    }
    const bool accumulate = truth(a[9]);
    const at::Tensor *gw = vector_of(s, a[7], "dweight"), *gb = vector_of(s, a[8], "dbias");
    if (accumulate && (!gw || !gb)) throw ValueError{"accumulate needs a dweight and a dbias to add to"};
    const at::ScalarType made = gw ? gw->scalar_type() : gb ? gb->scalar_type() : at::kFloat;
    at::Tensor dw = gw ? *gw : fresh({s.dim}, made, s.index), db = gb ? *gb : fresh({s.dim}, made, s.index);
    const Pair o = pair_of(s, &dw, &db, "dweight", "dbias");
    void* stream = stream_of(s.index);
    check(call([&] {
      return psgd_layernorm_backward(static_cast<psgd_layernorm*>(s.handle), grad.const_data_ptr(), gs,
                                     x.const_data_ptr(), d, r.stride, r.rows, mean, rstd, p.pa(), p.dtype,
                                     dx.mutable_data_ptr(), ds, dw.mutable_data_ptr(), db.mutable_data_ptr(), o.dtype,
                                     accumulate, stream);
    }));
    Object u(given_or_new(a[6], std::move(dx))), v(given_or_new(a[7], std::move(dw))), w(given_or_new(a[8], std::move(db)));
    return pack({&u, &v, &w});
  });
}

// -- distillation --------------------------------------------------------------------

// distill(logits, teacher_logits, teacher_indices, temperature, weights, grad_scale, dlogits, with_grad)
PyObject* py_distill(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor &z = values(a[0], "logits"), &t = values(a[1], "teacher_logits"), &at_ = tensor(a[2], "teacher_indices");
    if (!z.is_cuda()) throw ValueError{"logits must be a CUDA tensor"};
    const int index = z.get_device();
    const auto shape = z.sizes();
    if (shape.empty()) throw ValueError{"logits must have a vocabulary dimension"};
    const int64_t vocab = shape.back();
    const auto lead = shape.slice(0, shape.size() - 1);
    const psgd_dtype zd = dtype_of(z, index, "logits");
    const Rows r = rows_of(z, vocab, "logits");
    const auto tshape = t.sizes();
    if (tshape.empty() || tshape != at_.sizes() || tshape.slice(0, tshape.size() - 1) != lead)
      throw ValueError{"teacher_logits and teacher_indices must have the logits' leading shape and one k"};
    const int64_t k = tshape.back();
    const psgd_dtype td = dtype_of(t, index, "teacher_logits");
    const int bits = id_bits_of(at_, index, "teacher_indices");
    const int64_t ts = rows_of(t, k, "teacher_logits").stride, ns = rows_of(at_, k, "teacher_indices").stride;
    const float* w = nullptr;
    if (a[4] != Py_None) {
      const at::Tensor& wt = values(a[4], "weights");
      if (wt.scalar_type() != at::kFloat || wt.sizes() != lead || !wt.is_contiguous())
        throw ValueError{"weights must be a contiguous float32 tensor of the logits' leading shape"};
      on_device(wt, index, "weights");
      w = static_cast<const float*>(wt.const_data_ptr());
    }
    const bool with_grad = truth(a[7]);
    at::Tensor dz;
    int64_t ds = 0;
    if (!with_grad) {
      if (a[6] != Py_None) throw ValueError{"dlogits given with with_grad=False"};
    } else if (a[6] == Py_None) {
      dz = fresh(shape, z.scalar_type(), index);
      ds = vocab;
    } else {
      dz = values(a[6], "dlogits");
      if (dz.sizes() != shape || dz.scalar_type() != z.scalar_type())
        throw ValueError{"dlogits must have the logits' shape and type"};
      on_device(dz, index, "dlogits");
      ds = rows_of(dz, vocab, "dlogits").stride;
    }
    const double temperature = number(a[3]), scale = number(a[5]);
    at::Tensor losses = fresh(lead, at::kFloat, index);
    void* stream = stream_of(index);
    check(call([&] {
      return psgd_distill(z.const_data_ptr(), zd, r.stride, r.rows, vocab, t.const_data_ptr(), td, ts,
                          at_.const_data_ptr(), bits, ns, static_cast<int32_t>(std::min<int64_t>(k, INT32_MAX)), static_cast<float>(temperature), w,
                          static_cast<float>(scale), static_cast<float*>(losses.mutable_data_ptr()),
                          with_grad ? dz.mutable_data_ptr() : nullptr, ds, index, stream);
    }));
    Object l(given_or_new(Py_None, std::move(losses)));
    Object g(nullptr);
    if (with_grad) {
      g.p = given_or_new(a[6], std::move(dz));
    } else {
      Py_INCREF(Py_None);
      g.p = Py_None;
    }
    return pack({&l, &g});
  });
}

// What this file was built against: the library's build id, torch's version.
// (The hash is what build.py looks for.)
PyObject* py_built_with(PyObject*, PyObject*) {
  static const char hash[] = "psgd-bind-hash:" PSGD_BIND_HASH;
  return Py_BuildValue("(sss)", "psgd-source-hash:" PSGD_SOURCE_HASH, PSGD_BIND_TORCH, hash);
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {
    {"spec", FAST(py_spec), nullptr},
    {"closed", FAST(py_closed), nullptr},
    {"embedding_forward", FAST(py_embedding_forward), nullptr},
    {"embedding_backward", FAST(py_embedding_backward), nullptr},
    {"layernorm_forward", FAST(py_layernorm_forward), nullptr},
    {"layernorm_backward", FAST(py_layernorm_backward), nullptr},
    {"distill", FAST(py_distill), nullptr},
    {"built_with", py_built_with, METH_NOARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bind", "Calls of the training operators.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&kModule); }
