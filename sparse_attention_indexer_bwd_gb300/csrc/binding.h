// What the marshalling of the operators for Python shares: argument checks,
// results, errors. Nothing is computed here.
#pragma once
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <vector>

#include "indexer_train.h"

namespace binding {

using at::Tensor;

inline int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return IBWD_F32;
    case at::kBFloat16: return IBWD_BF16;
    case at::kHalf: return IBWD_F16;
    default: return -1;
  }
}
inline at::ScalarType type_of(int code) {
  return code == IBWD_F32 ? at::kFloat : code == IBWD_BF16 ? at::kBFloat16 : at::kHalf;
}

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] inline void refuse(PyObject* kind, const char* name, const char* what) {
  PyErr_Format(kind, "%s: %s", name, what);
  throw Refused{};
}

inline const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, name, "must be a torch.Tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided) refuse(PyExc_ValueError, name, "expected a dense tensor");
  return t;
}

// A [..., width] matrix whose rows step evenly.
struct Matrix {
  const Tensor* t = nullptr;
  int64_t rows = 0, width = 0, step = 0;
  int code = 0;
  at::IntArrayRef lead() const { return t->sizes().slice(0, t->dim() - 1); }
};

inline Matrix matrix(PyObject* o, const char* name) {
  Matrix m;
  const Tensor& t = tensor(o, name);
  m.t = &t;
  m.code = code_of(t.scalar_type());
  if (!t.is_cuda() || m.code < 0)
    refuse(PyExc_ValueError, name, "expected a CUDA tensor of float32, bfloat16 or float16");
  const auto size = t.sizes();
  const auto stride = t.strides();
  const int64_t dims = t.dim();
  if (dims < 2 || size[dims - 1] < 1) refuse(PyExc_ValueError, name, "expected [..., width >= 1]");
  m.width = size[dims - 1];
  if (m.width > INT_MAX) refuse(PyExc_ValueError, name, "the rows are too wide");
  // the library runs on the current device, on the stream that is current there
  if (t.device().index() != c10::cuda::current_device())
    refuse(PyExc_ValueError, name, "expected a tensor of the current device");
  m.rows = t.numel() / m.width;
  m.step = m.width;
  if (m.rows == 0 || t.is_contiguous()) return m;
  int64_t rows = 1;
  for (int64_t d = dims - 2; d >= 0; --d) {
    if (size[d] == 1) continue;
    if (rows == 1)
      m.step = stride[d];
    else if (stride[d] != m.step * rows)
      refuse(PyExc_ValueError, name, "the rows do not step evenly");
    rows *= size[d];
  }
  if ((m.width > 1 && stride[dims - 1] != 1) || m.step < m.width)
    refuse(PyExc_ValueError, name, "expected unit stride along rows that do not overlap");
  return m;
}

// A contiguous argument of the given shape (`lead`, then `last` unless < 0) and type.
inline const void* like(PyObject* o, const char* name, at::IntArrayRef lead, int64_t last, at::ScalarType type,
                 const Tensor& of) {
  const Tensor& t = tensor(o, name);
  const auto size = t.sizes();
  const size_t dims = lead.size() + (last >= 0 ? 1 : 0);
  if (t.scalar_type() != type || t.device() != of.device() || !t.is_contiguous() || size.size() != dims ||
      size.slice(0, lead.size()) != lead || (last >= 0 && size[dims - 1] != last))
    refuse(PyExc_ValueError, name, "expected a contiguous tensor of another shape, type or device");
  return t.const_data_ptr();
}
inline const void* like_or_null(PyObject* o, const char* name, at::IntArrayRef lead, int64_t last, at::ScalarType type,
                         const Tensor& of) {
  return o == Py_None ? nullptr : like(o, name, lead, last, type, of);
}

// Elements between the rows of a result.  Nothing beside the rows where the
// input's are whole 16-byte blocks; else as little as puts them where the
// input's lie in a line of 128 bytes, since the kernels take matrices whose
// rows begin alike by vectors (layer norm of 8192x5001 in bf16, rows 5003
// apart: 39 us, into contiguous rows 100).
inline int64_t result_step(const Matrix& of) {
  const int64_t size = (int64_t)of.t->element_size(), gap = of.step - of.width;
  if (of.rows <= 1 || (of.width * size % 16 == 0 && of.step * size % 16 == 0)) return of.width;
  return of.width + gap % (128 / size);
}

// An output matrix: given, or allocated.
struct Output {
  Tensor t;
  int64_t step;
  bool given = false;
  // After it was written: autograd finds an overwritten tensor by its version.
  void written() const {
    if (given && !t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  }
};
inline Output matrix_out(PyObject* o, const Matrix& of, int code) {
  const auto type = type_of(code);
  if (o == Py_None) {
    const auto options = of.t->options().dtype(type).requires_grad(false);
    const int64_t step = result_step(of), dims = of.t->dim();
    if (step == of.width) return {at::empty(of.t->sizes(), options), step};
    std::vector<int64_t> strides(dims, 1);
    for (int64_t d = dims - 2, s = step; d >= 0; s *= of.t->size(d--)) strides[d] = s;
    return {at::empty_strided(of.t->sizes(), strides, options), step};
  }
  const Matrix m = matrix(o, "out");
  if (m.t->sizes() != of.t->sizes() || m.code != code || m.t->device() != of.t->device())
    refuse(PyExc_ValueError, "out", "expected the shape and device of the input and the result's type");
  return {*m.t, m.step, true};
}

inline Tensor vector_out(at::IntArrayRef shape, at::ScalarType type, const Tensor& of) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(of.device()));
}

inline void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

inline PyObject* g_error = nullptr;  // IndexerBwdError(status, where)

inline void check(int status, const char* where) {
  if (status == IBWD_OK) return;
  if (PyObject* e = PyObject_CallFunction(g_error, "is", status, where)) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

// Calls the library without the interpreter lock, since a launch waits while
// the launch queue is full; a status other than OK becomes an IndexerBwdError.
template <typename... P, typename... A>
inline void call(const char* where, int (*f)(P...), A... a) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f(static_cast<P>(a)...);
  PyEval_RestoreThread(state);
  check(status, where);
}

inline PyObject* wrap(Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}

template <typename... T>
inline PyObject* tuple_of(T... t) {
  PyObject* items[] = {wrap(std::move(t))...};
  PyObject* r = PyTuple_New(sizeof...(T));
  for (size_t i = 0; i < sizeof...(T); ++i) {
    if (r)
      PyTuple_SET_ITEM(r, i, items[i]);
    else
      Py_XDECREF(items[i]);
  }
  return r;
}

inline float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}
inline long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

template <typename T>
T* data(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

inline void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "arguments", "wrong number");
}

// Runs a body that may throw: a refusal has its Python error set, torch's own
// errors (out of memory) become its Python errors.
template <typename F>
inline PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

}  // namespace binding
