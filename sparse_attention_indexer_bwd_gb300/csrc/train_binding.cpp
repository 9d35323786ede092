// Marshalling of the training operators for Python (train.py): argument
// checks, allocation of the results and the call of the C ABI, as one function
// a call.  A call from Python through ctypes spent 17 to 25 us of host time,
// most of it between the interpreter and the allocator; the smallest calls
// take 2 us on the GPU.  Nothing is computed here.
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

namespace {

using at::Tensor;

int code_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return IBWD_F32;
    case at::kBFloat16: return IBWD_BF16;
    case at::kHalf: return IBWD_F16;
    default: return -1;
  }
}
at::ScalarType type_of(int code) {
  return code == IBWD_F32 ? at::kFloat : code == IBWD_BF16 ? at::kBFloat16 : at::kHalf;
}

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const char* name, const char* what) {
  PyErr_Format(kind, "%s: %s", name, what);
  throw Refused{};
}

const Tensor& tensor(PyObject* o, const char* name) {
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

Matrix matrix(PyObject* o, const char* name) {
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
const void* like(PyObject* o, const char* name, at::IntArrayRef lead, int64_t last, at::ScalarType type,
                 const Tensor& of) {
  const Tensor& t = tensor(o, name);
  const auto size = t.sizes();
  const size_t dims = lead.size() + (last >= 0 ? 1 : 0);
  if (t.scalar_type() != type || t.device() != of.device() || !t.is_contiguous() || size.size() != dims ||
      size.slice(0, lead.size()) != lead || (last >= 0 && size[dims - 1] != last))
    refuse(PyExc_ValueError, name, "expected a contiguous tensor of another shape, type or device");
  return t.const_data_ptr();
}
const void* like_or_null(PyObject* o, const char* name, at::IntArrayRef lead, int64_t last, at::ScalarType type,
                         const Tensor& of) {
  return o == Py_None ? nullptr : like(o, name, lead, last, type, of);
}

// Elements between the rows of a result.  Nothing beside the rows where the
// input's are whole 16-byte blocks; else as little as puts them where the
// input's lie in a line of 128 bytes, since the kernels take matrices whose
// rows begin alike by vectors (layer norm of 8192x5001 in bf16, rows 5003
// apart: 39 us, into contiguous rows 100).
int64_t result_step(const Matrix& of) {
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
Output matrix_out(PyObject* o, const Matrix& of, int code) {
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

Tensor vector_out(at::IntArrayRef shape, at::ScalarType type, const Tensor& of) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(of.device()));
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

PyObject* g_error = nullptr;  // IndexerBwdError(status, where)

void check(int status, const char* where) {
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
void call(const char* where, int (*f)(P...), A... a) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f(static_cast<P>(a)...);
  PyEval_RestoreThread(state);
  check(status, where);
}

PyObject* wrap(Tensor t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(t));
}

template <typename... T>
PyObject* tuple_of(T... t) {
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

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return (float)v;
}
long integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

template <typename T>
T* data(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse(PyExc_TypeError, "arguments", "wrong number");
}

// Runs a body that may throw: a refusal has its Python error set, torch's own
// errors (out of memory) become its Python errors.
template <typename F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// gamma and beta: float32 or the type of x, both alike.
int weights(const Matrix& x, PyObject* gamma, PyObject* beta, const void** pg, const void** pb) {
  auto type = at::kFloat;
  for (PyObject* o : {gamma, beta})
    if (o != Py_None) {
      type = tensor(o, "gamma and beta").scalar_type();
      break;
    }
  if (type != at::kFloat && type != x.t->scalar_type())
    refuse(PyExc_ValueError, "gamma and beta", "expected float32 or the type of x");
  *pg = like_or_null(gamma, "gamma", {}, x.width, type, *x.t);
  *pb = like_or_null(beta, "beta", {}, x.width, type, *x.t);
  return code_of(type);
}

// (x, gamma, beta, eps, out type code or -1, out, stats)
PyObject* layer_norm_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const Matrix x = matrix(a[0], "x");
    const void *pg, *pb;
    const int wt = weights(x, a[1], a[2], &pg, &pb);
    const float eps = number(a[3]);
    int code = (int)integer(a[4]);
    if (code < 0) code = a[5] == Py_None ? x.code : matrix(a[5], "out").code;
    Output y = matrix_out(a[5], x, code);
    Tensor mean, rstd;
    if (a[6] == Py_True) {
      mean = vector_out(x.lead(), at::kFloat, *x.t);
      rstd = vector_out(x.lead(), at::kFloat, *x.t);
    }
    call("ibwd_layer_norm_fwd", ibwd_layer_norm_fwd, x.t->const_data_ptr(), x.code, x.step, pg, pb, wt,
         y.t.data_ptr(), code, y.step, data<float>(mean), data<float>(rstd), x.rows, (int)x.width, eps,
         stream_of(*x.t));
    y.written();
    return tuple_of(std::move(y.t), std::move(mean), std::move(rstd));
  });
}

// (dy, x, mean, rstd, gamma, out, weight_grads, workspace)
PyObject* layer_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    // it is written by its address and size
    if (a[6] == Py_True && a[7] != Py_None && !tensor(a[7], "workspace").is_contiguous())
      refuse(PyExc_ValueError, "workspace", "expected a contiguous tensor");
    const Matrix x = matrix(a[1], "x"), dy = matrix(a[0], "dy");
    if (dy.t->sizes() != x.t->sizes() || dy.t->device() != x.t->device())
      refuse(PyExc_ValueError, "dy", "expected the shape and device of x");
    const void *pg, *pb;
    const int wt = weights(x, a[4], Py_None, &pg, &pb);
    const auto mean = static_cast<const float*>(like(a[2], "mean", x.lead(), -1, at::kFloat, *x.t));
    const auto rstd = static_cast<const float*>(like(a[3], "rstd", x.lead(), -1, at::kFloat, *x.t));
    Output dx = matrix_out(a[5], x, x.code);
    Tensor dgamma, dbeta, work;
    void* ws = nullptr;
    size_t bytes = 0;
    if (a[6] == Py_True) {
      dgamma = vector_out({x.width}, at::kFloat, *x.t);
      dbeta = vector_out({x.width}, at::kFloat, *x.t);
      if (a[7] == Py_None)
        work = vector_out({(int64_t)ibwd_layer_norm_bwd_workspace_size(x.rows, (int)x.width)}, at::kByte, *x.t);
      else
        work = tensor(a[7], "workspace");
      ws = work.data_ptr();
      bytes = work.nbytes();
    }
    call("ibwd_layer_norm_bwd", ibwd_layer_norm_bwd, dy.t->const_data_ptr(), dy.code, dy.step, x.t->const_data_ptr(),
         x.code, x.step, pg, wt, mean, rstd, dx.t.data_ptr(), dx.step, data<float>(dgamma), data<float>(dbeta),
         x.rows, (int)x.width, ws, bytes, stream_of(*x.t));
    dx.written();
    return tuple_of(std::move(dx.t), std::move(dgamma), std::move(dbeta));
  });
}

// (logits, tokens, top_n, temperature)
PyObject* token_logprobs_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 4);
    const Matrix x = matrix(a[0], "logits");
    const auto tokens = static_cast<const int32_t*>(like_or_null(a[1], "tokens", x.lead(), -1, at::kInt, *x.t));
    const int top = (int)std::min<long>(std::max<long>(integer(a[2]), INT_MIN), INT_MAX);
    const float tau = number(a[3]);
    Tensor logprob, entropy = vector_out(x.lead(), at::kFloat, *x.t), lse = vector_out(x.lead(), at::kFloat, *x.t);
    if (tokens || a[1] != Py_None) logprob = vector_out(x.lead(), at::kFloat, *x.t);
    Tensor ids, best;
    if (top > 0 && top <= IBWD_MAX_TOP) {  // (the library refuses more)
      auto shape = x.lead().vec();
      shape.push_back(top);
      ids = vector_out(shape, at::kInt, *x.t);
      best = vector_out(shape, at::kFloat, *x.t);
    }
    call("ibwd_token_logprobs_fwd", ibwd_token_logprobs_fwd, x.t->const_data_ptr(), x.code, x.step, tokens, tau,
         data<float>(logprob), data<float>(entropy), data<float>(lse), data<int32_t>(ids), data<float>(best), top,
         x.rows, (int)x.width, stream_of(*x.t));
    return tuple_of(std::move(logprob), std::move(entropy), std::move(lse), std::move(ids), std::move(best));
  });
}

// (logits, tokens, lse, entropy, dlogprob, dentropy, temperature, out)
PyObject* token_logprobs_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 8);
    const Matrix x = matrix(a[0], "logits");
    auto rows = [&](int i, const char* name) {
      return static_cast<const float*>(like_or_null(a[i], name, x.lead(), -1, at::kFloat, *x.t));
    };
    // without a gradient of the log probabilities none comes through the tokens
    const int32_t* tokens = nullptr;
    if (a[4] != Py_None)
      tokens = static_cast<const int32_t*>(like_or_null(a[1], "tokens", x.lead(), -1, at::kInt, *x.t));
    like(a[2], "lse", x.lead(), -1, at::kFloat, *x.t);
    const float *lse = rows(2, "lse"), *entropy = rows(3, "entropy"), *da = rows(4, "dlogprob"),
                *dh = rows(5, "dentropy");
    const float tau = number(a[6]);
    Output dx = matrix_out(a[7], x, x.code);
    call("ibwd_token_logprobs_bwd", ibwd_token_logprobs_bwd, x.t->const_data_ptr(), x.code, x.step, tokens, tau, lse,
         entropy, da, dh, dx.t.data_ptr(), dx.step, x.rows, (int)x.width, stream_of(*x.t));
    dx.written();
    return wrap(std::move(dx.t));
  });
}

struct Kept {
  const int32_t* ids;
  const float* teacher;
  int64_t k;
};
Kept kept(const Matrix& x, PyObject* ids, PyObject* teacher) {
  const Tensor& t = tensor(ids, "ids");
  if (t.dim() != x.t->dim()) refuse(PyExc_ValueError, "ids", "expected [..., K] beside the logits");
  const int64_t k = t.size(t.dim() - 1);
  if (k > INT_MAX) refuse(PyExc_ValueError, "ids", "too many slots");
  return {static_cast<const int32_t*>(like(ids, "ids", x.lead(), k, at::kInt, *x.t)),
          static_cast<const float*>(like(teacher, "teacher", x.lead(), k, at::kFloat, *x.t)), k};
}

// (logits, ids, teacher, temperature)
PyObject* distill_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 4);
    const Matrix x = matrix(a[0], "logits");
    const Kept k = kept(x, a[1], a[2]);
    const float tau = number(a[3]);
    Tensor loss = vector_out(x.lead(), at::kFloat, *x.t), lse = vector_out(x.lead(), at::kFloat, *x.t);
    call("ibwd_distill_fwd", ibwd_distill_fwd, x.t->const_data_ptr(), x.code, x.step, k.ids, k.teacher, (int)k.k, tau,
         data<float>(loss), data<float>(lse), x.rows, (int)x.width, stream_of(*x.t));
    return tuple_of(std::move(loss), std::move(lse));
  });
}

// (logits, ids, teacher, lse, dloss, temperature, out)
PyObject* distill_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const Matrix x = matrix(a[0], "logits");
    const Kept k = kept(x, a[1], a[2]);
    const auto lse = static_cast<const float*>(like(a[3], "lse", x.lead(), -1, at::kFloat, *x.t));
    const auto dloss = static_cast<const float*>(like(a[4], "dloss", x.lead(), -1, at::kFloat, *x.t));
    const float tau = number(a[5]);
    Output dx = matrix_out(a[6], x, x.code);
    call("ibwd_distill_bwd", ibwd_distill_bwd, x.t->const_data_ptr(), x.code, x.step, k.ids, k.teacher, (int)k.k, tau,
         lse, dloss, dx.t.data_ptr(), dx.step, x.rows, (int)x.width, stream_of(*x.t));
    dx.written();
    return wrap(std::move(dx.t));
  });
}

// (logits, ids, teacher, row_weight, grad_scale, temperature, out)
PyObject* distill_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const Matrix x = matrix(a[0], "logits");
    const Kept k = kept(x, a[1], a[2]);
    const auto weight =
        static_cast<const float*>(like_or_null(a[3], "row_weight", x.lead(), -1, at::kFloat, *x.t));
    const float scale = number(a[4]), tau = number(a[5]);
    Tensor loss = vector_out(x.lead(), at::kFloat, *x.t);
    Output dx = matrix_out(a[6], x, x.code);
    call("ibwd_distill_grad", ibwd_distill_grad, x.t->const_data_ptr(), x.code, x.step, k.ids, k.teacher, (int)k.k,
         tau, weight, scale, data<float>(loss), dx.t.data_ptr(), dx.step, x.rows, (int)x.width, stream_of(*x.t));
    dx.written();
    return tuple_of(std::move(loss), std::move(dx.t));
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(layer_norm_fwd),     FAST(layer_norm_bwd), FAST(token_logprobs_fwd),
                         FAST(token_logprobs_bwd), FAST(distill_fwd),    FAST(distill_bwd),
                         FAST(distill_grad),       {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_train", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__train() { return PyModule_Create(&module); }
