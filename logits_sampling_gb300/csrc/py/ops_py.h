// ops_py.h -- what the Python calls share: arguments, checks, outputs, streams
// and errors.  No arithmetic.
#pragma once

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <optional>
#include <string>

#include "ls_sampler.h"

namespace {

PyObject* ls_error;  // the package's LSError(status, what); NULL until the library's functions are bound

// An error on its way to Python.
struct Fail {
  PyObject* type;
  std::string what;
};

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
constexpr int kMostArgs = 20;
struct Names {
  const char* function;
  int count, required;
  const char* text[kMostArgs];
  PyObject* name[kMostArgs];  // interned
};

// Fills out[] (NULL: absent, or None) from a vectorcall's arguments.
void parse(const Names& n, PyObject* const* args, Py_ssize_t positional, PyObject* keywords, PyObject** out) {
  if (positional > n.count)
    throw Fail{PyExc_TypeError, std::string(n.function) + "() takes at most " + std::to_string(n.count) + " arguments"};
  for (int i = 0; i < n.count; ++i) out[i] = i < positional ? args[i] : nullptr;
  const Py_ssize_t k = keywords ? PyTuple_GET_SIZE(keywords) : 0;
  for (Py_ssize_t q = 0; q < k; ++q) {
    PyObject* key = PyTuple_GET_ITEM(keywords, q);
    int at = -1;
    for (int i = 0; i < n.count && at < 0; ++i)
      if (key == n.name[i]) at = i;
    for (int i = 0; i < n.count && at < 0; ++i)
      if (PyUnicode_Compare(key, n.name[i]) == 0) at = i;
    if (at < 0)
      throw Fail{PyExc_TypeError, std::string(n.function) + "() got an unexpected keyword argument '" +
                                      PyUnicode_AsUTF8(key) + "'"};
    if (out[at])
      throw Fail{PyExc_TypeError, std::string(n.function) + "() got multiple values for argument '" + n.text[at] + "'"};
    out[at] = args[positional + q];
  }
  for (int i = 0; i < n.count; ++i) {
    if (out[i] == Py_None) out[i] = nullptr;
    if (i < n.required && !out[i])
      throw Fail{PyExc_TypeError, std::string(n.function) + "() misses argument '" + n.text[i] + "'"};
  }
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Fail{PyExc_TypeError, std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o, const char* what) {
  const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : [&] {
    PyObject* i = PyNumber_Index(o);
    if (!i) return -1ll;
    const long long r = PyLong_AsLongLong(i);
    Py_DECREF(i);
    return r;
  }();
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Fail{PyExc_TypeError, std::string(what) + " must be an integer"};
  }
  return v;
}

int32_t count32(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) throw Fail{PyExc_ValueError, std::string(what) + " is out of range"};
  return (int32_t)v;
}

float number(PyObject* o, float otherwise, const char* what) {
  if (!o) return otherwise;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Fail{PyExc_TypeError, std::string(what) + " must be a number"};
  }
  return (float)v;
}

// A logits matrix.
struct Matrix {
  const at::Tensor* t;
  void* p;
  ls_dtype dtype;
  int64_t rows, vocab, stride;
};
Matrix matrix(PyObject* o) {
  const at::Tensor& t = tensor(o, "logits");
  Matrix m;
  m.t = &t;
  if (t.scalar_type() == at::kFloat)
    m.dtype = LS_DTYPE_F32;
  else if (t.scalar_type() == at::kBFloat16)
    m.dtype = LS_DTYPE_BF16;
  else
    throw Fail{PyExc_TypeError, std::string("unsupported logits dtype ") + c10::toString(t.scalar_type())};
  if (t.dim() != 2) throw Fail{PyExc_ValueError, "logits must be 2-D [rows, vocab]"};
  if (t.stride(1) != 1) throw Fail{PyExc_ValueError, "logits rows must be contiguous (stride(1) == 1)"};
  if (!t.is_cuda()) throw Fail{PyExc_ValueError, "logits must be a CUDA tensor"};
  m.rows = t.size(0);
  m.vocab = t.size(1);
  m.stride = m.rows <= 1 && t.stride(0) < m.vocab ? m.vocab : t.stride(0);
  m.p = t.data_ptr();
  return m;
}

// Every tensor of a call lies on the logits' device, on which its kernels run.
void on_device(int64_t device, const Matrix& m, const char* what) {
  if (device != m.t->get_device())
    throw Fail{PyExc_ValueError, std::string(what) + " is on cuda:" + std::to_string(device) + ", the logits are on cuda:" +
                                     std::to_string(m.t->get_device())};
}
void on_device(const at::Tensor& t, const Matrix& m, const char* what) {
  if (!t.is_cuda()) throw Fail{PyExc_ValueError, std::string(what) + ": expected a CUDA tensor"};
  on_device(t.get_device(), m, what);
}

// The pointer of an optional contiguous device tensor of at least n entries.
template <typename T>
T* vec(PyObject* o, at::ScalarType type, const char* what, int64_t n, const Matrix& m) {
  if (!o) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != type)
    throw Fail{PyExc_TypeError, std::string(what) + " must be " + (type == at::kInt ? "int32" : "float32")};
  on_device(t, m, what);
  if (!t.is_contiguous()) throw Fail{PyExc_ValueError, std::string(what) + ": expected a contiguous tensor"};
  if (t.numel() < n)
    throw Fail{PyExc_ValueError,
               std::string(what) + " has " + std::to_string(t.numel()) + " entries, " + std::to_string(n) + " are needed"};
  return static_cast<T*>(t.data_ptr());
}
int32_t* i32(PyObject* o, const char* what, int64_t n, const Matrix& m) { return vec<int32_t>(o, at::kInt, what, n, m); }
float* f32(PyObject* o, const char* what, int64_t n, const Matrix& m) { return vec<float>(o, at::kFloat, what, n, m); }

// An output: the caller's tensor (checked), or a new one, made once the call's
// device and stream are current.
struct Output {
  PyObject* given = nullptr;
  at::Tensor made;
  void* p = nullptr;
  int64_t stride = 0;
  c10::SmallVector<int64_t, 2> shape;  // of a new one
  at::ScalarType type = at::kFloat;
  void make(const Matrix& m) {
    if (given) return;
    // without a turn through the dispatcher; the logits' device is the current one
    made = at::detail::empty_generic(shape, c10::cuda::CUDACachingAllocator::get(),
                                     c10::DispatchKeySet(c10::DispatchKey::CUDA), type, std::nullopt);
    p = made.data_ptr();
  }
  // A new reference.  To autograd a caller's tensor has been written in place: a
  // graph that saved it says so in its backward pass.  Inference tensors have no
  // version, and no graph can have saved one.
  PyObject* take() {
    if (!given) return THPVariable_Wrap(std::move(made));
    const at::Tensor& t = THPVariable_Unpack(given);
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    Py_INCREF(given);
    return given;
  }
};
Output out_matrix(PyObject* o, const Matrix& m, int64_t n, const char* what) {
  Output r;
  if (!o) {
    r.shape = {n, m.vocab};
    r.type = m.t->scalar_type();
    r.stride = m.vocab;
    return r;
  }
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != m.t->scalar_type() || t.dim() != 2 || t.size(0) < n || t.size(1) != m.vocab)
    throw Fail{PyExc_ValueError, std::string(what) + " must be [" + std::to_string(n) + ", " + std::to_string(m.vocab) +
                                     "] of the logits' type"};
  if (t.stride(1) != 1) throw Fail{PyExc_ValueError, std::string(what) + "'s rows must be contiguous (stride(1) == 1)"};
  on_device(t, m, what);
  r.given = o;
  r.p = t.data_ptr();
  r.stride = t.size(0) <= 1 && t.stride(0) < m.vocab ? m.vocab : t.stride(0);
  return r;
}
Output out_vec(PyObject* o, const Matrix& m, at::IntArrayRef shape, at::ScalarType type, const char* what) {
  Output r;
  if (o) {
    r.p = vec<void>(o, type, what, c10::multiply_integers(shape), m);
    r.given = o;
  } else {
    r.shape.assign(shape.begin(), shape.end());
    r.type = type;
  }
  return r;
}

// The stream a call runs on: the caller's (made current, so that outputs are
// allocated on it), or the current one of the logits' device.  That device is
// the current one while this lives: launches and device attributes follow it.
struct OnStream {
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* raw;
  OnStream(PyObject* o, const Matrix& m) {
    if (o) {
      auto attr = [&](const char* name) {
        PyObject* v = PyObject_GetAttrString(o, name);
        if (!v) {
          PyErr_Clear();
          throw Fail{PyExc_TypeError, "stream must be a torch.cuda.Stream"};
        }
        const long long r = PyLong_AsLongLong(v);
        Py_DECREF(v);
        return r;
      };
      on_device(attr("device_index"), m, "stream");
      guard.emplace(c10::cuda::CUDAStream::unpack3(attr("stream_id"), m.t->device().index(),
                                                   (c10::DeviceType)attr("device_type")));
    } else if (c10::cuda::current_device() != m.t->get_device()) {
      device.emplace(m.t->device());
    }
    raw = (void*)c10::cuda::getCurrentCUDAStream(m.t->get_device()).stream();
  }
};

// Runs a C call without the GIL; its failure becomes LSError.
template <typename F>
void call(const char* what, F f) {
  ls_status st;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  Py_END_ALLOW_THREADS;
  if (st == LS_OK) return;
  PyObject* args = Py_BuildValue("(is)", (int)st, what);
  PyObject* e = args ? PyObject_CallObject(ls_error, args) : nullptr;
  Py_XDECREF(args);
  if (e) {
    PyErr_SetObject(ls_error, e);
    Py_DECREF(e);
  }
  throw Fail{nullptr, ""};
}

template <typename F>
PyObject* entry(F f) {
  HANDLE_TH_ERRORS
  try {
    if (!ls_error) throw Fail{PyExc_RuntimeError, "the library is not bound"};
    return f();
  } catch (const Fail& e) {
    if (e.type) PyErr_SetString(e.type, e.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* pair(Output& a, Output& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, a.take());
  PyTuple_SET_ITEM(r, 1, b.take());
  return r;
}

}  // namespace
