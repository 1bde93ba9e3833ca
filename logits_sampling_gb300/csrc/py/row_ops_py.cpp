// row_ops_py.cpp -- the Python calls of include/ls_row_ops.h: argument checks,
// allocation of outputs, one call of the C ABI.  No arithmetic.
//
// A small call's kernels take 3 to 8 us on the device; marshalled in Python
// the call took 11 to 15 us of host time, most of it checks and tensor
// properties.  The functions here are plain CPython (vectorcall) functions over
// torch's C++ tensors.  The C ABI's functions are those of the library that the
// package has loaded: their addresses are handed over once (bind).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <string>

#include "ls_row_ops.h"

namespace {

decltype(&ls_process_logits) f_process;
decltype(&ls_top_log_probs) f_top;
decltype(&ls_distill_loss) f_loss;
decltype(&ls_distill_loss_backward) f_backward;
decltype(&ls_distill_loss_grad) f_grad;
PyObject* ls_error;      // the package's LSError(status, what)
PyObject* s_marshalled;  // "_marshalled": the address of what a LogitsParams keeps

// An error on its way to Python.
struct Fail {
  PyObject* type;
  std::string what;
};

// ---------------------------------------------------------------------------
// Arguments
// ---------------------------------------------------------------------------
constexpr int kMostArgs = 16;
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
    // without a turn through the dispatcher
    made = at::detail::empty_cuda(shape, type, m.t->device(), std::nullopt);
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

struct Teacher : ls_teacher {
  Teacher(PyObject* ids_, PyObject* log_probs_, int64_t n, const Matrix& m) {
    const at::Tensor& i = tensor(ids_, "teacher_ids");
    const at::Tensor& l = tensor(log_probs_, "teacher_log_probs");
    if (i.dim() != 2 || l.dim() != 2 || i.size(0) != n || l.size(0) != n || i.size(1) != l.size(1))
      throw Fail{PyExc_ValueError, "teacher_ids and teacher_log_probs must both be [" + std::to_string(n) + ", k]"};
    if (i.scalar_type() != at::kInt || l.scalar_type() != at::kFloat)
      throw Fail{PyExc_TypeError, "teacher_ids must be int32, teacher_log_probs float32"};
    k = count32(i.size(1), "k");
    if (k > 1 && (i.stride(1) != 1 || l.stride(1) != 1))
      throw Fail{PyExc_ValueError, "teacher_ids and teacher_log_probs must have contiguous rows"};
    if (n > 1 && i.stride(0) != l.stride(0))
      throw Fail{PyExc_ValueError, "teacher_ids and teacher_log_probs must have one row stride"};
    on_device(i, m, "teacher_ids");
    on_device(l, m, "teacher_log_probs");
    stride = n > 1 ? i.stride(0) : k;
    ids = static_cast<const int32_t*>(i.data_ptr());
    log_probs = static_cast<const float*>(l.data_ptr());
  }
};

// What a LogitsParams keeps at the address _marshalled (_Marshalled in _row_ops.py).
struct Marshalled {
  ls_logits_params params;
  int32_t device, count;  // the tensors' device and their number
  struct {
    const char* name;
    PyObject* tensor;
    const void* data;
    int64_t numel;
  } field[9];
};

// The struct of a LogitsParams.  It holds addresses, so a tensor that has been
// resized or given another storage since is refused.
const ls_logits_params* marshalled(PyObject* o, const Matrix& m) {
  if (!o) return nullptr;
  PyObject* address = PyObject_GetAttr(o, s_marshalled);
  const auto* p = address ? static_cast<const Marshalled*>(PyLong_AsVoidPtr(address)) : nullptr;
  Py_XDECREF(address);
  PyErr_Clear();
  if (!p) throw Fail{PyExc_TypeError, "params must be a LogitsParams"};
  on_device(p->device, m, "params");
  for (int q = 0; q < p->count; ++q) {
    const at::Tensor& t = THPVariable_Unpack(p->field[q].tensor);
    if (t.const_data_ptr() != p->field[q].data || t.numel() != p->field[q].numel)
      throw Fail{PyExc_ValueError, std::string("params' ") + p->field[q].name +
                                       " has been resized or given another storage: make a new LogitsParams"};
  }
  return &p->params;
}

ls_tail tail_of(PyObject* o) {
  if (!o) return LS_TAIL_BUCKET;
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "bucket") == 0) return LS_TAIL_BUCKET;
    if (PyUnicode_CompareWithASCIIString(o, "drop") == 0) return LS_TAIL_DROP;
    if (PyUnicode_CompareWithASCIIString(o, "renorm") == 0) return LS_TAIL_RENORM;
  }
  throw Fail{PyExc_ValueError, "tail must be one of ['bucket', 'drop', 'renorm']"};
}

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
    if (!f_process) throw Fail{PyExc_RuntimeError, "the library is not bound"};
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

// ---------------------------------------------------------------------------
// The calls
// ---------------------------------------------------------------------------
Names n_process = {"process_logits", 11, 1,
                   {"logits", "n", "params", "gather_indices", "token_to_request_index", "row_lens", "allowed_mask",
                    "mask_index", "out", "error_word", "stream"}};
PyObject* process_logits(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_process, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(o[1] ? integer(o[1], "n") : o[3] ? tensor(o[3], "gather_indices").numel() : m.rows, "n");
    const ls_logits_params* params = marshalled(o[2], m);
    const int32_t* mask = nullptr;
    int64_t mask_rows = 0, mask_stride = 0;
    if (o[6]) {
      const at::Tensor& t = tensor(o[6], "allowed_mask");
      if (t.dim() != 2 || t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
        throw Fail{PyExc_ValueError, "allowed_mask must be int32 [mask_rows, words] with contiguous rows"};
      on_device(t, m, "allowed_mask");
      mask = static_cast<const int32_t*>(t.data_ptr());
      mask_rows = t.size(0);
      mask_stride = mask_rows > 1 ? t.stride(0) : t.size(1);
    }
    const int32_t* gather = i32(o[3], "gather_indices", n, m);
    const int32_t* t2r = i32(o[4], "token_to_request_index", n, m);
    const int32_t* lens = i32(o[5], "row_lens", n, m);
    const int32_t* index = i32(o[7], "mask_index", n, m);
    int32_t* error = i32(o[9], "error_word", 1, m);
    Output out = out_matrix(o[8], m, n < 0 ? 0 : n, "out");
    const OnStream on(o[10], m);
    out.make(m);
    call("ls_process_logits", [&] {
      return f_process(m.p, m.dtype, m.rows, m.vocab, m.stride, n, gather, t2r, params, lens, mask, mask_rows,
                       mask_stride, index, out.p, out.stride, error, on.raw);
    });
    return out.take();
  });
}

Names n_top = {"top_log_probs", 10, 2,
               {"logits", "k", "n", "temperature", "gather_indices", "out_ids", "out_log_probs", "out_lse", "error_word",
                "stream"}};
PyObject* top_log_probs(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_top, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t k = count32(integer(o[1], "k"), "k");
    const int32_t n = count32(o[2] ? integer(o[2], "n") : o[4] ? tensor(o[4], "gather_indices").numel() : m.rows, "n");
    if (k < 1 || k > LS_MAX_TOP || n < 0)
      throw Fail{PyExc_ValueError, "k must lie in [1, " + std::to_string(LS_MAX_TOP) + "], n be 0 or more"};
    const float temperature = number(o[3], 1.f, "temperature");
    const int32_t* gather = i32(o[4], "gather_indices", n, m);
    int32_t* error = i32(o[8], "error_word", 1, m);
    Output ids = out_vec(o[5], m, {n, k}, at::kInt, "out_ids");
    Output lp = out_vec(o[6], m, {n, k}, at::kFloat, "out_log_probs");
    Output lse = out_vec(o[7], m, {n}, at::kFloat, "out_lse");
    const OnStream on(o[9], m);
    ids.make(m);
    lp.make(m);
    lse.make(m);
    call("ls_top_log_probs", [&] {
      return f_top(m.p, m.dtype, m.rows, m.vocab, m.stride, n, gather, k, temperature, static_cast<int32_t*>(ids.p),
                   static_cast<float*>(lp.p), static_cast<float*>(lse.p), error, on.raw);
    });
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, ids.take());
    PyTuple_SET_ITEM(r, 1, lp.take());
    PyTuple_SET_ITEM(r, 2, lse.take());
    return r;
  });
}

Names n_loss = {"distill_loss", 10, 3,
                {"logits", "teacher_ids", "teacher_log_probs", "temperature", "tail", "weights", "out", "out_stats",
                 "error_word", "stream"}};
PyObject* distill_loss(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_loss, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const Teacher teacher(o[1], o[2], n, m);
    const float temperature = number(o[3], 1.f, "temperature");
    const ls_tail tail = tail_of(o[4]);
    const float* weights = f32(o[5], "weights", n, m);
    int32_t* error = i32(o[8], "error_word", 1, m);
    Output loss = out_vec(o[6], m, {n}, at::kFloat, "out");
    Output stats = out_vec(o[7], m, {n, LS_DISTILL_STATS}, at::kFloat, "out_stats");
    const OnStream on(o[9], m);
    loss.make(m);
    stats.make(m);
    call("ls_distill_loss", [&] {
      return f_loss(m.p, m.dtype, m.vocab, m.stride, n, &teacher, temperature, tail, weights,
                    static_cast<float*>(loss.p), static_cast<float*>(stats.p), error, on.raw);
    });
    return pair(loss, stats);
  });
}

Names n_backward = {"distill_loss_backward", 10, 4,
                    {"logits", "teacher_ids", "teacher_log_probs", "stats", "grad_loss", "temperature", "tail", "weights",
                     "out", "stream"}};
PyObject* distill_loss_backward(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_backward, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const Teacher teacher(o[1], o[2], n, m);
    const float* stats = f32(o[3], "stats", (int64_t)n * LS_DISTILL_STATS, m);
    const float* grad_loss = f32(o[4], "grad_loss", n, m);
    const float temperature = number(o[5], 1.f, "temperature");
    const ls_tail tail = tail_of(o[6]);
    const float* weights = f32(o[7], "weights", n, m);
    Output grad = out_matrix(o[8], m, n, "out");
    const OnStream on(o[9], m);
    grad.make(m);
    call("ls_distill_loss_backward", [&] {
      return f_backward(m.p, m.dtype, m.vocab, m.stride, n, &teacher, temperature, tail, weights, stats, grad_loss,
                        grad.p, grad.stride, on.raw);
    });
    return grad.take();
  });
}

Names n_grad = {"distill_loss_grad", 10, 3,
                {"logits", "teacher_ids", "teacher_log_probs", "temperature", "tail", "weights", "out_loss", "out_grad",
                 "error_word", "stream"}};
PyObject* distill_loss_grad(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_grad, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const Teacher teacher(o[1], o[2], n, m);
    const float temperature = number(o[3], 1.f, "temperature");
    const ls_tail tail = tail_of(o[4]);
    const float* weights = f32(o[5], "weights", n, m);
    int32_t* error = i32(o[8], "error_word", 1, m);
    Output loss = out_vec(o[6], m, {n}, at::kFloat, "out_loss");
    Output grad = out_matrix(o[7], m, n, "out_grad");
    const OnStream on(o[9], m);
    loss.make(m);
    grad.make(m);
    call("ls_distill_loss_grad", [&] {
      return f_grad(m.p, m.dtype, m.vocab, m.stride, n, &teacher, temperature, tail, weights,
                    static_cast<float*>(loss.p), grad.p, grad.stride, error, on.raw);
    });
    return pair(loss, grad);
  });
}

// bind(LSError, addresses of the five C functions in the order of the header)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *err, *a[5];
  if (!PyArg_ParseTuple(args, "OOOOOO", &err, &a[0], &a[1], &a[2], &a[3], &a[4])) return nullptr;
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(err);
  ls_error = err;
  f_process = reinterpret_cast<decltype(f_process)>(p[0]);
  f_top = reinterpret_cast<decltype(f_top)>(p[1]);
  f_loss = reinterpret_cast<decltype(f_loss)>(p[2]);
  f_backward = reinterpret_cast<decltype(f_backward)>(p[3]);
  f_grad = reinterpret_cast<decltype(f_grad)>(p[4]);
  Py_RETURN_NONE;
}

#define LS_CALL(f, doc) \
  {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL | METH_KEYWORDS, doc}
PyMethodDef methods[] = {
    LS_CALL(process_logits,
            "process_logits(logits, n=None, params=None, gather_indices=None, token_to_request_index=None, row_lens=None,\n"
            "               allowed_mask=None, mask_index=None, out=None, error_word=None, stream=None) -> out\n\n"
            "ls_process_logits: penalties, biases (params, a LogitsParams) and masks (allowed_mask int32 [mask_rows,\n"
            ">= ceil(vocab / 32)]) on n logits rows.  Returns out, [n, vocab] of the logits' type; out may be the logits\n"
            "themselves (no gather_indices)."),
    LS_CALL(top_log_probs,
            "top_log_probs(logits, k, n=None, temperature=1.0, gather_indices=None, out_ids=None, out_log_probs=None,\n"
            "              out_lse=None, error_word=None, stream=None) -> (ids, log_probs, lse)\n\n"
            "ls_top_log_probs: the k best ids (int32 [n, k]) of each row, their log-probs (float32 [n, k]) and the row's\n"
            "log-sum-exp (float32 [n])."),
    LS_CALL(distill_loss,
            "distill_loss(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail='bucket', weights=None, out=None,\n"
            "             out_stats=None, error_word=None, stream=None) -> (loss, stats)\n\n"
            "ls_distill_loss: the loss per row (float32 [n]) and what distill_loss_backward needs (float32 [n, 8])."),
    LS_CALL(distill_loss_backward,
            "distill_loss_backward(logits, teacher_ids, teacher_log_probs, stats, grad_loss=None, temperature=1.0,\n"
            "                      tail='bucket', weights=None, out=None, stream=None) -> out\n\n"
            "ls_distill_loss_backward: the gradient, [n, vocab] of the logits' type; out may be the logits themselves."),
    LS_CALL(distill_loss_grad,
            "distill_loss_grad(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail='bucket', weights=None,\n"
            "                  out_loss=None, out_grad=None, error_word=None, stream=None) -> (loss, grad)\n\n"
            "ls_distill_loss_grad: loss (float32 [n]) and gradient ([n, vocab] of the logits' type) from one call; out_grad\n"
            "may be the logits themselves."),
    {"bind", bind, METH_VARARGS, "bind(error, process, top, loss, backward, grad): the C functions' addresses"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_row_ops_c", "The calls of include/ls_row_ops.h on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__row_ops_c() {
  s_marshalled = PyUnicode_InternFromString("_marshalled");
  for (Names* n : {&n_process, &n_top, &n_loss, &n_backward, &n_grad})
    for (int i = 0; i < n->count; ++i) n->name[i] = PyUnicode_InternFromString(n->text[i]);
  return PyModule_Create(&module);
}
