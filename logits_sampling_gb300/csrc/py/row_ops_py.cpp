// row_ops_py.cpp -- the Python calls of include/ls_row_ops.h, and the extension
// module: argument checks, allocation of outputs, one call of the C ABI.  No
// arithmetic.
//
// A small call's kernels take 3 to 8 us on the device; marshalled in Python
// the call took 11 to 15 us of host time, most of it checks and tensor
// properties.  The functions here are plain CPython (vectorcall) functions over
// torch's C++ tensors.  The C ABI's functions are those of the library that the
// package has loaded: their addresses are handed over once (bind).  The calls of
// include/ls_token_ops.h are in token_ops_py.h, what both share in ops_py.h.
#include "ls_row_ops.h"
#include "ops_py.h"
#include "token_ops_py.h"

namespace {

decltype(&ls_process_logits) f_process;
decltype(&ls_top_log_probs) f_top;
decltype(&ls_distill_loss) f_loss;
decltype(&ls_distill_loss_backward) f_backward;
decltype(&ls_distill_loss_grad) f_grad;
PyObject* s_marshalled;  // "_marshalled": the address of what a LogitsParams keeps

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

// bind(LSError, addresses of the C functions in the order of the headers)
PyObject* bind(PyObject*, PyObject* args) {
  void* const to[] = {&f_process, &f_top, &f_loss, &f_backward, &f_grad, &f_score, &f_score_backward, &f_policy,
                      &f_policy_backward, &f_policy_grad, &f_preference, &f_preference_backward};
  constexpr int kCount = sizeof(to) / sizeof(to[0]);
  if (PyTuple_GET_SIZE(args) != 1 + kCount) {
    PyErr_SetString(PyExc_TypeError, "bind() takes LSError and the address of each call");
    return nullptr;
  }
  void* p[kCount];
  for (int i = 0; i < kCount; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args, 1 + i));
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  for (int i = 0; i < kCount; ++i) memcpy(to[i], &p[i], sizeof(p[i]));
  ls_error = PyTuple_GET_ITEM(args, 0);
  Py_INCREF(ls_error);
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
    LS_CALL(token_log_probs, doc_score),
    LS_CALL(token_log_probs_backward, doc_score_backward),
    LS_CALL(policy_loss, doc_policy),
    LS_CALL(policy_loss_backward, doc_policy_backward),
    LS_CALL(policy_loss_grad, doc_policy_grad),
    LS_CALL(preference_loss, doc_preference),
    LS_CALL(preference_loss_backward, doc_preference_backward),
    {"bind", bind, METH_VARARGS, "bind(error, address of each call): the C functions"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_row_ops_c",
                      "The calls of include/ls_row_ops.h and include/ls_token_ops.h on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__row_ops_c() {
  s_marshalled = PyUnicode_InternFromString("_marshalled");
  for (Names* n : {&n_process, &n_top, &n_loss, &n_backward, &n_grad, &n_score, &n_score_backward, &n_policy,
                   &n_policy_backward, &n_policy_grad, &n_preference, &n_preference_backward})
    for (int i = 0; i < n->count; ++i) n->name[i] = PyUnicode_InternFromString(n->text[i]);
  return PyModule_Create(&module);
}
