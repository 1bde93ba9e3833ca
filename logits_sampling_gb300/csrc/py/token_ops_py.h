// token_ops_py.h -- the Python calls of include/ls_token_ops.h: argument checks,
// allocation of outputs, one call of the C ABI.  No arithmetic.
#pragma once

#include "ls_token_ops.h"
#include "ops_py.h"

namespace {

decltype(&ls_token_log_probs) f_score;
decltype(&ls_token_log_probs_backward) f_score_backward;
decltype(&ls_policy_loss) f_policy;
decltype(&ls_policy_loss_backward) f_policy_backward;
decltype(&ls_policy_loss_grad) f_policy_grad;
decltype(&ls_preference_loss) f_preference;
decltype(&ls_preference_loss_backward) f_preference_backward;

// The position of a text in a list; Fail when it is none of them.
int choice(PyObject* o, int otherwise, const char* what, const char* const* names, int count) {
  if (!o) return otherwise;
  std::string all;
  for (int i = 0; i < count; ++i) {
    if (PyUnicode_Check(o) && PyUnicode_CompareWithASCIIString(o, names[i]) == 0) return i;
    all += std::string(i ? ", '" : "'") + names[i] + "'";
  }
  throw Fail{PyExc_ValueError, std::string(what) + " must be one of [" + all + "]"};
}

bool truth(PyObject* o) {
  const int v = o ? PyObject_IsTrue(o) : 0;
  if (v < 0) {
    PyErr_Clear();
    throw Fail{PyExc_TypeError, "expected a truth value"};
  }
  return v != 0;
}

const int32_t* token_ids(PyObject* o, int32_t n, const Matrix& m) {
  const int32_t* ids = i32(o, "ids", n, m);
  if (tensor(o, "ids").numel() != n) throw Fail{PyExc_ValueError, "ids must have one entry per row of logits"};
  return ids;
}

PyObject* triple(Output& a, Output& b, Output& c) {
  PyObject* r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, a.take());
  PyTuple_SET_ITEM(r, 1, b.take());
  PyTuple_SET_ITEM(r, 2, c.take());
  return r;
}

Names n_score = {"token_log_probs", 9, 2,
                 {"logits", "ids", "temperature", "entropy", "out", "out_entropy", "out_stats", "error_word", "stream"}};
PyObject* token_log_probs(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_score, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const int32_t* ids = token_ids(o[1], n, m);
    const float temperature = number(o[2], 1.f, "temperature");
    const bool entropy = truth(o[3]) || o[5];
    int32_t* error = i32(o[7], "error_word", 1, m);
    Output lp = out_vec(o[4], m, {n}, at::kFloat, "out");
    Output h = entropy ? out_vec(o[5], m, {n}, at::kFloat, "out_entropy") : Output();
    Output stats = out_vec(o[6], m, {n, LS_TOKEN_STATS}, at::kFloat, "out_stats");
    const OnStream on(o[8], m);
    lp.make(m);
    if (entropy) h.make(m);
    stats.make(m);
    call("ls_token_log_probs", [&] {
      return f_score(m.p, m.dtype, m.vocab, m.stride, n, ids, temperature, static_cast<float*>(lp.p),
                     static_cast<float*>(h.p), static_cast<float*>(stats.p), error, on.raw);
    });
    PyObject* r = PyTuple_New(3);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, lp.take());
    if (!entropy) Py_INCREF(Py_None);
    PyTuple_SET_ITEM(r, 1, entropy ? h.take() : Py_None);
    PyTuple_SET_ITEM(r, 2, stats.take());
    return r;
  });
}
constexpr const char* doc_score =
    "token_log_probs(logits, ids, temperature=1.0, entropy=False, out=None, out_entropy=None, out_stats=None,\n"
    "                error_word=None, stream=None) -> (log_probs, entropy, stats)\n\n"
    "ls_token_log_probs: the log-prob of token ids[i] (int32 [n]) under each row (float32 [n]), the row's entropy\n"
    "(float32 [n], None unless asked for) and what token_log_probs_backward needs (float32 [n, 12]).";

Names n_score_backward = {"token_log_probs_backward", 8, 3,
                          {"logits", "ids", "stats", "grad_log_probs", "grad_entropy", "temperature", "out", "stream"}};
PyObject* token_log_probs_backward(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_score_backward, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const int32_t* ids = token_ids(o[1], n, m);
    const float* stats = f32(o[2], "stats", (int64_t)n * LS_TOKEN_STATS, m);
    const float* g_lp = f32(o[3], "grad_log_probs", n, m);
    const float* g_H = f32(o[4], "grad_entropy", n, m);
    const float temperature = number(o[5], 1.f, "temperature");
    Output grad = out_matrix(o[6], m, n, "out");
    const OnStream on(o[7], m);
    grad.make(m);
    call("ls_token_log_probs_backward", [&] {
      return f_score_backward(m.p, m.dtype, m.vocab, m.stride, n, ids, temperature, stats, g_lp, g_H, grad.p, grad.stride,
                              on.raw);
    });
    return grad.take();
  });
}
constexpr const char* doc_score_backward =
    "token_log_probs_backward(logits, ids, stats, grad_log_probs=None, grad_entropy=None, temperature=1.0, out=None,\n"
    "                         stream=None) -> out\n\n"
    "ls_token_log_probs_backward: the gradient, [n, vocab] of the logits' type; out may be the logits themselves.";

// The arguments that policy_loss and policy_loss_grad share: logits, ids, advantages, then these from place 3 on.
#define POLICY_NAMES                                                                                                 \
  "logits", "ids", "advantages", "old_log_probs", "ref_log_probs", "weights", "temperature", "clip_low", "clip_high", \
      "dual_clip", "kl_coef", "kl", "entropy_coef", "entropy"
struct Policy : ls_policy {
  float temperature;
  Policy(PyObject* const* o, int32_t n, const Matrix& m) {
    static const char* const kinds[] = {"k1", "k2", "k3"};
    advantages = f32(o[2], "advantages", n, m);
    old_log_probs = f32(o[3], "old_log_probs", n, m);
    ref_log_probs = f32(o[4], "ref_log_probs", n, m);
    weights = f32(o[5], "weights", n, m);
    temperature = number(o[6], 1.f, "temperature");
    clip_low = number(o[7], 0.2f, "clip_low");
    clip_high = number(o[8], 0.2f, "clip_high");
    dual_clip = number(o[9], 0.f, "dual_clip");
    kl_coef = number(o[10], 0.f, "kl_coef");
    kl = (ls_kl)choice(o[11], LS_KL_K3, "kl", kinds, 3);
    entropy_coef = number(o[12], 0.f, "entropy_coef");
    entropy = truth(o[13]);
  }
};

Names n_policy = {"policy_loss", 19, 3, {POLICY_NAMES, "out", "out_metrics", "out_stats", "error_word", "stream"}};
PyObject* policy_loss(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_policy, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const int32_t* ids = token_ids(o[1], n, m);
    const Policy policy(o, n, m);
    int32_t* error = i32(o[17], "error_word", 1, m);
    Output loss = out_vec(o[14], m, {n}, at::kFloat, "out");
    Output metrics = out_vec(o[15], m, {n, LS_POLICY_METRICS}, at::kFloat, "out_metrics");
    Output stats = out_vec(o[16], m, {n, LS_TOKEN_STATS}, at::kFloat, "out_stats");
    const OnStream on(o[18], m);
    loss.make(m);
    metrics.make(m);
    stats.make(m);
    call("ls_policy_loss", [&] {
      return f_policy(m.p, m.dtype, m.vocab, m.stride, n, ids, &policy, policy.temperature, static_cast<float*>(loss.p),
                      static_cast<float*>(metrics.p), static_cast<float*>(stats.p), error, on.raw);
    });
    return triple(loss, metrics, stats);
  });
}
constexpr const char* doc_policy =
    "policy_loss(logits, ids, advantages, old_log_probs=None, ref_log_probs=None, weights=None, temperature=1.0,\n"
    "            clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl='k3', entropy_coef=0.0, entropy=False,\n"
    "            out=None, out_metrics=None, out_stats=None, error_word=None, stream=None) -> (loss, metrics, stats)\n\n"
    "ls_policy_loss: the loss per row (float32 [n]), its metrics (float32 [n, 4]: log-prob, entropy, KL, ratio) and\n"
    "what policy_loss_backward needs (float32 [n, 12]).";

Names n_policy_backward = {"policy_loss_backward", 7, 3,
                           {"logits", "ids", "stats", "grad_loss", "temperature", "out", "stream"}};
Names n_preference_backward = {"preference_loss_backward", 7, 3,
                               {"logits", "ids", "stats", "grad_loss", "temperature", "out", "stream"}};
// Both backward calls: f(what they share, grad_loss and its entries, the output).
struct Back {
  Matrix m;
  int32_t n;
  const int32_t* ids;
  const float *stats, *grad_loss;
  int32_t entries;
  float temperature;
};
template <typename F>
PyObject* loss_backward(const Names& names, const char* what, bool per_row, PyObject* const* args, Py_ssize_t positional,
                        PyObject* keywords, F f) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(names, args, positional, keywords, o);
    Back b;
    b.m = matrix(o[0]);
    b.n = count32(b.m.rows, "rows");
    b.ids = token_ids(o[1], b.n, b.m);
    b.stats = f32(o[2], "stats", (int64_t)b.n * LS_TOKEN_STATS, b.m);
    b.grad_loss = f32(o[3], "grad_loss", per_row ? b.n : 0, b.m);
    b.entries = o[3] ? count32(tensor(o[3], "grad_loss").numel(), "grad_loss") : 0;
    if (o[3] && !b.entries) b.grad_loss = b.stats;  // it has no address and none of it is read, but it is not missing
    b.temperature = number(o[4], 1.f, "temperature");
    Output grad = out_matrix(o[5], b.m, b.n, "out");
    const OnStream on(o[6], b.m);
    grad.make(b.m);
    call(what, [&] { return f(b, grad, on.raw); });
    return grad.take();
  });
}
PyObject* policy_loss_backward(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return loss_backward(n_policy_backward, "ls_policy_loss_backward", true, args, positional, keywords,
                       [](const Back& b, const Output& grad, void* stream) {
                         return f_policy_backward(b.m.p, b.m.dtype, b.m.vocab, b.m.stride, b.n, b.ids, b.temperature,
                                                  b.stats, b.grad_loss, grad.p, grad.stride, stream);
                       });
}
PyObject* preference_loss_backward(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return loss_backward(n_preference_backward, "ls_preference_loss_backward", false, args, positional, keywords,
                       [](const Back& b, const Output& grad, void* stream) {
                         return f_preference_backward(b.m.p, b.m.dtype, b.m.vocab, b.m.stride, b.n, b.ids, b.temperature,
                                                      b.stats, b.entries, b.grad_loss, grad.p, grad.stride, stream);
                       });
}
constexpr const char* doc_policy_backward =
    "policy_loss_backward(logits, ids, stats, grad_loss=None, temperature=1.0, out=None, stream=None) -> out\n\n"
    "ls_policy_loss_backward: the gradient, [n, vocab] of the logits' type; out may be the logits themselves.";
constexpr const char* doc_preference_backward =
    "preference_loss_backward(logits, ids, stats, grad_loss=None, temperature=1.0, out=None, stream=None) -> out\n\n"
    "ls_preference_loss_backward: the gradient, [n, vocab] of the logits' type; grad_loss has an entry per pair; out may\n"
    "be the logits themselves.";

Names n_policy_grad = {"policy_loss_grad", 19, 3,
                       {POLICY_NAMES, "out_loss", "out_grad", "out_metrics", "error_word", "stream"}};
PyObject* policy_loss_grad(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    PyObject* o[kMostArgs];
    parse(n_policy_grad, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const int32_t* ids = token_ids(o[1], n, m);
    const Policy policy(o, n, m);
    int32_t* error = i32(o[17], "error_word", 1, m);
    Output loss = out_vec(o[14], m, {n}, at::kFloat, "out_loss");
    Output grad = out_matrix(o[15], m, n, "out_grad");
    Output metrics = out_vec(o[16], m, {n, LS_POLICY_METRICS}, at::kFloat, "out_metrics");
    const OnStream on(o[18], m);
    loss.make(m);
    grad.make(m);
    metrics.make(m);
    call("ls_policy_loss_grad", [&] {
      return f_policy_grad(m.p, m.dtype, m.vocab, m.stride, n, ids, &policy, policy.temperature,
                           static_cast<float*>(loss.p), static_cast<float*>(metrics.p), grad.p, grad.stride, error, on.raw);
    });
    return triple(loss, grad, metrics);
  });
}
constexpr const char* doc_policy_grad =
    "policy_loss_grad(logits, ids, advantages, old_log_probs=None, ref_log_probs=None, weights=None, temperature=1.0,\n"
    "                 clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl='k3', entropy_coef=0.0,\n"
    "                 entropy=False, out_loss=None, out_grad=None, out_metrics=None, error_word=None, stream=None)\n"
    "    -> (loss, grad, metrics)\n\n"
    "ls_policy_loss_grad: loss (float32 [n]), gradient ([n, vocab] of the logits' type) and metrics (float32 [n, 4]) from\n"
    "one call; out_grad may be the logits themselves.";

Names n_preference = {"preference_loss", 16, 3,
                      {"logits", "ids", "answer_offsets", "ref_log_probs", "weights", "temperature", "beta", "loss",
                       "label_smoothing", "margin", "average", "out", "out_log_ratios", "out_stats", "error_word",
                       "stream"}};
PyObject* preference_loss(PyObject*, PyObject* const* args, Py_ssize_t positional, PyObject* keywords) {
  return entry([&]() -> PyObject* {
    static const char* const kinds[] = {"sigmoid", "hinge", "ipo"};
    PyObject* o[kMostArgs];
    parse(n_preference, args, positional, keywords, o);
    const Matrix m = matrix(o[0]);
    const int32_t n = count32(m.rows, "rows");
    const int32_t* ids = token_ids(o[1], n, m);
    ls_preference p;
    p.answer_offsets = i32(o[2], "answer_offsets", 1, m);
    const int64_t answers = tensor(o[2], "answer_offsets").numel() - 1;
    if (answers % 2) throw Fail{PyExc_ValueError, "answer_offsets must have 2 * pairs + 1 entries"};
    p.pairs = count32(answers / 2, "pairs");
    p.ref_log_probs = f32(o[3], "ref_log_probs", n, m);
    p.weights = f32(o[4], "weights", n, m);
    const float temperature = number(o[5], 1.f, "temperature");
    p.beta = number(o[6], 0.1f, "beta");
    p.kind = (ls_preference_kind)choice(o[7], LS_PREFERENCE_SIGMOID, "loss", kinds, 3);
    p.label_smoothing = number(o[8], 0.f, "label_smoothing");
    p.margin = number(o[9], 0.f, "margin");
    p.average = truth(o[10]);
    int32_t* error = i32(o[14], "error_word", 1, m);
    Output loss = out_vec(o[11], m, {p.pairs}, at::kFloat, "out");
    Output ratios = out_vec(o[12], m, {answers}, at::kFloat, "out_log_ratios");
    Output stats = out_vec(o[13], m, {n, LS_TOKEN_STATS}, at::kFloat, "out_stats");
    const OnStream on(o[15], m);
    loss.make(m);
    ratios.make(m);
    stats.make(m);
    call("ls_preference_loss", [&] {
      return f_preference(m.p, m.dtype, m.vocab, m.stride, n, ids, &p, temperature, static_cast<float*>(loss.p),
                          static_cast<float*>(ratios.p), static_cast<float*>(stats.p), error, on.raw);
    });
    return triple(loss, ratios, stats);
  });
}
constexpr const char* doc_preference =
    "preference_loss(logits, ids, answer_offsets, ref_log_probs=None, weights=None, temperature=1.0, beta=0.1,\n"
    "                loss='sigmoid', label_smoothing=0.0, margin=0.0, average=False, out=None, out_log_ratios=None,\n"
    "                out_stats=None, error_word=None, stream=None) -> (loss, log_ratios, stats)\n\n"
    "ls_preference_loss: the loss per pair (float32 [pairs]), the log-ratio of each answer (float32 [2 * pairs], chosen\n"
    "and rejected in turn) and what preference_loss_backward needs (float32 [n, 12]).  answer_offsets int32\n"
    "[2 * pairs + 1]: pair p's chosen answer are the rows [offsets[2p], offsets[2p + 1]), its rejected one those up to\n"
    "offsets[2p + 2].";

}  // namespace
