// ls_tokens.cu -- the operators of include/ls_token_ops.h: log-probs of given
// tokens, the policy loss and the preference loss, with their gradients.
//
// token_kernel: a CTA per row streams it once for its maximum, sum and entropy
// term, works out the operator's scalars and, in the call that gives loss and
// gradient, reads the row again.  pair_kernel: a CTA per pair of answers sums
// their rows' terms and leaves each row's slope.  token_backward_kernel: one sweep
// over the logits with the two slopes that a forward call left of each row.
#include "ls_token_ops.cuh"

namespace lsg {
namespace ops {

constexpr int kTokenThreads = 256;

template <typename TIn, bool kEntropy, bool kGrad>
__global__ void __launch_bounds__(kTokenThreads, 4) token_kernel(const TokenArgs a, int upc) {
  constexpr int T = kTokenThreads;
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  constexpr int kFirst = kGrad ? LOAD_KEEP : LOAD_ONCE;
  __shared__ Moments red[T / 32];
  __shared__ TokenStats sh;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x;
  wait_for_previous();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, 0);
  Raw* grad = kGrad ? static_cast<Raw*>(a.out_grad) + i * a.grad_stride : nullptr;
  int32_t id;
  float w;
  if (!counts(a, i, id, w)) {
    if (kGrad) {
      const bool same = run.aligned_with(grad);
      uint32_t z[8] = {};
      for (int u = tid; u < run.n; u += T) run.store(grad, same, u, z);
    }
    if (tid == 0) skip_row(a, i);
    return;
  }
  typename Run<TIn, T>::Stage first;
  run.template prefetch<kFirst>(tid, first);
  const float x = guard(E::get(run.row[id]));
  const float c = kLog2e / a.temperature;
  RowSum<kEntropy> acc;
  Moments r;
  // NaN logits, without entropies: the first pass takes them as they come, and a
  // row whose sum is NaN is taken again with each of them read as -inf.
  bool dirty = false;
#pragma unroll 1
  for (;;) {
    acc.init(c);
    run.template stream<kFirst>(first, [&](int, typename Run<TIn, T>::Stage& v) {
      float um = kNegInf;
#pragma unroll
      for (int k = 0; k < kStage; ++k) {
        if (!kEntropy && dirty) Unit<TIn>::clean(v[k]);
        um = fmaxf(um, Unit<TIn>::max(v[k]));
      }
      acc.raise(um);
#pragma unroll
      for (int k = 0; k < kStage; ++k) acc.template add<TIn>(v[k]);
    });
    r = block_moments<T / 32, kEntropy>(acc.moments(), c, red);
    if (kEntropy || dirty || r.s == r.s) break;  // the same in every thread
    dirty = true;
    run.template prefetch<kFirst>(tid, first);
    __syncthreads();  // red is read
  }
  let_next_start();
  if (tid == 0) sh = finish_row(a, i, r, x, w, kEntropy);
  if (kGrad) {
    // From the row's end: what was read last is the likeliest to be in L2.
    run.template prefetch<LOAD_PLAIN>(run.last_stage(), first);
    __syncthreads();
    const uint32_t place = (uint32_t)run.place(id);
    RowGradient g;
    g.init(sh, sh.g_lp, sh.g_H, a.temperature);
    const bool same = run.aligned_with(grad);
    run.template stream_back<LOAD_PLAIN>(first, [&](int u, typename Run<TIn, T>::Stage& v) {
      const bool whole = run.whole(u) && same;
#pragma unroll
      for (int k = 0; k < kStage; ++k) {
        const int uk = u + k * T;
        g.template apply<TIn>(v[k], place - (uint32_t)uk * Unit<TIn>::kN);
        if (whole)
          store32(grad + run.index(uk), v[k]);
        else if (uk < run.n)
          run.store(grad, same, uk, v[k]);
      }
    });
  }
}

// The sums of a pair's two answers, its loss, and the slope of each of its rows.
constexpr int kPairThreads = 256;

struct PairArgs {
  ls_preference p;
  int32_t n;
  TokenStats* stats;
  float* out_loss;
  float* out_log_ratios;
  int32_t* error_word;
};

__global__ void __launch_bounds__(kPairThreads) pair_kernel(const PairArgs a) {
  constexpr int kW = kPairThreads / 32;
  __shared__ double red[4][kW];
  const int tid = threadIdx.x, lane = tid & 31;
  const int32_t p = (int32_t)blockIdx.x;
  wait_for_previous();
  let_next_start();
  const int32_t* at = a.p.answer_offsets + 2 * (int64_t)p;
  const int32_t lo = at[0], mid = at[1], hi = at[2];
  if (lo < 0 || mid < lo || hi < mid || hi > a.n) {
    if (tid == 0) {
      a.out_loss[p] = quiet_nan();
      if (a.out_log_ratios) a.out_log_ratios[2 * (int64_t)p] = a.out_log_ratios[2 * (int64_t)p + 1] = quiet_nan();
      if (a.error_word) atomicOr(a.error_word, LS_ROW_ERR_BAD_OFFSETS);
    }
    return;
  }
  double v[4] = {0.0, 0.0, 0.0, 0.0};  // sum and weight of the chosen, of the rejected answer
  for (int64_t i = lo + tid; i < hi; i += kPairThreads) {
    const float term = a.stats[i].term, w = a.stats[i].w;
    const bool first = i < mid;
    v[0] += first ? term : 0.f;
    v[1] += first ? w : 0.f;
    v[2] += first ? 0.f : term;
    v[3] += first ? 0.f : w;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[q] += __shfl_xor_sync(0xFFFFFFFFu, v[q], o);
    if (lane == 0) red[q][tid >> 5] = v[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = red[q][0];
#pragma unroll
    for (int k = 1; k < kW; ++k) v[q] += red[q][k];
  }
  float over[2] = {1.f, 1.f};
  if (a.p.average) {
    over[0] = v[1] != 0.0 ? (float)(1.0 / v[1]) : 0.f;
    over[1] = v[3] != 0.0 ? (float)(1.0 / v[3]) : 0.f;
    v[0] = v[1] != 0.0 ? v[0] / v[1] : 0.0;
    v[2] = v[3] != 0.0 ? v[2] / v[3] : 0.0;
  }
  const float u = (float)(v[0] - v[2]), beta = a.p.beta;
  const float h = (float)((double)beta * (v[0] - v[2]) - (double)a.p.margin);
  float loss, slope;  // of u
  if (a.p.kind == LS_PREFERENCE_SIGMOID) {
    const float e = a.p.label_smoothing, tail = log1pf(expf(-fabsf(h)));
    const float down = 1.f / (1.f + expf(h)), up = 1.f / (1.f + expf(-h));  // sigma(-h), sigma(h)
    loss = (1.f - e) * (fmaxf(-h, 0.f) + tail);
    if (e > 0.f) loss += e * (fmaxf(h, 0.f) + tail);
    slope = beta * (e * up - (1.f - e) * down);
    if (h != h) loss = slope = h;
  } else if (a.p.kind == LS_PREFERENCE_HINGE) {
    loss = h != h ? h : fmaxf(1.f - h, 0.f);
    slope = h != h ? h : h < 1.f ? -beta : 0.f;
  } else {
    const float d = u - 0.5f / beta;
    loss = d * d;
    slope = 2.f * d;
  }
  if (tid == 0) {
    a.out_loss[p] = loss;
    if (a.out_log_ratios) {
      a.out_log_ratios[2 * (int64_t)p] = (float)v[0];
      a.out_log_ratios[2 * (int64_t)p + 1] = (float)v[2];
    }
  }
  for (int64_t i = lo + tid; i < hi; i += kPairThreads) {
    const float w = a.stats[i].w;
    a.stats[i].g_lp = w == 0.f ? 0.f : i < mid ? slope * w * over[0] : -slope * w * over[1];
    a.stats[i].up = p;
  }
}

// The backward passes, in runs of a row.  In place (the gradient may replace the
// logits) each unit is read before the same thread writes it.
struct TokenBackArgs {
  const void* logits;
  int64_t vocab, row_stride;
  const int32_t* ids;
  float temperature;
  const TokenStats* stats;
  const float* up_lp;  // the gradient from above, by stats.up
  const float* up_H;
  int32_t ups;         // its entries
  float none_lp, none_H;  // where there is none
  void* out_grad;
  int64_t grad_stride;
};

constexpr int kTokenBackRun = 2048;  // units of a CTA's run

template <typename TIn>
__global__ void __launch_bounds__(kTokenThreads, 4) token_backward_kernel(const TokenBackArgs a, int runs, int upc) {
  constexpr int T = kTokenThreads;
  using Raw = typename Elem<TIn>::Raw;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)runs;
  wait_for_previous();
  let_next_start();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, (int)(blockIdx.x % (unsigned)runs));
  Raw* grad = static_cast<Raw*>(a.out_grad) + i * a.grad_stride;
  const bool same = run.aligned_with(grad);
  const float4* in = reinterpret_cast<const float4*>(a.stats + i);
  const float4 s0 = in[0], s1 = in[1];
  TokenStats st;
  st.M = s0.x;
  st.S = s0.y;
  st.H = s0.z;
  st.lp = s0.w;
  const int32_t up = __float_as_int(s1.z);
  const bool has = up >= 0 && up < a.ups;  // stats of another call do not lead out of bounds
  // a slope of 0 counts nothing, whatever the gradient from above
  const float g_lp = s1.x == 0.f ? 0.f : s1.x * (!a.up_lp ? a.none_lp : has ? a.up_lp[up] : quiet_nan());
  const float g_H = s1.y == 0.f ? 0.f : s1.y * (!a.up_H ? a.none_H : has ? a.up_H[up] : quiet_nan());
  if (g_lp == 0.f && g_H == 0.f) {
    uint32_t z[8] = {};
    for (int u = tid; u < run.n; u += T) run.store(grad, same, u, z);
    return;
  }
  typename Run<TIn, T>::Stage first;
  run.template prefetch<LOAD_PLAIN>(tid, first);
  const uint32_t place = (uint32_t)run.place(a.ids[i]);  // -1, past every unit, in another CTA's run
  RowGradient g;
  g.init(st, g_lp, g_H, a.temperature);
  run.template stream<LOAD_PLAIN>(first, [&](int u, typename Run<TIn, T>::Stage& v) {
    const bool whole = run.whole(u) && same;
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const int uk = u + k * T;
      g.template apply<TIn>(v[k], place - (uint32_t)uk * Unit<TIn>::kN);
      if (whole)
        store32(grad + run.index(uk), v[k]);
      else if (uk < run.n)
        run.store(grad, same, uk, v[k]);
    }
  });
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
template <bool kEntropy, bool kGrad>
static ls_status launch_tokens(const TokenArgs& a, ls_dtype dtype, cudaStream_t st) {
  const int upc = (int)row_units(a.vocab, dtype);
  const dim3 grid((unsigned)a.n);
  return dtype == LS_DTYPE_BF16
             ? launch_kernel(token_kernel<bf16_tag, kEntropy, kGrad>, grid, kTokenThreads, 1, 0, st, a, upc)
             : launch_kernel(token_kernel<float, kEntropy, kGrad>, grid, kTokenThreads, 1, 0, st, a, upc);
}

static ls_status forward(const TokenArgs& a, ls_dtype dtype, bool entropy, cudaStream_t st) {
  return entropy ? launch_tokens<true, false>(a, dtype, st) : launch_tokens<false, false>(a, dtype, st);
}

static ls_status backward(const TokenBackArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t units = row_units(a.vocab, dtype);
  const int sms = device_attr<cudaDevAttrMultiProcessorCount>();
  const int upc = (units + kTokenBackRun - 1) / kTokenBackRun * n >= 8 * sms ? kTokenBackRun : kTokenThreads * kStage;
  const int64_t runs = (units + upc - 1) / upc;
  if (runs * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(runs * n));
  return dtype == LS_DTYPE_BF16
             ? launch_kernel(token_backward_kernel<bf16_tag>, grid, kTokenThreads, 1, 0, st, a, (int)runs, upc)
             : launch_kernel(token_backward_kernel<float>, grid, kTokenThreads, 1, 0, st, a, (int)runs, upc);
}

static bool finite(float v) { return v - v == 0.f; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks that the calls share.
static bool rows_ok(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, const int32_t* ids,
                    float temperature) {
  return matrix_ok(logits, dtype, vocab, row_stride) && ids && temperature > 0.f && finite(temperature);
}
static bool policy_ok(const ls_policy* p) {
  return p && p->advantages && p->clip_low >= 0.f && p->clip_low <= 1.f && p->clip_high >= 0.f &&
         (p->dual_clip == 0.f || (p->dual_clip >= 1.f && finite(p->dual_clip))) && finite(p->kl_coef) &&
         (p->kl_coef == 0.f || p->ref_log_probs) && (p->kl == LS_KL_K1 || p->kl == LS_KL_K2 || p->kl == LS_KL_K3) &&
         finite(p->entropy_coef);
}
static bool preference_ok(const ls_preference* p) {
  if (!p || !p->answer_offsets || p->pairs < 0 || p->pairs >= 1 << 30 || !(p->beta > 0.f) || !finite(p->beta) ||
      !finite(p->margin))
    return false;
  if (p->kind != LS_PREFERENCE_SIGMOID && p->kind != LS_PREFERENCE_HINGE && p->kind != LS_PREFERENCE_IPO) return false;
  if (!(p->label_smoothing >= 0.f && p->label_smoothing <= 0.5f)) return false;
  return (p->kind == LS_PREFERENCE_SIGMOID || p->label_smoothing == 0.f) &&
         (p->kind != LS_PREFERENCE_IPO || p->margin == 0.f);
}
static bool grad_ok(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n, void* grad,
                    int64_t grad_stride) {
  return matrix_ok(grad, dtype, vocab, grad_stride) &&
         overlap_ok(logits, n, row_stride, grad, n, grad_stride, vocab, dtype, true);
}

static TokenArgs rows_of(const void* logits, int64_t vocab, int64_t row_stride, int32_t n, const int32_t* ids,
                         float temperature, TokenKind kind) {
  TokenArgs a = {};
  a.logits = logits;
  a.vocab = vocab;
  a.row_stride = row_stride;
  a.n = n;
  a.ids = ids;
  a.temperature = temperature;
  a.kind = kind;
  return a;
}

// The three backward calls: what stands for a missing gradient differs.
static ls_status backward_call(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                               const int32_t* ids, float temperature, const float* stats, const float* up_lp,
                               const float* up_H, int32_t ups, float none, void* out_grad, int64_t grad_stride, void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !stats || !aligned16(stats) ||
      !grad_ok(logits, dtype, vocab, row_stride, n, out_grad, grad_stride))
    return LS_ERR_INVALID_ARG;
  const TokenBackArgs a{logits, vocab, row_stride, ids,  temperature, reinterpret_cast<const TokenStats*>(stats),
                        up_lp,  up_H,  ups,        none, none,        out_grad,
                        grad_stride};
  return backward(a, dtype, n, stream);
}

}  // namespace ops
}  // namespace lsg

using namespace lsg;
using namespace lsg::ops;

extern "C" {

ls_status ls_token_log_probs(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                             const int32_t* ids, float temperature, float* out_log_probs, float* out_entropy,
                             float* out_stats, int32_t* error_word, void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !out_log_probs || !out_stats ||
      !aligned16(out_stats))
    return LS_ERR_INVALID_ARG;
  TokenArgs a = rows_of(logits, vocab, row_stride, n, ids, temperature, KIND_SCORE);
  a.out_loss = out_log_probs;
  a.out_entropy = out_entropy;
  a.out_stats = reinterpret_cast<TokenStats*>(out_stats);
  a.error_word = error_word;
  return forward(a, dtype, out_entropy != nullptr, static_cast<cudaStream_t>(stream));
}

ls_status ls_token_log_probs_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride,
                                      int32_t n, const int32_t* ids, float temperature, const float* stats,
                                      const float* grad_log_probs, const float* grad_entropy, void* out_grad,
                                      int64_t grad_stride, void* stream) {
  return backward_call(logits, dtype, vocab, row_stride, n, ids, temperature, stats, grad_log_probs, grad_entropy, n, 0.f,
                       out_grad, grad_stride, stream);
}

ls_status ls_policy_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                         const int32_t* ids, const ls_policy* policy, float temperature, float* out_loss,
                         float* out_metrics, float* out_stats, int32_t* error_word, void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !policy_ok(policy) || !out_loss || !out_stats ||
      !aligned16(out_stats) || !aligned16(out_metrics))
    return LS_ERR_INVALID_ARG;
  TokenArgs a = rows_of(logits, vocab, row_stride, n, ids, temperature, KIND_POLICY);
  a.policy = *policy;
  a.out_loss = out_loss;
  a.out_metrics = reinterpret_cast<float4*>(out_metrics);
  a.out_stats = reinterpret_cast<TokenStats*>(out_stats);
  a.error_word = error_word;
  return forward(a, dtype, policy->entropy || policy->entropy_coef != 0.f, static_cast<cudaStream_t>(stream));
}

ls_status ls_policy_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                  const int32_t* ids, float temperature, const float* stats, const float* grad_loss,
                                  void* out_grad, int64_t grad_stride, void* stream) {
  return backward_call(logits, dtype, vocab, row_stride, n, ids, temperature, stats, grad_loss, grad_loss, n, 1.f,
                       out_grad, grad_stride, stream);
}

ls_status ls_policy_loss_grad(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                              const int32_t* ids, const ls_policy* policy, float temperature, float* out_loss,
                              float* out_metrics, void* out_grad, int64_t grad_stride, int32_t* error_word,
                              void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !policy_ok(policy) || !out_loss ||
      !aligned16(out_metrics) || !grad_ok(logits, dtype, vocab, row_stride, n, out_grad, grad_stride))
    return LS_ERR_INVALID_ARG;
  TokenArgs a = rows_of(logits, vocab, row_stride, n, ids, temperature, KIND_POLICY);
  a.policy = *policy;
  a.out_loss = out_loss;
  a.out_metrics = reinterpret_cast<float4*>(out_metrics);
  a.out_grad = out_grad;
  a.grad_stride = grad_stride;
  a.error_word = error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return policy->entropy || policy->entropy_coef != 0.f ? launch_tokens<true, true>(a, dtype, st)
                                                        : launch_tokens<false, true>(a, dtype, st);
}

ls_status ls_preference_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                             const int32_t* ids, const ls_preference* preference, float temperature, float* out_loss,
                             float* out_log_ratios, float* out_stats, int32_t* error_word, void* stream) {
  if (n < 0 || !preference_ok(preference)) return LS_ERR_INVALID_ARG;
  if (preference->pairs > 0 && !out_loss) return LS_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n > 0) {
    if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !out_stats || !aligned16(out_stats))
      return LS_ERR_INVALID_ARG;
    TokenArgs a = rows_of(logits, vocab, row_stride, n, ids, temperature, KIND_PREFERENCE);
    a.policy.weights = preference->weights;
    a.policy.ref_log_probs = preference->ref_log_probs;
    a.offsets = preference->answer_offsets;
    a.pairs = preference->pairs;
    a.out_stats = reinterpret_cast<TokenStats*>(out_stats);
    a.error_word = error_word;
    const ls_status rc = forward(a, dtype, false, st);
    if (rc != LS_OK) return rc;
  }
  if (preference->pairs == 0) return LS_OK;
  const PairArgs p{*preference, n, reinterpret_cast<TokenStats*>(out_stats), out_loss, out_log_ratios, error_word};
  return launch_kernel(pair_kernel, dim3((unsigned)preference->pairs), kPairThreads, 1, 0, st, p);
}

ls_status ls_preference_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                      const int32_t* ids, float temperature, const float* stats, int32_t pairs,
                                      const float* grad_loss, void* out_grad, int64_t grad_stride, void* stream) {
  if (pairs < 0) return LS_ERR_INVALID_ARG;
  return backward_call(logits, dtype, vocab, row_stride, n, ids, temperature, stats, grad_loss, nullptr, pairs, 1.f,
                       out_grad, grad_stride, stream);
}

}  // extern "C"
