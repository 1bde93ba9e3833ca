/*
 * ls_token_ops.h -- C ABI of the operators that train on sampled tokens (part
 * of libls_sampler.so; statuses, dtypes and row errors are those of
 * ls_sampler.h):
 *
 *   ls_token_log_probs            log-probs of given tokens (and entropies) of
 *   ls_token_log_probs_backward   logits rows: what a sampling policy and a
 *                                 reference model think of a rollout
 *   ls_policy_loss                the clipped policy loss with a KL term and an
 *   ls_policy_loss_backward       entropy bonus, its gradient, or both from one
 *   ls_policy_loss_grad           call
 *   ls_preference_loss            the preference loss of pairs of answers and
 *   ls_preference_loss_backward   its gradient
 *
 * Every call is asynchronous on the caller's stream, allocates nothing and
 * never synchronises with the host.  Buffers are device memory owned by the
 * caller; parameter structs are small host structs of device pointers and
 * numbers.  The same inputs, at the same alignment, give the same bits.
 *
 * Row i of n reads x = logits row i and token ids[i].  With z = x / temperature:
 *   q  = softmax(z)          lp = ln q[ids[i]]          H = -sum_j q_j ln q_j
 * All in fp32.  NaN logits are read as -inf; -inf entries have q = 0 and add
 * nothing to H; a row with +inf entries shares its mass equally among them.
 *
 * A row does not count where ids[i] lies outside [0, vocab) (padding, rejected
 * drafts), where weights[i] is 0, and, in the preference loss, outside the
 * answers: whatever it holds, its outputs are 0, and its gradient is 0 whatever
 * the gradient from above holds.  A row that counts and has no entry above -inf
 * gives NaN and sets LS_ROW_ERR_NO_FINITE in *error_word.
 */
#ifndef LS_TOKEN_OPS_H
#define LS_TOKEN_OPS_H

#include "ls_sampler.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more row error: answer_offsets descend or leave [0, n]. */
enum { LS_ROW_ERR_BAD_OFFSETS = 16 };

/* Floats per row that the losses leave for their backward passes. */
#define LS_TOKEN_STATS 12
/* Floats per row of a policy loss's metrics: lp, H (0 unless it was asked for), the KL estimate, the ratio. */
#define LS_POLICY_METRICS 4

/*
 * ls_token_log_probs -- out_log_probs[i] = lp, out_entropy[i] = H.
 *
 *   ids            device int32[n]
 *   temperature    finite, > 0, and with log2(e) / temperature finite (4.3e-39 and more)
 *   out_log_probs  device float[n]
 *   out_entropy    device float[n], or NULL: no entropies
 *   out_stats      device float[LS_TOKEN_STATS * n], 16-byte aligned: what the
 *                  backward pass needs
 */
ls_status ls_token_log_probs(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                             const int32_t* ids, float temperature, float* out_log_probs, float* out_entropy,
                             float* out_stats, int32_t* error_word, void* stream);

/*
 * ls_token_log_probs_backward -- the gradient of
 * sum_i grad_log_probs[i] * lp_i + grad_entropy[i] * H_i:
 *   d/dx_j = (g_lp * ([j = ids[i]] - q_j) - g_H * q_j * (ln q_j + H)) / temperature
 *
 *   stats           what ls_token_log_probs wrote for the same inputs (with
 *                   entropies, where grad_entropy is given)
 *   grad_log_probs,
 *   grad_entropy    device float[n] or NULL (0)
 *   out_grad        n x grad_stride elements of the logits' dtype; may be the
 *                   logits themselves (grad_stride == row_stride); any other
 *                   overlap is refused
 */
ls_status ls_token_log_probs_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride,
                                      int32_t n, const int32_t* ids, float temperature, const float* stats,
                                      const float* grad_log_probs, const float* grad_entropy, void* out_grad,
                                      int64_t grad_stride, void* stream);

/* Estimates of KL(policy || reference) from one token, d = ref - lp. */
typedef enum {
  LS_KL_K1 = 0, /* -d */
  LS_KL_K2 = 1, /* d^2 / 2 */
  LS_KL_K3 = 2  /* exp(d) - d - 1 */
} ls_kl;

/* What a policy loss takes beside the logits and the tokens. */
typedef struct {
  const float* advantages;    /* device [n] */
  const float* old_log_probs; /* device [n]: lp under the policy that sampled; NULL: lp itself, held fixed (ratio 1) */
  const float* ref_log_probs; /* device [n]: lp under the reference; NULL: no KL term (kl_coef 0) */
  const float* weights;       /* device [n] or NULL (1) */
  float clip_low, clip_high;  /* the ratio counts within [1 - clip_low, 1 + clip_high]; clip_low in [0, 1], clip_high
                                 >= 0 (+inf: no bound) */
  float dual_clip;            /* >= 1: a loss from a negative advantage counts a ratio up to this; 0: no such bound */
  float kl_coef;              /* finite */
  ls_kl kl;
  float entropy_coef;         /* finite */
  int32_t entropy;            /* nonzero: metrics hold H even where entropy_coef is 0 */
} ls_policy;

/*
 * ls_policy_loss -- with r = exp(lp - old) and A = advantages[i]:
 *   u = r A        v = clamp(r, 1 - clip_low, 1 + clip_high) A
 *   s = min(u, v), and where A < 0 and dual_clip is set: max(s, dual_clip A)
 *   loss[i] = weights[i] * (-s + kl_coef * KL - entropy_coef * H)
 * The gradient goes through u where u <= v and the bound of dual_clip does not
 * hold, through KL and through H.  A = 0 gives s = 0 whatever r is.  A log-ratio
 * of two log-probs of -inf (a token that both sides exclude) is 0.  Ratio and KL
 * are those of lp as it is returned in fp32: where old and ref are what this call gave
 * for the same rows before, they are 1 and 0 (another call may add a row up in another
 * order: within a rounding).  Where the loss is infinite (a token that one
 * side alone excludes) its gradient is not finite.
 *
 *   out_loss     device float[n]
 *   out_metrics  device float[LS_POLICY_METRICS * n], 16-byte aligned, or NULL
 *   out_stats    as for ls_token_log_probs
 */
ls_status ls_policy_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                         const int32_t* ids, const ls_policy* policy, float temperature, float* out_loss,
                         float* out_metrics, float* out_stats, int32_t* error_word, void* stream);

/* The gradient of sum_i grad_loss[i] * loss[i] (grad_loss NULL: 1); stats are
 * those of ls_policy_loss for the same inputs, out_grad as above. */
ls_status ls_policy_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                  const int32_t* ids, float temperature, const float* stats, const float* grad_loss,
                                  void* out_grad, int64_t grad_stride, void* stream);

/* The loss and its gradient for grad_loss = 1 from one call, for a training
 * loop that knows its row weights (such as 1 / tokens) beforehand. */
ls_status ls_policy_loss_grad(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                              const int32_t* ids, const ls_policy* policy, float temperature, float* out_loss,
                              float* out_metrics, void* out_grad, int64_t grad_stride, int32_t* error_word,
                              void* stream);

typedef enum {
  LS_PREFERENCE_SIGMOID = 0, /* (1 - e) ln(1 + exp(-h)) + e ln(1 + exp(h)), e = label_smoothing */
  LS_PREFERENCE_HINGE = 1,   /* max(0, 1 - h) */
  LS_PREFERENCE_IPO = 2      /* (u - 1 / (2 beta))^2 */
} ls_preference_kind;

/* Pairs of answers: pair p's chosen answer are the rows [answer_offsets[2p],
 * answer_offsets[2p + 1]), its rejected one those up to answer_offsets[2p + 2]. */
typedef struct {
  const int32_t* answer_offsets; /* device [2 * pairs + 1], not descending, within [0, n] */
  int32_t pairs;                 /* < 2^30 */
  const float* ref_log_probs;    /* device [n]: lp under the reference; NULL: 0 (a loss without reference) */
  const float* weights;          /* device [n] or NULL (1) */
  ls_preference_kind kind;
  float beta;            /* finite, > 0 */
  float label_smoothing; /* [0, 0.5], SIGMOID only (else 0) */
  float margin;          /* finite, SIGMOID and HINGE only (else 0) */
  int32_t average;       /* nonzero: an answer's sum is divided by the sum of its weights */
} ls_preference;

/*
 * ls_preference_loss -- with s(answer) = sum of weights[i] * (lp_i - ref_i)
 * over its rows (divided by the sum of weights[i]; 0 where that is 0),
 * u = s(chosen) - s(rejected) and h = beta u - margin: the loss of each pair.
 * A difference of two log-probs of -inf is 0.  A pair whose offsets descend,
 * or leave [0, n] or what the list's first and last offset span, gives
 * NaN, gradient 0 and LS_ROW_ERR_BAD_OFFSETS.  Where such a pair leaves a row in
 * the answers of two others, its gradient is the first one's alone.
 *
 *   out_loss        device float[pairs]
 *   out_log_ratios  device float[2 * pairs]: s of each answer, or NULL
 *   out_stats       as for ls_token_log_probs
 */
ls_status ls_preference_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                             const int32_t* ids, const ls_preference* preference, float temperature, float* out_loss,
                             float* out_log_ratios, float* out_stats, int32_t* error_word, void* stream);

/* The gradient of sum_p grad_loss[p] * loss[p] (grad_loss device float[pairs],
 * or NULL: 1); stats are those of ls_preference_loss for the same inputs.  A row
 * of a pair at or past `pairs` gets NaN. */
ls_status ls_preference_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                      const int32_t* ids, float temperature, const float* stats, int32_t pairs,
                                      const float* grad_loss, void* out_grad, int64_t grad_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LS_TOKEN_OPS_H */
