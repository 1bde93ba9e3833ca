/*
 * ls_row_ops.h -- C ABI of the operators on logits rows that stand around the
 * sampler (part of libls_sampler.so; statuses, dtypes and row errors are those
 * of ls_sampler.h):
 *
 *   ls_process_logits         before sampling: repetition, presence and
 *                             frequency penalties, per-request biases, packed
 *                             masks of allowed tokens (grammars)
 *   ls_top_log_probs          beside sampling: the k best ids of a row, their
 *                             log-probs and the row's log-sum-exp; also the
 *                             targets of a distillation
 *   ls_distill_loss,
 *   ls_distill_loss_backward,
 *   ls_distill_loss_grad      training a student on a teacher's top log-probs:
 *                             the loss, its gradient, or both in one call
 *
 * Every call is asynchronous on the caller's stream, allocates nothing, never
 * synchronises with the host and launches one kernel (ls_process_logits on large
 * batches: two).  Buffers are device memory owned by the caller; parameter
 * structs are small host structs of device pointers.  Results do not depend on the order in which CTAs run: the
 * same inputs give the same bits.
 */
#ifndef LS_ROW_OPS_H
#define LS_ROW_OPS_H

#include "ls_sampler.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more row error: mask_index[i] outside [-1, mask_rows). */
enum { LS_ROW_ERR_BAD_MASK = 8 };

/* Per-request parameters of ls_process_logits: device arrays indexed by
 * request, owned by the caller.  Any group may be absent (NULL). */
typedef struct {
  const int32_t* tokens;       /* [num_requests, token_stride]: each request's ids, prompt first; NULL: no penalties */
  int64_t token_stride;        /* >= token_capacity */
  int32_t token_capacity;      /* ids that a row of `tokens` may hold (< 2^30); lengths are clamped to it */
  const int32_t* prompt_lens;  /* ids of the prompt (NULL: 0) */
  const int32_t* seq_lens;     /* ids in all, prompt included (may be NULL when row_lens is given) */
  const float* repetition;     /* rho > 0; NULL: 1 */
  const float* presence;       /* NULL: 0 */
  const float* frequency;      /* NULL: 0 */
  const int32_t* bias_offsets; /* [num_requests + 1]: request r owns entries [offsets[r], offsets[r+1]), clamped to
                                  [0, bias_count); NULL: none */
  const int32_t* bias_ids;     /* [bias_count], distinct within a request */
  const float* bias_values;    /* [bias_count] */
  int32_t bias_count;          /* < 2^30 */
  int32_t num_requests;
} ls_logits_params;

/*
 * ls_process_logits -- out[i] = row i after penalties, bias and mask.
 *
 * Row i reads x = logits[gather_indices[i]] (or row i) and takes the
 * parameters of request r = token_to_request_index[i] (or i).  Its history is
 * the first L ids of tokens[r], L = row_lens[i] when given, else seq_lens[r];
 * the first prompt_lens[r] of them are the prompt.  With seen(j): j occurs in
 * the history; c(j): occurrences of j past the prompt:
 *     y = seen(j) ? (x > 0 ? x / rho : x * rho) : x
 *     y = y - frequency * c(j) - (c(j) > 0 ? presence : 0)
 *     y = y + bias(j)
 *     y = -inf where the mask's bit j is 0
 * computed in fp32 and rounded once to the logits' type; an entry that nothing
 * touches is copied bit for bit.  Ids outside [0, vocab) (padding, rejected
 * drafts) count nothing.  A touched entry that is NaN, or that would become
 * NaN (inf - inf), gives -inf, the value as which the sampler reads NaN.
 *
 *   params        NULL: no penalties and no bias
 *   row_lens      device int32[n] or NULL.  The verify rows of a speculative
 *                 step give row q of a request the first q drafts this way
 *   allowed_mask  device, mask_rows x mask_stride words of 32 bits, or NULL:
 *                 bit j % 32 of word j / 32 is 1 where id j is allowed
 *   mask_index    device int32[n] or NULL: the mask row of row i, -1 for none
 *                 (NULL: mask row i; mask_rows >= n)
 *   out           n x out_stride elements of the logits' dtype.  out == logits
 *                 works in place (no gather_indices, out_stride ==
 *                 row_stride); any other overlap is refused
 * A mask that allows nothing leaves a row of -inf, to which the sampler
 * answers -1.  Bad rows (gather, request or mask index out of range) are
 * filled with NaN and set their bit in *error_word.
 */
ls_status ls_process_logits(const void* logits, ls_dtype dtype, int64_t logits_rows, int64_t vocab,
                            int64_t row_stride, int32_t n, const int32_t* gather_indices,
                            const int32_t* token_to_request_index, const ls_logits_params* params,
                            const int32_t* row_lens, const int32_t* allowed_mask, int64_t mask_rows,
                            int64_t mask_stride, const int32_t* mask_index, void* out, int64_t out_stride,
                            int32_t* error_word, void* stream);

/*
 * ls_set_process_policy -- which kernels ls_process_logits launches, for every
 * later call in the process (tests and tuning; all write the same values):
 *   0   chosen from the batch (default)
 *   1   one kernel, which settles each tile's touched entries itself
 *   2   a copying kernel and, with params, a second one that settles each row's
 *       touched entries and overlaps the first
 * Returns LS_OK, or LS_ERR_INVALID_ARG for any other value (unchanged).
 */
int ls_set_process_policy(int policy);

/* Largest k of ls_top_log_probs and of the distillation calls. */
#define LS_MAX_TOP 256

/*
 * ls_top_log_probs -- the k best entries of each row.
 *
 * With z = logits / temperature: ids of the k largest entries, the largest
 * first and ties to the lower id; log_probs = z - lse; lse = ln sum exp(z).
 * Special values as for the sampler: NaN is read as -inf; -inf entries are
 * never listed (where fewer than k remain: id -1, log-prob -inf); a row with
 * +inf entries has lse +inf and shares its mass equally among them.  A row
 * without an entry above -inf, or with a bad gather index, gives id -1,
 * log-probs and lse NaN and its bit in *error_word.
 *
 *   k              1 <= k <= min(vocab, LS_MAX_TOP)
 *   temperature    finite, > 0
 *   out_ids        device int32[n * k]
 *   out_log_probs  device float[n * k]
 *   out_lse        device float[n] or NULL
 * LS_ERR_UNSUPPORTED: vocab above ls_row_ops_max_vocab(dtype).
 */
ls_status ls_top_log_probs(const void* logits, ls_dtype dtype, int64_t logits_rows, int64_t vocab,
                           int64_t row_stride, int32_t n, const int32_t* gather_indices, int32_t k,
                           float temperature, int32_t* out_ids, float* out_log_probs, float* out_lse,
                           int32_t* error_word, void* stream);

/* What the loss makes of the teacher's mass outside its k entries. */
typedef enum {
  LS_TAIL_DROP = 0,   /* nothing: the sum stops at the k entries */
  LS_TAIL_RENORM = 1, /* the k probabilities are scaled to sum to 1 */
  LS_TAIL_BUCKET = 2  /* one further outcome, "none of them", with what is left of either side's mass */
} ls_tail;

/* Teacher's targets: row-major [n, stride], each row k ids (distinct) and
 * their natural log-probs at the loss's temperature.  An id outside [0, vocab)
 * and a log-prob of -inf or NaN count nothing (padding). */
typedef struct {
  const int32_t* ids;
  const float* log_probs;
  int64_t stride; /* >= k */
  int32_t k;      /* 1 <= k <= LS_MAX_TOP */
} ls_teacher;

/* Floats per row that ls_distill_loss leaves for ls_distill_loss_backward. */
#define LS_DISTILL_STATS 8

/*
 * ls_distill_loss -- loss[i] = weights[i] * KL(teacher || student) of row i.
 *
 * With z = logits / temperature, q = softmax(z), p_k = exp(log_probs[k]) and
 * P = sum p_k:
 *   DROP     sum_k p_k (ln p_k - ln q_k)
 *   RENORM   the same with p_k / P (P below 2^-100: no targets)
 *   BUCKET   DROP plus p_r (ln p_r - ln q_r), p_r = max(0, 1 - P), q_r the
 *            student's mass outside the k ids (the term is left out where
 *            p_r = 0 or no entry above -inf lies outside them)
 * All in fp32.  NaN logits are read as -inf.  A row of weight 0 is not read:
 * loss 0, gradient 0 whatever grad_loss holds.  A row without an entry above
 * -inf: loss and gradient NaN, LS_ROW_ERR_NO_FINITE.
 *
 *   weights    device float[n] or NULL (1)
 *   out_loss   device float[n]
 *   out_stats  device float[LS_DISTILL_STATS * n], 16-byte aligned, or NULL:
 *              what the backward pass needs of each row
 * LS_ERR_UNSUPPORTED: vocab above ls_row_ops_max_vocab(dtype).
 */
ls_status ls_distill_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                          const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                          float* out_loss, float* out_stats, int32_t* error_word, void* stream);

/*
 * ls_distill_loss_backward -- the gradient of sum_i grad_loss[i] * loss[i].
 *
 *   d/dx_j = g / T * (A q_j - [j one of the ids] p_j - [j none of them] p_r q_j / q_r)
 *   g = weights[i] * grad_loss[i];  A = P (DROP), 1 (RENORM), P + p_r (BUCKET)
 * (the p_r terms in BUCKET only, where the loss has its tail term).
 *
 *   stats      what ls_distill_loss wrote for the same inputs
 *   grad_loss  device float[n] or NULL (1)
 *   out_grad   n x grad_stride elements of the logits' dtype; may be the logits
 *              themselves (grad_stride == row_stride); any other overlap is
 *              refused
 */
ls_status ls_distill_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                   const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                                   const float* stats, const float* grad_loss, void* out_grad, int64_t grad_stride,
                                   void* stream);

/*
 * ls_distill_loss_grad -- the loss and its gradient for grad_loss = 1 from one
 * read of the logits: for a training loop that knows its row weights (such as
 * 1 / tokens) beforehand.  out_grad as for ls_distill_loss_backward.
 */
ls_status ls_distill_loss_grad(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                               const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                               float* out_loss, void* out_grad, int64_t grad_stride, int32_t* error_word,
                               void* stream);

/* Largest vocab that ls_top_log_probs and the distillation calls accept for a
 * dtype on the current device, or 0 when no CUDA device is available.
 * ls_process_logits has no such limit below 2^31 - 1. */
int64_t ls_row_ops_max_vocab(ls_dtype dtype);

#ifdef __cplusplus
}
#endif

#endif /* LS_ROW_OPS_H */
