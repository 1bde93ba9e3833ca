// ls_distill.cu -- the distillation loss from a teacher's top log-probs and
// its gradient (ls_distill_loss, ls_distill_loss_backward,
// ls_distill_loss_grad).
//
// One CTA per row.  A bitmap in shared memory marks the teacher's ids; maximum
// and sum of exponentials are taken over the entries outside them, so that the
// mass outside (q_r) is a sum of its own and not a difference of two sums; the
// at most 256 entries inside join afterwards.
#include "ls_row_ops.cuh"

namespace lsg {
namespace ops {

struct DistillArgs {
  const void* logits;
  int64_t vocab, row_stride;
  ls_teacher t;
  float temperature;
  int tail;
  const float* weights;
  const float* grad_loss;
  const float4* stats_in;
  float* out_loss;
  float4* out_stats;
  void* out_grad;
  int64_t grad_stride;
  int32_t* error_word;
};

struct OpMaxF {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// exp((v - M) / T) for v <= M; entries at an infinite maximum share it.
__device__ __forceinline__ float rel_exp(float v, float M, float c) { return v == M ? 1.f : ex2((v - M) * c); }

template <typename TIn, bool kLoss, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  extern __shared__ uint32_t bits[];  // ceil(vocab / 32)
  __shared__ float red_f[kWarps];
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x, V = a.vocab;
  const float w = a.weights ? a.weights[i] : 1.f;
  const Raw* row = static_cast<const Raw*>(a.logits) + i * a.row_stride;
  Raw* grad = kGrad ? static_cast<Raw*>(a.out_grad) + i * a.grad_stride : nullptr;
  if (w == 0.f) {
    if (kGrad)
      for (int64_t j = tid; j < V; j += kThreads) grad[j] = E::put(0.f);
    if (tid == 0 && kLoss) {
      a.out_loss[i] = 0.f;
      if (a.out_stats) a.out_stats[i] = make_float4(0.f, 1.f, 0.f, 1.f);
    }
    return;
  }
  // the teacher's entry of this thread
  int id = -1;
  float t = kNegInf, p = 0.f, x = kNegInf;
  if (tid < a.t.k) {
    id = a.t.ids[i * a.t.stride + tid];
    t = a.t.log_probs[i * a.t.stride + tid];
    if (id < 0 || (int64_t)id >= V || !(t > kNegInf)) id = -1;
    if (id >= 0) {
      x = guard(E::get(row[id]));
      p = expf(t);
    }
  }
  const int words = (int)((V + 31) / 32);
  for (int q = tid; q < words; q += kThreads) bits[q] = 0u;
  __syncthreads();
  if (id >= 0) atomicOr(&bits[id >> 5], 1u << (id & 31));
  const float P = block_reduce(p, OpAddF(), red_f);  // the barriers inside order the bitmap too
  auto listed = [&](int64_t j) { return (bits[j >> 5] >> (j & 31)) & 1u; };

  const float c = kLog2e / a.temperature;
  float M, S, Mr, Sr;
  if (kLoss) {
    float m = kNegInf;
    for (int64_t j = tid; j < V; j += kThreads)
      if (!listed(j)) m = fmaxf(m, guard(E::get(row[j])));
    Mr = block_reduce(m, OpMaxF(), red_f);
    float s = 0.f;
    if (Mr > kNegInf)
      for (int64_t j = tid; j < V; j += kThreads)
        if (!listed(j)) s += rel_exp(guard(E::get(row[j])), Mr, c);
    Sr = block_reduce(s, OpAddF(), red_f);
    M = fmaxf(Mr, block_reduce(x, OpMaxF(), red_f));
    S = block_reduce(id >= 0 && M > kNegInf ? rel_exp(x, M, c) : 0.f, OpAddF(), red_f);
    if (Mr > kNegInf) S += Sr * rel_exp(Mr, M, c);
    if (tid == 0 && a.out_stats) a.out_stats[i] = make_float4(M, S, Mr, Sr);
  } else {
    const float4 st = a.stats_in[i];
    M = st.x;
    S = st.y;
    Mr = st.z;
    Sr = st.w;
  }
  if (M == kNegInf) {
    if (kGrad)
      for (int64_t j = tid; j < V; j += kThreads) grad[j] = E::put(quiet_nan());
    if (tid == 0 && kLoss) {
      a.out_loss[i] = quiet_nan();
      if (a.error_word) atomicOr(a.error_word, LS_ROW_ERR_NO_FINITE);
    }
    return;
  }
  float lnP = 0.f;
  float A = P;
  if (a.tail == LS_TAIL_RENORM) {
    lnP = logf(P);
    p = p / P;
    if (!(P > 0.f)) p = 0.f;
    A = P > 0.f ? 1.f : 0.f;
  }
  float pr = 0.f;
  if (a.tail == LS_TAIL_BUCKET && Mr > kNegInf) {
    pr = fmaxf(1.f - P, 0.f);
    A = P + pr;
  }
  if (kLoss) {
    const float lnS = logf(S);
    float term = 0.f;
    if (p > 0.f) term = p * ((t - lnP) - ((x == M ? 0.f : (x - M) / a.temperature) - lnS));
    if (tid == 0 && pr > 0.f)
      term += pr * (logf(pr) - ((Mr == M ? 0.f : (Mr - M) / a.temperature) + logf(Sr / S)));
    const float kl = block_reduce(term, OpAddF(), red_f);
    if (tid == 0) a.out_loss[i] = w * kl;
  }
  if (kGrad) {
    const float g = w * (a.grad_loss ? a.grad_loss[i] : 1.f) / a.temperature;
    const float gA = g * (A / S), gR = pr > 0.f ? g * (pr / Sr) : 0.f;
    for (int64_t j = tid; j < V; j += kThreads) {
      if (listed(j)) continue;
      const float v = guard(E::get(row[j]));
      float d = gA * rel_exp(v, M, c);
      if (gR != 0.f) d -= gR * rel_exp(v, Mr, c);
      grad[j] = E::put(d);
    }
    if (id >= 0) grad[id] = E::put(gA * rel_exp(x, M, c) - g * p);
  }
}

template <typename TIn, bool kLoss, bool kGrad>
static ls_status launch(const DistillArgs& a, int32_t n, cudaStream_t st) {
  const size_t smem = (size_t)((a.vocab + 31) / 32) * 4;
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(distill_kernel<TIn, kLoss, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return LS_ERR_CUDA;
  distill_kernel<TIn, kLoss, kGrad><<<dim3((unsigned)n), dim3(kThreads), smem, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}

template <bool kLoss, bool kGrad>
static ls_status dispatch(const DistillArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == LS_DTYPE_BF16 ? launch<bf16_tag, kLoss, kGrad>(a, n, st) : launch<float, kLoss, kGrad>(a, n, st);
}

// The checks that the three calls share.
static ls_status check(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, const ls_teacher* t,
                       float temperature, ls_tail tail) {
  if (!matrix_ok(logits, dtype, vocab, row_stride) || !t || !t->ids || !t->log_probs || t->k < 1 ||
      t->k > LS_MAX_TOP || t->stride < t->k)
    return LS_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || temperature > 3.4028235e38f) return LS_ERR_INVALID_ARG;
  if (tail != LS_TAIL_DROP && tail != LS_TAIL_RENORM && tail != LS_TAIL_BUCKET) return LS_ERR_INVALID_ARG;
  return vocab > max_row(dtype) ? LS_ERR_UNSUPPORTED : LS_OK;
}

static bool stats_ok(const float* s) { return (reinterpret_cast<uintptr_t>(s) & 15u) == 0; }

}  // namespace ops
}  // namespace lsg

using namespace lsg;
using namespace lsg::ops;

extern "C" {

ls_status ls_distill_loss(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                          const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                          float* out_loss, float* out_stats, int32_t* error_word, void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  const ls_status rc = check(logits, dtype, vocab, row_stride, teacher, temperature, tail);
  if (rc != LS_OK) return rc;
  if (!out_loss || !stats_ok(out_stats)) return LS_ERR_INVALID_ARG;
  const DistillArgs a{logits,  vocab,   row_stride, *teacher, temperature, (int)tail,
                      weights, nullptr, nullptr,    out_loss, reinterpret_cast<float4*>(out_stats),
                      nullptr, 0,       error_word};
  return dispatch<true, false>(a, dtype, n, stream);
}

ls_status ls_distill_loss_backward(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                                   const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                                   const float* stats, const float* grad_loss, void* out_grad, int64_t grad_stride,
                                   void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  const ls_status rc = check(logits, dtype, vocab, row_stride, teacher, temperature, tail);
  if (rc != LS_OK) return rc;
  if (!stats || !stats_ok(stats) || !matrix_ok(out_grad, dtype, vocab, grad_stride) ||
      !overlap_ok(logits, n, row_stride, out_grad, n, grad_stride, vocab, dtype, true))
    return LS_ERR_INVALID_ARG;
  const DistillArgs a{logits,   vocab,     row_stride,  *teacher, temperature, (int)tail,
                      weights,  grad_loss, reinterpret_cast<const float4*>(stats), nullptr, nullptr,
                      out_grad, grad_stride, nullptr};
  return dispatch<false, true>(a, dtype, n, stream);
}

ls_status ls_distill_loss_grad(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                               const ls_teacher* teacher, float temperature, ls_tail tail, const float* weights,
                               float* out_loss, void* out_grad, int64_t grad_stride, int32_t* error_word,
                               void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  const ls_status rc = check(logits, dtype, vocab, row_stride, teacher, temperature, tail);
  if (rc != LS_OK) return rc;
  if (!out_loss || !matrix_ok(out_grad, dtype, vocab, grad_stride) ||
      !overlap_ok(logits, n, row_stride, out_grad, n, grad_stride, vocab, dtype, true))
    return LS_ERR_INVALID_ARG;
  const DistillArgs a{logits,  vocab,   row_stride, *teacher, temperature, (int)tail,   weights,
                      nullptr, nullptr, out_loss,   nullptr,  out_grad,    grad_stride, error_word};
  return dispatch<true, true>(a, dtype, n, stream);
}

}  // extern "C"
