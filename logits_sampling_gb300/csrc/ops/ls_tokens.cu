// ls_tokens.cu -- the operators of include/ls_token_ops.h: log-probs of given
// tokens, the policy loss and the preference loss, with their gradients.
//
// token_kernel: a row over a CTA, or over a cluster where there are few, streamed
// once for its sum and entropy term; the operator's scalars follow in the same
// launch.  pair_kernel: a CTA per pair of answers sums their rows' terms and leaves
// each row's slope.  token_backward_kernel: one sweep over the logits with the two
// slopes that a forward call left of each row, for all three operators.  Loss and
// gradient from one call are in ls_token_grad.cu.
#include "ls_token_ops.cuh"

namespace lsg {
namespace ops {

// Bound by DRAM where there are rows enough (a kernel that only reads reaches 7.7 TB/s):
// 2048 x 128256 bf16 78 us (6.7 TB/s), with entropies 84 (each stage's maximum is looked
// for), 1024 x 262144 fp32 with entropies 150 (7.2). Fewer rows by what is in flight: 672 x
// 151936 32.6 us (6.3 TB/s), 64 x 128256 7.1, one row of 32000 3.6 (launch, two reads
// one after the other, barrier, scalars).
template <typename TIn, bool kEntropy, int T>
__global__ void __launch_bounds__(T, 1024 / T) token_kernel(const TokenArgs a, int upc) {
  __shared__ Moments red[T / 32];
  __shared__ Part parts[kMaxCluster];
  const int tid = threadIdx.x;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  wait_for_previous();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, rank);
  Stages<TIn, T> st;
  st.init(run);
  typename Run<TIn, T>::Stage first;
  if (st.whole > 0) st.template load<LOAD_ONCE>(0, first);
  RowInputs in;
  if (!counts(a, i, in.id, in.w)) {
    if (tid == 0 && rank == 0) skip_row(a, i);
    return;  // every CTA of the row leaves here, before any cluster barrier
  }
  if (C > 1) cluster_arrive();  // the peers' shared memory may be written once all have arrived
  load_inputs<TIn>(a, i, in);
  const float c = a.c;
  Moments r;
  bool careful = false;
#pragma unroll 1
  for (;;) {
    RowSum<kEntropy> acc;
    sum_run<LOAD_ONCE, false>(run, st, first, acc, c, careful, Kept<T>{nullptr, 0});
    r = block_moments<T / 32, kEntropy>(acc.moments(), c, red);
    if (careful || sum_ok(r)) break;  // the same in every thread
    careful = true;
    __syncthreads();  // red is read
  }
  let_next_start();
  if (C > 1) cluster_moments<kEntropy>(r, careful, c, parts, C, rank);
  if (tid == 0 && rank == 0) finish_row<kEntropy>(a, i, r, in, careful);
}

// The sums of a pair's two answers, its loss, and the slope of each of its rows.
// Terms cancel, so they are added with what each addition loses.  One CTA, one
// chain of reads and sums: with its row kernel one pair of 22 rows takes 5.9 us; in
// fp64 9.6.
constexpr int kPairThreads = 256;

struct Exact {
  float hi, lo;
  __device__ __forceinline__ void add(float v, float low = 0.f) {
    float lost = 0.f;
    hi = two_sum(hi, v, lost);
    lo += (lost == lost ? lost : 0.f) + low;  // an infinite sum loses nothing
  }
  __device__ __forceinline__ float value() const { return hi + lo; }
};

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
  __shared__ Exact red[4][kW];
  const int tid = threadIdx.x, lane = tid & 31;
  const int32_t p = (int32_t)blockIdx.x;
  const int32_t* at = a.p.answer_offsets + 2 * (int64_t)p;
  // after a row kernel, which has waited for whatever wrote them, the offsets are there
  if (a.n == 0) wait_for_previous();
  const int32_t lo = at[0], mid = at[1], hi = at[2];
  // the row kernel has looked at rows from the list's first to its last offset only
  const int32_t least = max(a.p.answer_offsets[0], 0), most = min(a.p.answer_offsets[2 * (int64_t)a.p.pairs], a.n);
  wait_for_previous();
  let_next_start();
  if (lo < least || mid < lo || hi < mid || hi > most) {
    if (tid == 0) {
      a.out_loss[p] = quiet_nan();
      if (a.out_log_ratios) a.out_log_ratios[2 * (int64_t)p] = a.out_log_ratios[2 * (int64_t)p + 1] = quiet_nan();
      if (a.error_word) atomicOr(a.error_word, LS_ROW_ERR_BAD_OFFSETS);
    }
    return;
  }
  Exact v[4] = {};  // sum and weight of the chosen, of the rejected answer
  float mine = 0.f;  // the weight of this thread's first row
  const int64_t first = (int64_t)lo + tid;  // past 2^31 in the last rows of the largest batch
  for (int64_t i = first; i < hi; i += kPairThreads) {
    const float term = a.stats[i].term, w = a.stats[i].w, term_lo = a.stats[i].term_lo;
    if (i == first) mine = w;
    const int k = i < mid ? 0 : 2;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      v[q].add(k == q ? term : 0.f, k == q ? term_lo : 0.f);
      v[q + 1].add(k == q ? w : 0.f);
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      v[q].add(__shfl_xor_sync(0xFFFFFFFFu, v[q].hi, o), __shfl_xor_sync(0xFFFFFFFFu, v[q].lo, o));
    if (lane == 0) red[q][tid >> 5] = v[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[q] = red[q][0];
#pragma unroll
    for (int k = 1; k < kW; ++k) v[q].add(red[q][k].hi, red[q][k].lo);
  }
  float over[2] = {1.f, 1.f};
  if (a.p.average) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float w = v[2 * k + 1].value();
      over[k] = w != 0.f ? 1.f / w : 0.f;
      v[2 * k] = Exact{w != 0.f ? v[2 * k].value() / w : 0.f, 0.f};
    }
  }
  const float s[2] = {v[0].value(), v[2].value()};
  v[0].add(-v[2].hi, -v[2].lo);
  const float u = v[0].value(), beta = a.p.beta;
  const float h = fmaf(beta, u, -a.p.margin);
  float loss, slope;  // of u
  if (a.p.kind == LS_PREFERENCE_SIGMOID) {
    const float e = a.p.label_smoothing, small = expf(-fabsf(h)), tail = log1pf(small);
    const float far = 1.f / (1.f + small), near = small * far;  // sigma(|h|), sigma(-|h|)
    loss = (1.f - e) * (fmaxf(-h, 0.f) + tail);
    if (e > 0.f) loss += e * (fmaxf(h, 0.f) + tail);
    slope = beta * (e * (h > 0.f ? far : near) - (1.f - e) * (h > 0.f ? near : far));
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
      a.out_log_ratios[2 * (int64_t)p] = s[0];
      a.out_log_ratios[2 * (int64_t)p + 1] = s[1];
    }
  }
  for (int64_t i = first; i < hi; i += kPairThreads) {
    const float w = i == first ? mine : a.stats[i].w;
    const float g = w == 0.f ? 0.f : i < mid ? slope * w * over[0] : -slope * w * over[1];
    // of two pairs (a list that descends elsewhere may give a row to both) the first: the slope and the pair in one word
    atomicMin(reinterpret_cast<unsigned long long*>(&a.stats[i].g_lp),
              (unsigned long long)(uint32_t)p << 32 | __float_as_uint(g));
  }
}

// The backward passes, in runs of a row.  In place (the gradient may replace the
// logits) each unit is read before the same thread writes it.
struct TokenBackArgs {
  const void* logits;
  int64_t vocab, row_stride;
  const int32_t* ids;
  float c;  // log2(e) / T
  const TokenStats* stats;
  const float* up_lp;  // the gradient from above, by stats.up
  const float* up_H;
  int32_t ups;         // its entries
  float none_lp, none_H;  // where there is none
  void* out_grad;
  int64_t grad_stride;
};

// CTAs of 128 threads with runs of four stages (32 KB), fewer where that would
// leave SMs without a second wave.  2048 x 128256 bf16, one row in four of them
// without a gradient, with runs of 1 / 2 / 4 stages 162 / 144 / 141 us; without such
// rows 164 / 153 / 154 (the measured copy rate); one row 1.8 / 2.1 / 2.7; 256 threads
// the same.  Each run pays for a row's scalars again, 44 bytes and twenty operations;
// working them out from the row's sum here instead of in the forward pass took 333 x
// 32000 from 7.2 to 8.7 us.
constexpr int kBackThreads = 128;
constexpr int kBackRun = 4;  // stages at most

template <typename TIn>
__global__ void __launch_bounds__(kBackThreads, 1024 / kBackThreads)
    token_backward_kernel(const TokenBackArgs a, int runs, int upc) {
  constexpr int T = kBackThreads;
  using Raw = typename Elem<TIn>::Raw;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)runs;
  wait_for_previous();
  let_next_start();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, (int)(blockIdx.x % (unsigned)runs));
  Raw* grad = static_cast<Raw*>(a.out_grad) + i * a.grad_stride;
  Stages<TIn, T> stages;
  stages.init(run);
  typename Run<TIn, T>::Stage first;
  // before the row's scalars are known, but where rows may wait: one without a gradient is not read there
  const bool early = upc < kBackRun * T * kStage;
  if (early && stages.whole > 0) stages.template load<LOAD_PLAIN>(0, first);
  const float4* in = reinterpret_cast<const float4*>(a.stats + i);
  const float4 s0 = in[0], s1 = in[1];
  TokenStats st;
  st.M = s0.x;
  st.over = s0.y;
  st.id_lp = s0.z;
  st.id_H = s0.w;
  st.mean = s1.w;
  st.dirty = in[2].x;
  const int32_t id = a.ids[i], up = __float_as_int(s1.y);
  const bool has = up >= 0 && up < a.ups;  // stats of another call do not lead out of bounds
  // a slope of 0 counts nothing, whatever the gradient from above
  const float g_lp = s1.x == 0.f ? 0.f : s1.x * (!a.up_lp ? a.none_lp : has ? a.up_lp[up] : quiet_nan());
  const float g_H = s1.z == 0.f ? 0.f : s1.z * (!a.up_H ? a.none_H : has ? a.up_H[up] : quiet_nan());
  // an id that has left the vocabulary since the forward call: its place would be next to the row
  const bool in_vocab = id >= 0 && (int64_t)id < a.vocab;
  if (!in_vocab || (g_lp == 0.f && g_H == 0.f)) {
    const bool same = run.aligned_with(grad);
    uint32_t z[8] = {};
    for (int u = tid; u < run.n; u += T) run.store(grad, same, u, z);
    return;
  }
  if (!early && stages.whole > 0) stages.template load<LOAD_PLAIN>(0, first);
  RowGradient g;
  g.init(st, g_lp, g_H, a.c);
  gradient_run<false>(run, stages, first, g, grad, Kept<T>{nullptr, 0});
  const int place = run.place(id);  // the thread that has written it writes it again
  if (place >= 0 && tid == stages.owner(run, place)) grad[id] = Elem<TIn>::put(g.at_id);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// How a batch is laid out on the SMs, which hold 1024 threads of these kernels
// each.  Measured, us (threads of a CTA x CTAs of a row):
//   few rows of 128 KB and more: a row over as many CTAs as find room at once.  8
//     rows of 256 KB 256x8 4.1, 256x4 4.7, 256x1 6.6; 64 of them 6.8, 6.9, 10.4; of 64
//     KB 5.1, 4.2, 4.2
//   else one CTA per row, the largest for which every row has its own at once.
//     Rows of 256 KB with 512 / 256 / 192 / 128 threads: 304 of them 14.3, 15.6, 16.9,
//     20.1; 608 25.9, 24.7, 25.3, 26.9; 760 34.6, 36.2, 30.2, 31.5; 1216 48.8, 46.6,
//     49.0, 46.2
//   more rows than that: 128 or 192 threads, whichever leaves the last wave
//     fuller.  1400 63.3 with 128, 53.4 with 192; 2048 76.4, 77.5 (waves of .68, .70)
struct ForwardPlan {
  int threads, ctas;
};
static ForwardPlan forward_plan(int32_t n, int64_t bytes) {
  const int sms = device_attr<cudaDevAttrMultiProcessorCount>();
  if (bytes <= 16 * 1024 || sms <= 0) return {128, 1};
  if (n <= 128 && bytes >= 128 * 1024) {
    int c = 1;
    while (c < kMaxCluster && n * c * 2 <= 512) c *= 2;
    return {256, c};
  }
  if (n <= 5 * sms) return {n <= 2 * sms ? 512 : n <= 4 * sms ? 256 : 192, 1};
  // the rows of the last wave, in sixty-fourths of one
  const auto last = [&](int per_sm) { return (int)((int64_t)((n - 1) % (per_sm * sms) + 1) * 64 / (per_sm * sms)); };
  return {n > 8 * sms && last(5) > last(8) + 4 ? 192 : 128, 1};
}

template <typename TIn, bool kEntropy>
static ls_status pick_forward(const TokenArgs& a, ls_dtype dtype, cudaStream_t st) {
  const int64_t units = row_units(a.vocab, dtype);
  const ForwardPlan p = forward_plan(a.n, units * 32);
  const int upc = (int)((units + p.ctas - 1) / p.ctas);
  if ((int64_t)a.n * p.ctas > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)a.n * p.ctas);
  return p.threads == 128   ? launch_kernel(token_kernel<TIn, kEntropy, 128>, grid, 128, p.ctas, 0, st, a, upc)
         : p.threads == 192 ? launch_kernel(token_kernel<TIn, kEntropy, 192>, grid, 192, p.ctas, 0, st, a, upc)
         : p.threads == 256 ? launch_kernel(token_kernel<TIn, kEntropy, 256>, grid, 256, p.ctas, 0, st, a, upc)
                            : launch_kernel(token_kernel<TIn, kEntropy, 512>, grid, 512, p.ctas, 0, st, a, upc);
}

static ls_status forward(const TokenArgs& a, ls_dtype dtype, bool entropy, cudaStream_t st) {
  if (dtype == LS_DTYPE_BF16)
    return entropy ? pick_forward<bf16_tag, true>(a, dtype, st) : pick_forward<bf16_tag, false>(a, dtype, st);
  return entropy ? pick_forward<float, true>(a, dtype, st) : pick_forward<float, false>(a, dtype, st);
}

static ls_status backward(const TokenBackArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  constexpr int kStep = kBackThreads * kStage;  // units of a stage
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t units = row_units(a.vocab, dtype);
  const int sms = device_attr<cudaDevAttrMultiProcessorCount>();
  int upc = kBackRun * kStep;
  while (upc > kStep && (units + upc - 1) / upc * n < 16 * sms) upc /= 2;
  const int64_t runs = (units + upc - 1) / upc;
  if (runs * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(runs * n));
  return dtype == LS_DTYPE_BF16
             ? launch_kernel(token_backward_kernel<bf16_tag>, grid, kBackThreads, 1, 0, st, a, (int)runs, upc)
             : launch_kernel(token_backward_kernel<float>, grid, kBackThreads, 1, 0, st, a, (int)runs, upc);
}

static bool finite(float v) { return v - v == 0.f; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The checks that the calls share.
static bool rows_ok(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, const int32_t* ids,
                    float temperature) {
  return matrix_ok(logits, dtype, vocab, row_stride) && ids && temperature > 0.f && finite(temperature) &&
         finite(kLog2e / temperature);
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
  a.c = kLog2e / temperature;
  a.inv_T = 1.f / temperature;
  a.kind = kind;
  return a;
}

// The three backward calls: what stands for a missing gradient differs.
static ls_status backward_call(const void* logits, ls_dtype dtype, int64_t vocab, int64_t row_stride, int32_t n,
                               const int32_t* ids, float temperature, const float* stats, const float* up_lp,
                               const float* up_H, int32_t ups, float none, void* out_grad, int64_t grad_stride,
                               void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!rows_ok(logits, dtype, vocab, row_stride, ids, temperature) || !stats || !aligned16(stats) ||
      !grad_ok(logits, dtype, vocab, row_stride, n, out_grad, grad_stride))
    return LS_ERR_INVALID_ARG;
  const TokenBackArgs a{logits, vocab, row_stride, ids,  kLog2e / temperature, reinterpret_cast<const TokenStats*>(stats),
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
  return token_grad(a, dtype, policy->entropy || policy->entropy_coef != 0.f, static_cast<cudaStream_t>(stream));
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
