// ls_distill.cu -- the distillation loss from a teacher's top log-probs and
// its gradient (ls_distill_loss, ls_distill_loss_backward,
// ls_distill_loss_grad).
//
// Loss, and loss with gradient (distill_kernel): a row over the CTAs of a
// cluster (ls_stream.cuh).  A bit per unit in shared memory marks those that hold
// one of the teacher's ids, and a small hash table says which of their entries
// do; the running maximum and sum skip them, so that the mass outside them (q_r) is
// a sum of its own rather than a difference of two.  With the entries outside
// of maximum M_r and e_j = exp((x_j - M_r) / T), the gradient outside the ids
// is one multiple of e_j:
//     d_j = g / T * e_j * kappa,   kappa = A exp((M_r - M) / T) / S - p_r / S_r
// and the at most 256 ids follow one by one: g / T * (alpha exp((x - M) / T) -
// p), alpha = A / S.  M_r, kappa, M, alpha and the scale of p are the row's
// `stats`: the backward pass (distill_backward_kernel) reads them and nothing
// else of the forward pass, and is one sweep over the logits.  In the
// call that gives both, each CTA reads its run a second time for the gradient;
// runs are short enough that what is in flight stays in L2.
#include "ls_stream.cuh"

namespace lsg {
namespace ops {

// What the backward pass needs of a row (LS_DISTILL_STATS floats).
struct alignas(16) RowStats {
  float M, alpha, Mr, kappa, scale, pad[3];
};
static_assert(sizeof(RowStats) == sizeof(float) * LS_DISTILL_STATS, "the header's size of a row's stats");

struct DistillArgs {
  const void* logits;
  int64_t vocab, row_stride;
  ls_teacher t;
  float temperature;
  int tail;
  const float* weights;
  const float* grad_loss;
  const RowStats* stats_in;
  float* out_loss;
  RowStats* out_stats;
  void* out_grad;
  int64_t grad_stride;
  int32_t* error_word;
};

// A teacher's mass below this is none to renormalise (its reciprocal would overflow).
constexpr float kLeastMass = 7.8886e-31f;  // 2^-100

// Gradient of a unit outside the ids: coef * exp((x - m) / T), coef over
// x.scale where x is fast.
template <typename TIn>
__device__ __forceinline__ void unit_grad(uint32_t (&w)[8], const ExpAgainst& x, float coef) {
  constexpr int kN = Unit<TIn>::kN;
  const f32x2 c2 = pack2(coef, coef);
  uint32_t o[8];
  if (x.fast) {
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float a, b;
      unpack2(mul2(x.pair_fast(Unit<TIn>::pair(w, q)), c2), a, b);
      Unit<TIn>::set_pair(o, q, a, b);
    }
  } else {
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float a, b;
      unpack2(mul2(x.pair_slow(Unit<TIn>::pair(w, q)), c2), a, b);
      Unit<TIn>::set_pair(o, q, a, b);
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) w[q] = o[q];
}

constexpr int kHeld = 2 * LS_MAX_TOP;               // slots of the table of units that hold one
static_assert((kHeld & (kHeld - 1)) == 0, "a power of two");

struct DistillShared {
  float2 ms[kMaxCluster];  // each CTA's maximum and sum over the entries outside the ids
  float2 red[8];
  float x[LS_MAX_TOP];     // the student's logits at the ids (-inf where there is none)
  float p[LS_MAX_TOP];
  float lp[LS_MAX_TOP];
  int unit[kHeld];         // a unit of the run, -1: free
  uint32_t entries[kHeld]; // a bit for each of its entries that is one of the ids
  RowStats st;
};

__device__ __forceinline__ int held_home(int u) { return (int)(((uint32_t)u * 0x9E3779B1u) >> 16) & (kHeld - 1); }
// Notes that entry e of unit u is one of the ids (never more than half full).
__device__ __forceinline__ void hold(DistillShared& sh, int u, int e) {
  int at = held_home(u);
  for (int t = 0; t < kHeld; ++t) {
    const int was = atomicCAS(&sh.unit[at], -1, u);
    if (was == -1 || was == u) {
      atomicOr(&sh.entries[at], 1u << e);
      return;
    }
    at = (at + 1) & (kHeld - 1);
  }
}
__device__ __forceinline__ uint32_t held_entries(const DistillShared& sh, int u) {
  int at = held_home(u);
  for (int t = 0; t < kHeld; ++t) {
    const int has = sh.unit[at];
    if (has == u) return sh.entries[at];
    if (has == -1) return 0u;
    at = (at + 1) & (kHeld - 1);
  }
  return 0u;
}

// Bound by DRAM, and by rows that start and end together: the loss of 2048 x
// 128256 bf16 takes 87 us (6.0 TB/s, 0.90 of the measured copy rate), of 600 such
// rows, one wave, 27 us (5.6 TB/s), of 1024 x 262144 fp32 163 us (6.6 TB/s, 0.98).
// With the gradient the last takes 406 us (5.3 TB/s, 0.79: a quarter of the second
// read misses L2, and each row waits once for its whole cluster; fewer CTAs per
// SM, 441 us with three and 549 with two, lose more than they hit), 2048 x 128256
// bf16 204 us (5.1 TB/s).
template <typename TIn, bool kGrad, int T>
__global__ void __launch_bounds__(T, 1024 / T) distill_kernel(const DistillArgs a, int upc) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  constexpr int kN = Unit<TIn>::kN;
  constexpr int kFirst = kGrad ? LOAD_KEEP : LOAD_ONCE;
  constexpr int kOwn = LS_MAX_TOP / T;  // teacher entries per thread
  static_assert(kOwn * T == LS_MAX_TOP, "");
  extern __shared__ uint4 dyn_smem[];
  __shared__ DistillShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  wait_for_previous();
  Run<TIn, T> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, rank);
  Raw* grad = kGrad ? static_cast<Raw*>(a.out_grad) + i * a.grad_stride : nullptr;
  // the teacher's entries of this thread, beside the weight that decides whether they matter
  const float w = a.weights ? a.weights[i] : 1.f;
  int id[kOwn];
  float t[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int k = tid + q * T;
    id[q] = k < a.t.k ? a.t.ids[i * a.t.stride + k] : -1;
    t[q] = k < a.t.k ? a.t.log_probs[i * a.t.stride + k] : kNegInf;
  }
  if (w == 0.f) {  // every CTA of the row leaves here, before any cluster barrier
    if (kGrad) {
      const bool same = run.aligned_with(grad);
      uint32_t z[8] = {};
      for (int u = tid; u < run.n; u += T) run.store(grad, same, u, z);
    }
    if (tid == 0 && rank == 0) {
      a.out_loss[i] = 0.f;
      if (a.out_stats) a.out_stats[i] = RowStats{0.f, 0.f, 0.f, 0.f, 1.f, {}};
    }
    return;
  }
  typename Run<TIn, T>::Stage first;
  run.template prefetch<kFirst>(tid, first);
  if (C > 1) cluster_arrive();  // the peers' shared memory may be written once all have arrived
  // a bit per unit of the run
  uint32_t* bits = reinterpret_cast<uint32_t*>(dyn_smem);
  for (int q = tid; q < (run.n + 127) / 128; q += T) dyn_smem[q] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int q = 0; q < kHeld / T; ++q) {
    sh.unit[tid + q * T] = -1;
    sh.entries[tid + q * T] = 0u;
  }
  __syncthreads();
  // the student's logits at the ids, on their way while the run streams
  typename E::Raw x[kOwn];
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    if (id[q] < 0 || (int64_t)id[q] >= a.vocab || !(t[q] > kNegInf)) id[q] = -1;
    x[q] = id[q] >= 0 ? run.row[id[q]] : E::neg_inf();
    const int place = id[q] >= 0 ? run.place(id[q]) : -1;
    if (place >= 0) {
      atomicOr(&bits[place / kN >> 5], 1u << (place / kN & 31));
      hold(sh, place / kN, place % kN);
    }
  }
  __syncthreads();
  const float c = kLog2e / a.temperature;
  OnlineSum acc;
  // NaN logits: the first pass takes them as they come, and a run whose sum is
  // NaN is taken again with each of them read as -inf.
  bool dirty = false;
  float2 mine_ms;
#pragma unroll 1
  for (;;) {
    acc.init(c);
    run.template stream<kFirst>(first, [&](int u, typename Run<TIn, T>::Stage& v) {
      float um = kNegInf;
#pragma unroll
      for (int k = 0; k < kStage; ++k) {
        const int uk = u + k * T;
        const uint32_t word = uk - lane < run.n ? bits[uk >> 5] : 0u;  // the warp's 32 units
        if (word >> lane & 1u) Unit<TIn>::drop(v[k], held_entries(sh, uk));
        if (dirty) Unit<TIn>::clean(v[k]);
        um = fmaxf(um, Unit<TIn>::max(v[k]));
      }
      acc.raise(um);
#pragma unroll
      for (int k = 0; k < kStage; ++k) acc.template add<TIn>(v[k]);
    });
    mine_ms = block_lse<T / 32>(acc.x.m, acc.sum(), c, sh.red);
    if (dirty || mine_ms.y == mine_ms.y) break;  // the same in every thread of the CTA
    dirty = true;
    run.template prefetch<kFirst>(tid, first);
    __syncthreads();  // sh.red is read
  }
  let_next_start();
#pragma unroll
  for (int q = 0; q < kOwn; ++q) {
    const int k = tid + q * T;
    sh.lp[k] = t[q];
    sh.p[k] = id[q] >= 0 ? expf(t[q]) : 0.f;
    sh.x[k] = guard(E::get(x[q]));
    if (id[q] >= 0 && run.place(id[q]) < 0) id[q] = -1;  // from here on: those of this run
  }
  if (C > 1) {
    cluster_wait();  // every CTA of the cluster runs
    if (tid < C) peer_store2(peer_addr(smem_addr(&sh.ms[rank]), tid), mine_ms.x, mine_ms.y);
    cluster_arrive();
    cluster_wait();
  } else {
    if (tid == 0) sh.ms[0] = mine_ms;
    __syncthreads();
  }
  if (tid < 32) {  // the row's scalars, in each CTA from the same numbers
    constexpr int kPer = LS_MAX_TOP / 32;
    const float2 ms = lane < C ? sh.ms[lane] : make_float2(kNegInf, 0.f);
    const float Mr = warp_max(ms.x);
    const float Sr = Mr > kNegInf ? warp_reduce(ms.x > kNegInf ? ms.y * rel_exp(ms.x, Mr, c) : 0.f, OpAddF()) : 0.f;
    float xk[kPer], mt = kNegInf, P = 0.f;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      xk[q] = sh.x[lane + 32 * q];
      mt = fmaxf(mt, xk[q]);
      P += sh.p[lane + 32 * q];
    }
    const float M = fmaxf(Mr, warp_max(mt));
    P = warp_reduce(P, OpAddF());
    float total = 0.f;
    if (M > kNegInf) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) total += xk[q] > kNegInf ? rel_exp(xk[q], M, c) : 0.f;
    }
    total = warp_reduce(total, OpAddF());
    const float rest = Mr > kNegInf ? rel_exp(Mr, M, c) : 0.f;
    total += Sr * rest;
    float A = P, scale = 1.f, pr = 0.f;
    if (a.tail == LS_TAIL_RENORM) {
      const bool some = P >= kLeastMass;
      A = some ? 1.f : 0.f;
      scale = some ? 1.f / P : 0.f;
    } else if (a.tail == LS_TAIL_BUCKET && Mr > kNegInf) {
      pr = fmaxf(1.f - P, 0.f);
      A = P + pr;
    }
    RowStats st = {M, A / total, Mr, 0.f, scale, {}};
    if (Mr > kNegInf) st.kappa = st.alpha * rest - (pr > 0.f ? pr / Sr : 0.f);
    if (M == kNegInf) st.alpha = st.kappa = quiet_nan();
    if (lane == 0) sh.st = st;
    if (rank == 0) {
      const float lnS = logf(total), lnP = a.tail == LS_TAIL_RENORM ? logf(P) : 0.f;
      float kl = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float pk = sh.p[lane + 32 * q] * scale;
        if (pk > 0.f)
          kl += pk * ((sh.lp[lane + 32 * q] - lnP) - ((xk[q] == M ? 0.f : (xk[q] - M) / a.temperature) - lnS));
      }
      if (lane == 0 && pr > 0.f) kl += pr * (logf(pr) - ((Mr == M ? 0.f : (Mr - M) / a.temperature) + logf(Sr / total)));
      kl = warp_reduce(kl, OpAddF());
      if (lane == 0) {
        a.out_loss[i] = M == kNegInf ? quiet_nan() : w * kl;
        if (a.out_stats) a.out_stats[i] = st;
        if (a.error_word && M == kNegInf) atomicOr(a.error_word, LS_ROW_ERR_NO_FINITE);
      }
    }
  }
  if (kGrad) {
    // From the run's end: what was read last is the likeliest to be in L2.
    if (run.n > 0) run.template prefetch<LOAD_PLAIN>(run.last_stage(), first);
    __syncthreads();
    const RowStats st = sh.st;
    const float g = w / a.temperature;
    ExpAgainst against;
    against.init(st.Mr, c);
    const float coef = g * st.kappa * against.scale;
    const bool same = run.aligned_with(grad);
    if (run.n > 0)
      run.template stream_back<LOAD_PLAIN>(first, [&](int u, typename Run<TIn, T>::Stage& v) {
        const bool whole = run.whole(u) && same;
#pragma unroll
        for (int k = 0; k < kStage; ++k) {
          const int uk = u + k * T;
          if (dirty) Unit<TIn>::clean(v[k]);
          unit_grad<TIn>(v[k], against, coef);
          if (whole)
            store32(grad + run.index(uk), v[k]);
          else if (uk < run.n)
            run.store(grad, same, uk, v[k]);
        }
      });
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kOwn; ++q)
      if (id[q] >= 0) {
        const int k = tid + q * T;
        grad[id[q]] = E::put(g * (st.alpha * rel_exp(sh.x[k], st.M, c) - sh.p[k] * st.scale));
      }
  }
}

// The backward pass alone, in runs of a row.  In place (the gradient may replace
// the logits) each unit is read before the same thread writes it, and the logits
// at the ids are read before anything is written.  Bound by DRAM: 2048 x 128256
// bf16 156 us (6.7 TB/s, the measured copy rate), 1024 x 262144 fp32 312 us; 193
// and 313 in tiles of 512 units held in registers, which pay a tile's start and
// ids for 16 KB.  Runs of 1024 units 160 and 322 us, of 4096 162 and 315.  Batches
// that would leave SMs idle have runs of one stage.
constexpr int kBackThreads = 256;
constexpr int kBackRun = 2048;  // units of a CTA's run
static_assert(kBackThreads >= LS_MAX_TOP, "a thread per teacher entry");

template <typename TIn>
__global__ void __launch_bounds__(kBackThreads, 4) distill_backward_kernel(const DistillArgs a, int runs, int upc) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)runs;
  wait_for_previous();
  let_next_start();
  Run<TIn, kBackThreads> run;
  run.init(a.logits, i, a.row_stride, a.vocab, upc, (int)(blockIdx.x % (unsigned)runs));
  Raw* grad = static_cast<Raw*>(a.out_grad) + i * a.grad_stride;
  const float w = a.weights ? a.weights[i] : 1.f;
  const float g = w * (a.grad_loss ? a.grad_loss[i] : 1.f) / a.temperature;
  const bool same = run.aligned_with(grad);
  if (w == 0.f || g == 0.f) {  // a row of weight 0 counts nothing, whatever the gradient of its loss
    uint32_t z[8] = {};
    for (int u = tid; u < run.n; u += kBackThreads) run.store(grad, same, u, z);
    return;
  }
  typename Run<TIn, kBackThreads>::Stage first;
  run.template prefetch<LOAD_PLAIN>(tid, first);
  const RowStats st = a.stats_in[i];
  const float c = kLog2e / a.temperature;
  int id = -1;
  float x = kNegInf, p = 0.f;
  if (tid < a.t.k) {
    id = a.t.ids[i * a.t.stride + tid];
    const float t = a.t.log_probs[i * a.t.stride + tid];
    if (id < 0 || (int64_t)id >= a.vocab || !(t > kNegInf) || run.place(id) < 0) id = -1;
    if (id >= 0) {
      p = expf(t) * st.scale;
      x = guard(E::get(run.row[id]));
    }
  }
  const float top = g * (st.alpha * rel_exp(x, st.M, c) - p);
  ExpAgainst against;
  against.init(st.Mr, c);
  const float coef = g * st.kappa * against.scale;
  __syncthreads();
  run.template stream<LOAD_PLAIN>(first, [&](int u, typename Run<TIn, kBackThreads>::Stage& v) {
    const bool whole = run.whole(u) && same;
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const int uk = u + k * kBackThreads;
      Unit<TIn>::clean(v[k]);
      unit_grad<TIn>(v[k], against, coef);
      if (whole)
        store32(grad + run.index(uk), v[k]);
      else if (uk < run.n)
        run.store(grad, same, uk, v[k]);
    }
  });
  __syncthreads();
  if (id >= 0) grad[id] = E::put(top);
}

// Bytes of a CTA's run at most.  In the call that reads it twice the runs in
// flight share L2 with the gradients being written: 2048 x 128256 bf16 takes 204
// us with runs of up to 128 KB, 227 with 256 KB and 215 with 64 KB.
constexpr int64_t kRunTwice = 128 * 1024;
constexpr int64_t kRunOnce = 640 * 1024;

// CTAs of 256 threads, four to an SM (128 threads, eight to an SM: 42 us against
// 34 on 672 x 151936 bf16, whose rows then leave an SM 18 warps).
constexpr int kDistillThreads = 256;

template <typename TIn, bool kGrad>
static ls_status launch(const DistillArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const StreamPlan plan = plan_stream(n, a.vocab, dtype, kGrad ? kRunTwice : kRunOnce, 512 / kDistillThreads);
  const size_t smem = ((size_t)plan.upc + 127) / 128 * 16;  // a bit per unit
  return launch_rows(distill_kernel<TIn, kGrad, kDistillThreads>, a, plan, kDistillThreads, smem, n, st, done);
}

template <bool kGrad>
static ls_status dispatch(const DistillArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == LS_DTYPE_BF16 ? launch<bf16_tag, kGrad>(a, dtype, n, st) : launch<float, kGrad>(a, dtype, n, st);
}

static ls_status dispatch_backward(const DistillArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t units = row_units(a.vocab, dtype);
  const int sms = device_attr<cudaDevAttrMultiProcessorCount>();
  const int upc = (units + kBackRun - 1) / kBackRun * n >= 8 * sms ? kBackRun : kBackThreads * kStage;
  const int64_t runs = (units + upc - 1) / upc;
  if (runs * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(runs * n));
  return dtype == LS_DTYPE_BF16
             ? launch_kernel(distill_backward_kernel<bf16_tag>, grid, kBackThreads, 1, 0, st, a, (int)runs, upc)
             : launch_kernel(distill_backward_kernel<float>, grid, kBackThreads, 1, 0, st, a, (int)runs, upc);
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
                      weights, nullptr, nullptr,    out_loss, reinterpret_cast<RowStats*>(out_stats),
                      nullptr, 0,       error_word};
  return dispatch<false>(a, dtype, n, stream);
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
                      weights,  grad_loss, reinterpret_cast<const RowStats*>(stats), nullptr, nullptr,
                      out_grad, grad_stride, nullptr};
  return dispatch_backward(a, dtype, n, stream);
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
  return dispatch<true>(a, dtype, n, stream);
}

}  // extern "C"
