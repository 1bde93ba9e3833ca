// ls_distill.cu -- the distillation loss from a teacher's top log-probs and
// its gradient (ls_distill_loss, ls_distill_loss_backward,
// ls_distill_loss_grad).
//
// Loss, and loss with gradient (distill_kernel): the row lies in the shared
// memory of a cluster (ls_slice.cuh) and is read from global memory once.  The
// teacher's entries are taken out of it first (their logits go to every CTA,
// their places become -inf), so the sums that follow run over the entries
// outside them, and the mass outside (q_r) is a sum of its own rather than a
// difference of two.  With R the row's entries outside the ids, of maximum
// M_r, and e_j = exp((x_j - M_r) / T), the gradient outside the ids is one
// multiple of e_j:
//     d_j = g / T * e_j * kappa,   kappa = A exp((M_r - M) / T) / S - p_r / S_r
// and the at most 256 ids follow one by one: g / T * (alpha exp((x - M) / T) -
// p), alpha = A / S.  M_r, kappa, M, alpha and the scale of p are the row's
// `stats`: the backward pass (distill_backward_kernel) reads them and nothing
// else of the forward pass, and is one sweep over the logits in tiles.
#include "ls_slice.cuh"

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

// Gradient of a unit outside the ids: coef * exp((x - m) / T).
template <typename TIn>
__device__ __forceinline__ uint4 unit_grad(uint4 w, const ExpAgainst& x, float coef_fast, float coef) {
  constexpr int kN = Unit<TIn>::kN;
  w = Unit<TIn>::clean(w);
  float d[kN];
  if (x.fast) {
#pragma unroll
    for (int q = 0; q < kN / 2; ++q)
      unpack2(mul2(x.pair_fast(Unit<TIn>::pair(w, q)), pack2(coef_fast, coef_fast)), d[2 * q], d[2 * q + 1]);
  } else {
#pragma unroll
    for (int q = 0; q < kN / 2; ++q)
      unpack2(mul2(x.pair_slow(Unit<TIn>::pair(w, q)), pack2(coef, coef)), d[2 * q], d[2 * q + 1]);
  }
  return Unit<TIn>::make(d);
}

__device__ __forceinline__ void store_unit(void* p, uint4 v) {
  asm volatile("st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Writes the slice's entries of an output row: unit by unit where the output
// row starts at the input row's alignment, else entry by entry.  `unit(u)`
// gives the 16 bytes that belong to the slice's unit u.
template <typename TIn, typename F>
__device__ __forceinline__ void write_slice(const Slice<TIn>& s, typename Elem<TIn>::Raw* out, F unit) {
  using Raw = typename Elem<TIn>::Raw;
  constexpr int kN = Unit<TIn>::kN;
  const int f = s.full_first(), l = s.full_last();
  const bool same = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(s.row)) & 15u) == 0;
  for (int u = threadIdx.x; u < s.n; u += kSliceThreads) {
    const uint4 v = unit(u);
    const int64_t j = s.index(u * kN);
    if (same && u >= f && u < l) {
      store_unit(out + j, v);
    } else {
      Raw e[kN];
      memcpy(e, &v, 16);
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (j + q >= 0 && j + q < s.V) out[j + q] = e[q];
    }
  }
}

// Everything of a row but its entries: written by warp 0 of each CTA from the
// same numbers, so every CTA holds the same bits.
struct RowShared {
  uint64_t bars[kChunks];
  float2 ms[kMaxCluster];  // each CTA's maximum and sum over the entries outside the ids
  float x[LS_MAX_TOP];     // the student's logits at the ids (-inf where there is none)
  float p[LS_MAX_TOP];
  float lp[LS_MAX_TOP];
  float red[kSliceWarps];
  RowStats st;
};

template <typename TIn, bool kGrad>
__global__ void __launch_bounds__(kSliceThreads, 3) distill_kernel(const DistillArgs a, int upc) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  extern __shared__ uint4 slice_smem[];
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  const float w = a.weights ? a.weights[i] : 1.f;
  Slice<TIn> s;
  s.init(slice_smem, a.logits, i, a.row_stride, a.vocab, upc, rank);
  Raw* grad = kGrad ? static_cast<Raw*>(a.out_grad) + i * a.grad_stride : nullptr;
  if (w == 0.f) {  // every CTA of the row leaves here, before any cluster barrier
    if (kGrad) write_slice<TIn>(s, grad, [](int) { return make_uint4(0u, 0u, 0u, 0u); });
    if (tid == 0 && rank == 0) {
      a.out_loss[i] = 0.f;
      if (a.out_stats) a.out_stats[i] = RowStats{0.f, 0.f, 0.f, 0.f, 1.f, {}};
    }
    return;
  }
  s.start(sh.bars);
  if (C > 1) cluster_arrive();  // the peers' shared memory may be written once all have arrived
  // the teacher's entry of this thread
  int id = -1;
  float x = kNegInf, p = 0.f;
  if (tid < LS_MAX_TOP) {
    float t = kNegInf;
    if (tid < a.t.k) {
      id = a.t.ids[i * a.t.stride + tid];
      t = a.t.log_probs[i * a.t.stride + tid];
      if (id < 0 || (int64_t)id >= a.vocab || !(t > kNegInf)) id = -1;
      if (id >= 0) p = expf(t);
    }
    sh.lp[tid] = t;
    sh.p[tid] = p;
    if (id < 0) sh.x[tid] = kNegInf;
  }
  bool stalled = false;
  for (int k = 0; k < kChunks; ++k)
    if (!mbar_wait(&sh.bars[k])) stalled = true;
  __syncthreads();
  if (C > 1) cluster_wait();
  const int mine = id >= 0 ? s.entry(id) : -1;
  if (mine >= 0) {
    x = guard(E::get(s.raw()[mine]));
    if (C > 1) {
      for (int q = 0; q < C; ++q) peer_store(peer_addr(smem_addr(&sh.x[tid]), q), x);
    } else {
      sh.x[tid] = x;
    }
    s.raw()[mine] = E::neg_inf();
  }
  __syncthreads();
  const float c = kLog2e / a.temperature;
  const float m = block_max(slice_max(s, sh.bars, &stalled), sh.red);
  ExpAgainst against;
  against.init(m, c);
  const float sum = block_sum(slice_sum(s, against), sh.red);
  if (tid < C) {
    if (C > 1)
      peer_store2(peer_addr(smem_addr(&sh.ms[rank]), tid), m, sum);
    else
      sh.ms[0] = make_float2(m, sum);
  }
  if (C > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (tid < 32) {
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
    float S = 0.f;
    if (M > kNegInf) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) S += xk[q] > kNegInf ? rel_exp(xk[q], M, c) : 0.f;
    }
    S = warp_reduce(S, OpAddF());
    const float rest = Mr > kNegInf ? rel_exp(Mr, M, c) : 0.f;
    S += Sr * rest;
    float A = P, scale = 1.f, pr = 0.f;
    if (a.tail == LS_TAIL_RENORM) {
      const bool some = P >= kLeastMass;
      A = some ? 1.f : 0.f;
      scale = some ? 1.f / P : 0.f;
    } else if (a.tail == LS_TAIL_BUCKET && Mr > kNegInf) {
      pr = fmaxf(1.f - P, 0.f);
      A = P + pr;
    }
    RowStats st = {M, A / S, Mr, 0.f, scale, {}};
    if (Mr > kNegInf) st.kappa = st.alpha * rest - (pr > 0.f ? pr / Sr : 0.f);
    if (M == kNegInf) st.alpha = st.kappa = quiet_nan();
    if (lane == 0) sh.st = st;
    __syncwarp();
    if (rank == 0) {
      const float lnS = logf(S), lnP = a.tail == LS_TAIL_RENORM ? logf(P) : 0.f;
      float kl = 0.f;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float pk = sh.p[lane + 32 * q] * scale;
        if (pk > 0.f)
          kl += pk * ((sh.lp[lane + 32 * q] - lnP) - ((xk[q] == M ? 0.f : (xk[q] - M) / a.temperature) - lnS));
      }
      if (lane == 0 && pr > 0.f) kl += pr * (logf(pr) - ((Mr == M ? 0.f : (Mr - M) / a.temperature) + logf(Sr / S)));
      kl = warp_reduce(kl, OpAddF());
      if (lane == 0) {
        a.out_loss[i] = M == kNegInf ? quiet_nan() : w * kl;
        if (a.out_stats) a.out_stats[i] = st;
        if (a.error_word && M == kNegInf) atomicOr(a.error_word, LS_ROW_ERR_NO_FINITE);
      }
    }
  }
  if (stalled && a.error_word) atomicOr(a.error_word, LS_ROW_ERR_STALLED);
  if (kGrad) {
    __syncthreads();
    const RowStats st = sh.st;
    const float g = w / a.temperature;
    against.init(st.Mr, c);
    const float coef = g * st.kappa;
    write_slice<TIn>(s, grad, [&](int u) { return unit_grad<TIn>(s.buf[u], against, coef * against.scale, coef); });
    __syncthreads();
    if (mine >= 0) grad[id] = E::put(g * (st.alpha * rel_exp(x, st.M, c) - p * st.scale));
  }
}

// The backward pass alone: a tile of kBackUnits units per thread, loaded to
// registers before anything is written (the gradient may replace the logits).
constexpr int kBackThreads = 256;
constexpr int kBackUnits = 4;

template <typename TIn>
__global__ void __launch_bounds__(kBackThreads) distill_backward_kernel(const DistillArgs a, int tiles) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  constexpr int kN = Unit<TIn>::kN;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)tiles;
  const int tile = (int)(blockIdx.x % (unsigned)tiles);
  Raw* grad = static_cast<Raw*>(a.out_grad) + i * a.grad_stride;
  const float g = (a.weights ? a.weights[i] : 1.f) * (a.grad_loss ? a.grad_loss[i] : 1.f) / a.temperature;
  Slice<TIn> s;  // of this tile, left in global memory
  s.init(nullptr, a.logits, i, a.row_stride, a.vocab, kBackThreads * kBackUnits, tile);
  const int f = s.full_first(), l = s.full_last();
  const RowStats st = a.stats_in[i];
  const float c = kLog2e / a.temperature;
  uint4 v[kBackUnits];
  if (g != 0.f) {
#pragma unroll
    for (int k = 0; k < kBackUnits; ++k) {
      const int u = tid + k * kBackThreads;
      const int64_t j = s.index(u * kN);
      if (u >= f && u < l) {
        asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                     : "l"(s.row + j));
      } else if (u < s.n) {
        Raw e[kN];
#pragma unroll
        for (int q = 0; q < kN; ++q) e[q] = j + q >= 0 && j + q < s.V ? s.row[j + q] : E::neg_inf();
        memcpy(&v[k], e, 16);
      }
    }
  }
  int id = -1;
  float x = kNegInf, p = 0.f;
  if (tid < a.t.k && g != 0.f) {
    id = a.t.ids[i * a.t.stride + tid];
    const float t = a.t.log_probs[i * a.t.stride + tid];
    if (id < 0 || (int64_t)id >= a.vocab || !(t > kNegInf) || s.entry(id) < 0) id = -1;
    if (id >= 0) {
      p = expf(t) * st.scale;
      x = guard(E::get(s.row[id]));
    }
  }
  ExpAgainst against;
  against.init(st.Mr, c);
  const float coef = g * st.kappa;
  const bool same = ((reinterpret_cast<uintptr_t>(grad) ^ reinterpret_cast<uintptr_t>(s.row)) & 15u) == 0;
  __syncthreads();  // every load of the tile is done
#pragma unroll
  for (int k = 0; k < kBackUnits; ++k) {
    const int u = tid + k * kBackThreads;
    if (u >= s.n) break;
    const uint4 d = g == 0.f ? make_uint4(0u, 0u, 0u, 0u) : unit_grad<TIn>(v[k], against, coef * against.scale, coef);
    const int64_t j = s.index(u * kN);
    if (same && u >= f && u < l) {
      store_unit(grad + j, d);
    } else {
      Raw e[kN];
      memcpy(e, &d, 16);
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (j + q >= 0 && j + q < s.V) grad[j + q] = e[q];
    }
  }
  __syncthreads();
  if (id >= 0) grad[id] = E::put(g * (st.alpha * rel_exp(x, st.M, c) - p));
}

template <typename TIn, bool kGrad>
static ls_status launch(const DistillArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const SlicePlan plan = plan_slices(n, a.vocab, dtype);
  return launch_slices(distill_kernel<TIn, kGrad>, a, plan, plan.smem, n, st, done);
}

template <bool kGrad>
static ls_status dispatch(const DistillArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == LS_DTYPE_BF16 ? launch<bf16_tag, kGrad>(a, dtype, n, st) : launch<float, kGrad>(a, dtype, n, st);
}

static ls_status dispatch_backward(const DistillArgs& a, ls_dtype dtype, int32_t n, void* stream) {
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t e = dtype == LS_DTYPE_F32 ? 4 : 2;
  const int64_t units = (a.vocab * e + 15 - e) / 16 + 1;
  const int64_t tiles = (units + kBackThreads * kBackUnits - 1) / (kBackThreads * kBackUnits);
  if (tiles * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(tiles * n)), block(kBackThreads);
  if (dtype == LS_DTYPE_BF16)
    distill_backward_kernel<bf16_tag><<<grid, block, 0, st>>>(a, (int)tiles);
  else
    distill_backward_kernel<float><<<grid, block, 0, st>>>(a, (int)tiles);
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
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
