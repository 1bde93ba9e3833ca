// ls_top.cu -- the k best entries of each logits row, their log-probs and the
// row's log-sum-exp (ls_top_log_probs).
//
// A row over the CTAs of a cluster (ls_stream.cuh).  Per row:
//  1. One pass: each thread's running maximum and sum of exponentials, and in
//     shared memory the maximum of each stage (a few units of a thread), as the
//     upper 16 bits of its order-preserving key: exact for bf16, rounded down
//     in key order for fp32, so that a maximum at or above v keeps a key at or
//     above that of v.
//  2. A lower bound of the k-th largest entry.  In each of the w warps that hold
//     units, the ceil(k / w)-th largest lane maximum: at least k entries of the
//     run are at or above the least of these.  For large k that is far below
//     the k-th entry (k = 256: the least of all lane maxima), so the bound is
//     raised to about the k-th largest stage maximum (tighten).  The largest
//     bound over the cluster's CTAs is one too: (max, sum, bound) are exchanged
//     over the cluster.
//  3. The stages whose maximum reaches the bound are read again and their
//     entries at or above it collected as 64-bit keys (value, then lower index).
//     More than kLocal of them -- ties in the main: constant rows, rows masked
//     with one low value -- are cut to the run's own k best (select_ties).
//  4. The keys go to the first CTA's shared memory (over its stage maxima, which
//     every CTA is done with), which ranks them and writes the k best.
#include "ls_stream.cuh"

namespace lsg {
namespace ops {

constexpr int kLocal = 512;      // keys that a CTA sends at most
constexpr int kCandidates = 512;  // stages listed for the second read
constexpr int kTakeMost = 16;     // lane maxima of a warp taken away one by one
constexpr int kRankMost = 384;   // keys placed by counting; more are sorted
static_assert(kLocal >= LS_MAX_TOP, "a run's own k best must fit");

struct TopArgs {
  const void* logits;
  int64_t logits_rows, vocab, row_stride;
  const int32_t* gather;
  int32_t k;
  float temperature;
  int32_t* out_ids;
  float* out_lp;
  float* out_lse;
  int32_t* error_word;
};

constexpr int kMostWarps = 8;

struct TopShared {
  float2 ms[kMaxCluster];
  float2 red[kMostWarps];
  float bound[kMaxCluster];
  float redf[kMostWarps];
  int warp_n[kMostWarps];
  int candidates;               // stages that reach the bound
  uint32_t stage[kCandidates];  // the first of them
  unsigned int total;  // keys sent to this CTA
  int count;           // keys of this CTA
  int base;            // their place among those sent
  alignas(16) unsigned long long keys[kLocal];
};

// Block-wide sum of small counts.
template <int kWarps>
__device__ __forceinline__ int block_count(int v, int* red) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xFFFFFFFFu, (threadIdx.x & 31) < kWarps ? red[threadIdx.x & 31] : 0);
}

__device__ __forceinline__ uint16_t stage_key(float v) { return (uint16_t)(f32_key(v) >> 16); }

// f(value, place in the run) for each entry at or above `least` of the stage that
// begins with unit u and has the words w.  Few are: their bits are gathered
// first and then walked, in little code (code that runs once per row is paid for
// in instruction fetches).
template <typename TIn, int T, typename F>
__device__ __forceinline__ void visit_words(const Run<TIn, T>& run, int u, const typename Run<TIn, T>::Stage& w, float least,
                                            F f) {
  constexpr int kN = Unit<TIn>::kN;
  uint32_t hits[kStage];
#pragma unroll
  for (int k = 0; k < kStage; ++k) {
    hits[k] = 0u;
    if (u + k * T >= run.n) break;
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float x, y;
      unpack2(Unit<TIn>::pair(w[k], q), x, y);
      hits[k] |= (x >= least ? 1u : 0u) << (2 * q) | (y >= least ? 2u : 0u) << (2 * q);
    }
  }
  // Their values by a chain of selects: an index into the words would put them,
  // and with them the whole stream, into local memory.
#pragma unroll
  for (int k = 0; k < kStage; ++k)
#pragma unroll 1
    for (uint32_t h = u + k * T < run.n ? hits[k] : 0u; h; h &= h - 1) {
      const int e = __ffs((int)h) - 1;
      f(entry_at<TIn>(w[k], e), (u + k * T) * kN + e);
    }
}

// Visits the run's entries whose stage maximum is at least `least`.
template <typename TIn, int T, typename F>
__device__ __forceinline__ void visit_stages(const Run<TIn, T>& run, const uint16_t* stages, float least, F f) {
  const uint16_t least_key = stage_key(least);
  for (int b = threadIdx.x, u = threadIdx.x; u < run.n; b += T, u += kStage * T)
    if (stages[b] >= least_key) {
      typename Run<TIn, T>::Stage w;
#pragma unroll
      for (int k = 0; k < kStage; ++k)
        if (u + k * T < run.n) run.load(u + k * T, w[k]);
      visit_words<TIn, T>(run, u, w, least, f);
    }
}

// The run's k best exactly, for any number of ties: `bound` has at least k
// entries at or above it.  If fewer than k lie above it, it is the k-th largest
// value; else that is found by bisection of the keys above it.  Entries above
// the cut all belong to the answer, and of those equal to it the lowest
// indices, taken in order of the run.
template <typename TIn, int T>
__device__ __noinline__ void select_ties(const Run<TIn, T>& run, const uint16_t* stages, int k, float bound, TopShared& sh) {
  constexpr int kN = Unit<TIn>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto above = [&](uint32_t key) {  // entries whose key is above `key`
    int n = 0;
    visit_stages<TIn, T>(run, stages, f32_from_key(key), [&](float v, int) { n += guard(v) == v && f32_key(v) > key; });
    return block_count<T / 32>(n, sh.warp_n);
  };
  uint32_t cut = max(f32_key(bound), f32_key(kNegInf) + 1u);  // -inf is never listed
  if (above(cut) >= k) {
    uint32_t lo = cut, hi = f32_key(kPosInf);  // at least k keys are above lo, fewer than k above hi
    while (hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2u;
      if (above(mid) >= k)
        lo = mid;
      else
        hi = mid;
    }
    cut = hi;
  }
  const float cut_value = f32_from_key(cut);
  __syncthreads();
  if (tid == 0) sh.count = 0;
  __syncthreads();
  visit_stages<TIn, T>(run, stages, cut_value, [&](float v, int place) {
    if (v > cut_value) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kLocal) sh.keys[at] = argmax_key(v, run.j0 + place);
    }
  });
  __syncthreads();
  int have = sh.count;  // fewer than k
  for (int u0 = 0; u0 < run.n && have < k; u0 += T) {
    const int u = u0 + tid;
    float v[kN];
    int n = 0;
    if (u < run.n) {
      uint32_t w[8];
      run.load(u, w);
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) unpack2(Unit<TIn>::pair(w, q), v[2 * q], v[2 * q + 1]);
#pragma unroll
      for (int e = 0; e < kN; ++e) n += v[e] == cut_value;
    }
    int before = n;  // ties up to and with this lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, before, o);
      if (lane >= o) before += t;
    }
    __syncthreads();
    if (lane == 31) sh.warp_n[warp] = before;
    __syncthreads();
    int at = have + before - n, all = 0;
#pragma unroll
    for (int q = 0; q < (T / 32); ++q) {
      if (q < warp) at += sh.warp_n[q];
      all += sh.warp_n[q];
    }
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (v[e] == cut_value) {
          if (at < k) sh.keys[at] = argmax_key(v[e], run.index(u) + e);
          ++at;
        }
    }
    have = min(have + all, k);
  }
  __syncthreads();
  if (tid == 0) sh.count = have;
  __syncthreads();
}

// A value with at least k stage maxima at or above it and, where values allow,
// at most k / 8 more (-inf where there are fewer than k): bisection of the
// 16-bit keys up to the run's maximum.
template <int T>
__device__ __noinline__ float tighten(int units, const uint16_t* stages, int k, float most, TopShared& sh) {
  uint32_t lo = stage_key(kNegInf), hi = stage_key(most) + 1u;
  while (hi - lo > 1u) {
    const uint32_t mid = lo + (hi - lo) / 2u;
    int n = 0;
    for (int b = threadIdx.x, u = threadIdx.x; u < units; b += T, u += kStage * T)
      n += stages[b] >= mid;
    n = block_count<T / 32>(n, sh.warp_n);
    if (n >= k) {
      lo = mid;
      if (n <= k + k / 8) break;
    } else {
      hi = mid;
    }
  }
  return lo == stage_key(kNegInf) ? kNegInf : f32_from_key(lo << 16);
}

// Descending sort of n keys in shared memory (n a power of two).
template <int T>
__device__ __noinline__ void sort_keys(unsigned long long* keys, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += T) {
        const int a = 2 * t - (t & (stride - 1)), b = a + stride;
        const unsigned long long x = keys[a], y = keys[b];
        if ((x < y) == ((a & size) == 0)) {
          keys[a] = y;
          keys[b] = x;
        }
      }
    }
  __syncthreads();
}

// Bound by DRAM while rows stream and by the latency of steps 2 to 4 while they
// do not; several rows on an SM cover each other's, but the steps after the last
// rows' streams run alone.  20 best of 672 x 151936 bf16 take 44 us (4.6 TB/s, 0.69
// of the measured copy rate), 64 of 2048 x 128256 bf16 100 us (5.3 TB/s, 0.79), 64
// of 1024 x 262144 fp32 184 us (5.8 TB/s, 0.87), 5 of 4 x 1000 fp32 6.2 us a call.
// On few rows the steps after the stream decide, which grow with k: 1 / 20 / 64 / 128
// / 256 best of 4 x 262144 bf16 take 9.3 / 12.8 / 24 / 41 / 77 us.  A thread's own
// best stage is read again without being listed first: 44 us against 49 on the first
// of these.
template <typename TIn, int T>
__global__ void __launch_bounds__(T, 1024 / T) top_kernel(const TopArgs a, int upc) {
  extern __shared__ uint4 dyn_smem[];  // keys of the stage maxima, then the entries sent to the first CTA
  __shared__ TopShared sh;
  uint16_t* stages = reinterpret_cast<uint16_t*>(dyn_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  const int k = a.k;
  wait_for_previous();
  const int64_t src = a.gather ? a.gather[i] : i;
  int32_t* ids = a.out_ids + i * k;
  float* lp = a.out_lp + i * k;
  auto fail = [&](int32_t bit) {
    for (int q = tid; q < k; q += T) {
      ids[q] = -1;
      lp[q] = quiet_nan();
    }
    if (tid == 0) {
      if (a.out_lse) a.out_lse[i] = quiet_nan();
      if (a.error_word) atomicOr(a.error_word, bit);
    }
  };
  if (src < 0 || src >= a.logits_rows) {  // every CTA of the row leaves here, before any cluster barrier
    if (rank == 0) fail(LS_ROW_ERR_BAD_GATHER);
    return;
  }
  Run<TIn, T> run;
  run.init(a.logits, src, a.row_stride, a.vocab, upc, rank);
  typename Run<TIn, T>::Stage first;
  run.prefetch(tid, first);
  if (C > 1) cluster_arrive();
  if (tid == 0) {
    sh.count = sh.candidates = 0;
    sh.total = 0u;
  }
  if (run.n > 0) stages[(run.n - 1) / (kStage * T) * T + tid] = 0;  // the last stage need not have units of every warp
  const float c = kLog2e / a.temperature;
  float mine;  // this thread's maximum, and the stage that holds it
  int best;
  float2 mine_ms;
  // NaN logits: the first pass takes them as they come, and a run whose sum is
  // NaN is taken again with each of them read as -inf.
#pragma unroll 1
  for (bool dirty = false;; dirty = true) {
    OnlineSum acc;
    acc.init(c);
    mine = kNegInf;
    best = -1;
    run.stream(first, [&](int u, typename Run<TIn, T>::Stage& v) {
      float um = kNegInf;
#pragma unroll
      for (int q = 0; q < kStage; ++q) {
        if (dirty) Unit<TIn>::clean(v[q]);
        um = fmaxf(um, Unit<TIn>::max(v[q]));
      }
      // u = tid + stage * kStage * T
      stages[(u - tid) / kStage + tid] = stage_key(um);
      if (um > mine) {
        mine = um;
        best = u;
      }
      acc.raise(um);
#pragma unroll
      for (int q = 0; q < kStage; ++q) acc.template add<TIn>(v[q]);
    });
    mine_ms = block_lse<T / 32>(acc.x.m, acc.sum(), c, sh.red);
    if (dirty || mine_ms.y == mine_ms.y) break;  // the same in every thread of the CTA
    run.prefetch(tid, first);
    __syncthreads();  // sh.red is read
  }
  let_next_start();
  // Most stages that reach the bound are some thread's best (for k = 64 of 128256
  // entries 73 of 107, for k = 20 34 of 38): read those again while the bound is
  // worked out.
  if (best >= 0) {
#pragma unroll
    for (int q = 0; q < kStage; ++q)
      if (best + q * T < run.n) run.load(best + q * T, first[q]);
  }
  const int warps = min((T / 32), (run.n + 31) / 32);
  float bound = kPosInf;
  if (warp < warps) {
    const int j = (k + warps - 1) / warps;
    if (j <= kTakeMost) {  // take the largest away j - 1 times
      float left = mine;
      for (int q = 1; q < j; ++q) {
        const unsigned int at = __ballot_sync(0xFFFFFFFFu, left == warp_max(left));
        if (lane == __ffs((int)at) - 1) left = kNegInf;
      }
      bound = warp_max(left);
    } else {
      bound = kNegInf;  // tighten() starts from nothing
    }
  }
  if (lane == 0) sh.redf[warp] = bound;
  __syncthreads();
  bound = run.n > 0 ? warp_min(sh.redf[tid & ((T / 32) - 1)]) : kNegInf;
  if (run.n > 0 && (k + warps - 1) / warps > kTakeMost) bound = tighten<T>(run.n, stages, k, mine_ms.x, sh);
  if (C > 1) {
    cluster_wait();  // every CTA of the cluster runs
    if (tid < C) {
      peer_store2(peer_addr(smem_addr(&sh.ms[rank]), tid), mine_ms.x, mine_ms.y);
      peer_store(peer_addr(smem_addr(&sh.bound[rank]), tid), bound);
    }
    cluster_arrive();
    cluster_wait();
  } else {
    if (tid == 0) {
      sh.ms[0] = mine_ms;
      sh.bound[0] = bound;
    }
    __syncthreads();
  }
  const float2 ms = lane < C ? sh.ms[lane] : make_float2(kNegInf, 0.f);
  const float M = warp_max(ms.x);
  if (M == kNegInf) {  // the same in every CTA
    if (rank == 0) fail(LS_ROW_ERR_NO_FINITE);
    return;
  }
  bound = warp_max(lane < C ? sh.bound[lane] : kNegInf);
  auto take = [&](float v, int place) {
    if (v > kNegInf) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kLocal) sh.keys[at] = argmax_key(v, run.j0 + place);
    }
  };
  // The other stages are listed first (eight keys of any thread's at a time) and
  // then read again, one per thread: a thread reading its own as it met them
  // would wait for memory once per stage.
  const uint16_t bound_key = stage_key(bound);
  const int own = (best - tid) / kStage + tid;  // the place of this thread's best stage
  const bool has_own = best >= 0 && stage_key(mine) >= bound_key;
  if (has_own) stages[own] = 0;
  __syncthreads();
  const int slots = (run.n + kStage * T - 1) / (kStage * T) * T;
  for (int q = tid * 8; q < slots; q += T * 8) {
    const uint4 eight = *reinterpret_cast<const uint4*>(&stages[q]);
    const uint32_t words[4] = {eight.x, eight.y, eight.z, eight.w};
    uint32_t hits = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hits |= ((words[k] & 0xFFFFu) >= bound_key ? 1u : 0u) << (2 * k);
      hits |= ((words[k] >> 16) >= bound_key ? 1u : 0u) << (2 * k + 1);
    }
    for (; hits; hits &= hits - 1) {
      const int at = atomicAdd(&sh.candidates, 1);
      if (at < kCandidates) sh.stage[at] = (uint32_t)(q + __ffs((int)hits) - 1);
    }
  }
  __syncthreads();
  const int listed = sh.candidates;
  int u = has_own ? best : -1;
#pragma unroll 1
  for (int q = tid;; q += T) {  // its own, then of the list
    if (u >= 0) visit_words<TIn, T>(run, u, first, bound, take);
    if (listed > kCandidates || q >= listed) break;
    const int b = (int)sh.stage[q], who = b % T;
    u = (b - who) * kStage + who;
#pragma unroll
    for (int k = 0; k < kStage; ++k)
      if (u + k * T < run.n) run.load(u + k * T, first[k]);
  }
  if (listed > kCandidates) visit_stages<TIn, T>(run, stages, bound, take);
  __syncthreads();
  if (sh.count > kLocal) {
    if (has_own) stages[own] = stage_key(mine);
    __syncthreads();
    select_ties<TIn, T>(run, stages, k, bound, sh);
  }
  const int n_local = sh.count;
  // to the first CTA, over its stage maxima
  unsigned long long* all = reinterpret_cast<unsigned long long*>(dyn_smem);
  int n = n_local;
  if (C > 1) {
    if (tid == 0) sh.base = (int)peer_add(peer_addr(smem_addr(&sh.total), 0), (uint32_t)n_local);
    cluster_arrive();
    cluster_wait();  // every CTA is done with its stage maxima
    const int base = sh.base;
    for (int q = tid; q < n_local; q += T) peer_store(peer_addr(smem_addr(&all[base + q]), 0), sh.keys[q]);
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    n = (int)sh.total;
  } else if (n <= kRankMost) {
    all = sh.keys;
  } else {
    for (int q = tid; q < n; q += T) all[q] = sh.keys[q];
    __syncthreads();
  }
  const float total = warp_reduce(ms.x > kNegInf ? ms.y * rel_exp(ms.x, M, c) : 0.f, OpAddF());
  const float lnS = logf(total);
  auto put = [&](int at, unsigned long long key) {
    const float v = f32_from_key((uint32_t)(key >> 32));
    ids[at] = argmax_index(key);
    lp[at] = (v == M ? 0.f : (v - M) / a.temperature) - lnS;
  };
  if (n <= kRankMost) {
    if (tid == 0 && (n & 1)) all[n] = 0ull;  // pairs: below every key
    __syncthreads();
    for (int q = tid; q < n; q += T) {
      const unsigned long long key = all[q];
      int at = 0;
#pragma unroll 4
      for (int o = 0; o < n; o += 2) {
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&all[o]);
        at += (two.x > key) + (two.y > key);
      }
      if (at < k) put(at, key);
    }
  } else {
    int size = 1;
    while (size < n) size <<= 1;
    for (int q = n + tid; q < size; q += T) all[q] = 0ull;  // below every key
    sort_keys<T>(all, size);
    for (int q = tid; q < min(n, k); q += T) put(q, all[q]);
  }
  for (int q = n + tid; q < k; q += T) {
    ids[q] = -1;
    lp[q] = kNegInf;
  }
  if (tid == 0 && a.out_lse) a.out_lse[i] = M / a.temperature + lnS;
}

// CTAs of 128 threads, eight to an SM: with 256 threads a row's steps after the
// stream ran beside fewer others (top 20 of 672 x 151936 bf16 50 us against 41).
constexpr int kTopThreads = 128;
constexpr int64_t kRunTop = 640 * 1024;  // bytes of a CTA's run at most

template <typename TIn>
static ls_status launch_top(const TopArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const StreamPlan plan = plan_stream(n, a.vocab, dtype, kRunTop, 512 / kTopThreads);
  // a key per stage of every thread; the entries of every CTA, padded to a power of two
  const size_t stages = ((size_t)plan.upc + kStage * kTopThreads - 1) / (kStage * kTopThreads);
  const size_t maxima = stages * kTopThreads * sizeof(uint16_t);
  const size_t keys = (size_t)plan.ctas * kLocal * sizeof(unsigned long long);
  return launch_rows(top_kernel<TIn, kTopThreads>, a, plan, kTopThreads, maxima > keys ? maxima : keys, n, st, done);
}

}  // namespace ops
}  // namespace lsg

using namespace lsg;
using namespace lsg::ops;

extern "C" ls_status ls_top_log_probs(const void* logits, ls_dtype dtype, int64_t logits_rows, int64_t vocab,
                                      int64_t row_stride, int32_t n, const int32_t* gather_indices, int32_t k,
                                      float temperature, int32_t* out_ids, float* out_log_probs, float* out_lse,
                                      int32_t* error_word, void* stream) {
  if (n < 0 || k < 1 || !(temperature > 0.f) || temperature > 3.4028235e38f) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!matrix_ok(logits, dtype, vocab, row_stride) || logits_rows < 1 || !out_ids || !out_log_probs || k > vocab ||
      k > LS_MAX_TOP)
    return LS_ERR_INVALID_ARG;
  if (!gather_indices && (int64_t)n > logits_rows) return LS_ERR_INVALID_ARG;
  if (vocab > max_row(dtype)) return LS_ERR_UNSUPPORTED;
  TopArgs a{logits,      logits_rows, vocab,         row_stride, gather_indices, k,
            temperature, out_ids,     out_log_probs, out_lse,    error_word};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == LS_DTYPE_BF16 ? launch_top<bf16_tag>(a, dtype, n, st) : launch_top<float>(a, dtype, n, st);
}

extern "C" int64_t ls_row_ops_max_vocab(ls_dtype dtype) {
  if (device_attr<cudaDevAttrMaxSharedMemoryPerBlockOptin>() <= 0) return 0;
  return max_row(dtype);
}
