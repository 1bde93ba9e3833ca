// ls_top.cu -- the k best entries of each logits row, their log-probs and the
// row's log-sum-exp (ls_top_log_probs).
//
// The row lies in the shared memory of a cluster (ls_slice.cuh), read from
// global memory once.  Per row:
//  1. Each thread's maximum and the CTA's sum of exponentials.  In each of the w
//     warps that hold entries, the ceil(k / w)-th largest lane maximum: at least
//     k entries of the slice are at or above the least of these, so that is a
//     lower bound of the k-th largest entry, and the largest such bound over
//     the cluster's CTAs is one too.
//  2. (max, sum, bound) are exchanged over the cluster; each CTA collects its
//     entries at or above the bound as 64-bit keys (value, then lower index).
//     More than kLocal of them -- ties in the main: constant rows, rows masked
//     with one low value -- are cut to the slice's own k best (select_ties).
//  3. The keys go to the first CTA's shared memory (over its slice, which every
//     CTA is done with), which ranks them and writes the k best.
#include "ls_slice.cuh"

namespace lsg {
namespace ops {

constexpr int kLocal = 512;      // keys that a CTA sends at most
constexpr int kRankMost = 384;   // keys placed by counting; more are sorted
static_assert(kLocal >= LS_MAX_TOP, "a slice's own k best must fit");

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

struct TopShared {
  uint64_t bars[kChunks];
  float2 ms[kMaxCluster];
  float bound[kMaxCluster];
  float red[kSliceWarps];
  int warp_n[kSliceWarps];
  unsigned int total;  // keys sent to this CTA
  int count;           // keys of this CTA
  int base;            // their place among those sent
  unsigned long long keys[kLocal];
};

// Block-wide sum of small counts.
__device__ __forceinline__ int block_count(int v, int* red) {
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xFFFFFFFFu, (threadIdx.x & 31) < kSliceWarps ? red[threadIdx.x & 31] : 0);
}

// The slice's entries of a predicate on (key, index), counted.
template <typename TIn, typename F>
__device__ __forceinline__ int count_entries(const Slice<TIn>& s, int* red, F test) {
  constexpr int kN = Unit<TIn>::kN;
  int n = 0;
  for (int u = threadIdx.x; u < s.n; u += kSliceThreads) {
    const uint4 w = Unit<TIn>::clean(s.buf[u]);
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float a, b;
      unpack2(Unit<TIn>::pair(w, q), a, b);
      n += (test(f32_key(a)) ? 1 : 0) + (test(f32_key(b)) ? 1 : 0);
    }
  }
  return block_count(n, red);
}

// The slice's k best exactly, for any number of ties: `bound` has at least k
// entries at or above it.  If fewer than k lie above it, it is the k-th largest
// value; else that is found by bisection of the keys above it.  Entries above
// the cut all belong to the answer, and of those equal to it the lowest
// indices, taken in order of the slice.
template <typename TIn>
__device__ void select_ties(const Slice<TIn>& s, int k, float bound, TopShared& sh) {
  constexpr int kN = Unit<TIn>::kN;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t low = f32_key(kNegInf);
  uint32_t cut = max(f32_key(bound), low + 1u);  // -inf is never listed
  uint32_t hi = 0xFFFFFFFFu;                     // fewer than k keys are above hi
  if (count_entries(s, sh.warp_n, [&](uint32_t key) { return key > cut; }) >= k) {
    uint32_t lo = cut;  // at least k keys are above lo
    while (hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2u;
      if (count_entries(s, sh.warp_n, [&](uint32_t key) { return key > mid; }) >= k)
        lo = mid;
      else
        hi = mid;
    }
    cut = hi;
  }
  __syncthreads();
  if (tid == 0) sh.count = 0;
  __syncthreads();
  for (int u = tid; u < s.n; u += kSliceThreads) {
    const uint4 w = Unit<TIn>::clean(s.buf[u]);
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float v[2];
      unpack2(Unit<TIn>::pair(w, q), v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (f32_key(v[e]) > cut) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kLocal) sh.keys[at] = argmax_key(v[e], s.index(u * kN + 2 * q + e));
        }
    }
  }
  __syncthreads();
  int have = sh.count;  // fewer than k
  for (int u0 = 0; u0 < s.n && have < k; u0 += kSliceThreads) {
    const int u = u0 + tid;
    float v[kN];
    int n = 0;
    if (u < s.n) {
      const uint4 w = Unit<TIn>::clean(s.buf[u]);
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) unpack2(Unit<TIn>::pair(w, q), v[2 * q], v[2 * q + 1]);
#pragma unroll
      for (int e = 0; e < kN; ++e) n += f32_key(v[e]) == cut;
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
    for (int q = 0; q < kSliceWarps; ++q) {
      if (q < warp) at += sh.warp_n[q];
      all += sh.warp_n[q];
    }
    if (n > 0) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (f32_key(v[e]) == cut) {
          if (at < k) sh.keys[at] = argmax_key(v[e], s.index(u * kN + e));
          ++at;
        }
    }
    have = min(have + all, k);
  }
  __syncthreads();
  if (tid == 0) sh.count = have;
  __syncthreads();
}

// Descending sort of n keys in shared memory (n a power of two).
__device__ void sort_keys(unsigned long long* keys, int n) {
  for (int size = 2; size <= n; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n / 2; t += kSliceThreads) {
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

template <typename TIn>
__global__ void __launch_bounds__(kSliceThreads, 3) top_kernel(const TopArgs a, int upc) {
  constexpr int kN = Unit<TIn>::kN;
  extern __shared__ uint4 slice_smem[];
  __shared__ TopShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int64_t i = blockIdx.x / (unsigned)C;
  const int k = a.k;
  const int64_t src = a.gather ? a.gather[i] : i;
  int32_t* ids = a.out_ids + i * k;
  float* lp = a.out_lp + i * k;
  auto fail = [&](int32_t bit) {
    for (int q = tid; q < k; q += kSliceThreads) {
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
  Slice<TIn> s;
  s.init(slice_smem, a.logits, src, a.row_stride, a.vocab, upc, rank);
  if (tid == 0) {
    sh.count = 0;
    sh.total = 0u;
  }
  s.start(sh.bars);
  if (C > 1) cluster_arrive();
  bool stalled = false;
  const float mine = slice_max(s, sh.bars, &stalled);
  // the j-th largest lane maximum of each warp that holds units (ties ranked by lane)
  const int warps = min(kSliceWarps, (s.n + 31) / 32);
  float bound = kPosInf;
  if (warp < warps) {
    const int j = (k + warps - 1) / warps;
    int above = 0;
#pragma unroll
    for (int o = 0; o < 32; ++o) {
      const float v = __shfl_sync(0xFFFFFFFFu, mine, o);
      above += v > mine || (v == mine && o < lane);
    }
    bound = j > 32 ? kNegInf : warp_max(above == j - 1 ? mine : kNegInf);
  }
  const float c = kLog2e / a.temperature;
  const float m = block_max(mine, sh.red);
  __syncthreads();
  if (lane == 0) sh.red[warp] = bound;
  __syncthreads();
  bound = s.n > 0 ? warp_min(sh.red[tid & (kSliceWarps - 1)]) : kNegInf;
  ExpAgainst against;
  against.init(m, c);
  const float sum = block_sum(slice_sum(s, against), sh.red);
  if (C > 1) {
    cluster_wait();  // every CTA of the cluster runs
    if (tid < C) {
      peer_store2(peer_addr(smem_addr(&sh.ms[rank]), tid), m, sum);
      peer_store(peer_addr(smem_addr(&sh.bound[rank]), tid), bound);
    }
    cluster_arrive();
    cluster_wait();
  } else {
    if (tid == 0) {
      sh.ms[0] = make_float2(m, sum);
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
  // entries at or above the bound
  for (int u = tid; u < s.n; u += kSliceThreads) {
    const uint4 w = s.buf[u];
    if (Unit<TIn>::max(w) < bound) continue;
#pragma unroll
    for (int q = 0; q < kN / 2; ++q) {
      float v[2];
      unpack2(Unit<TIn>::pair(w, q), v[0], v[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (v[e] >= bound && v[e] > kNegInf) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < kLocal) sh.keys[at] = argmax_key(v[e], s.index(u * kN + 2 * q + e));
        }
    }
  }
  __syncthreads();
  if (sh.count > kLocal) select_ties(s, k, bound, sh);
  const int n_local = sh.count;
  // to the first CTA, over its slice
  unsigned long long* all = reinterpret_cast<unsigned long long*>(slice_smem);
  int n = n_local;
  if (C > 1) {
    if (tid == 0) sh.base = (int)peer_add(peer_addr(smem_addr(&sh.total), 0), (uint32_t)n_local);
    cluster_arrive();
    cluster_wait();  // every CTA is done with its slice
    const int base = sh.base;
    for (int q = tid; q < n_local; q += kSliceThreads) peer_store(peer_addr(smem_addr(&all[base + q]), 0), sh.keys[q]);
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    n = (int)sh.total;
  } else {
    for (int q = tid; q < n; q += kSliceThreads) all[q] = sh.keys[q];
    __syncthreads();
  }
  const float S = warp_reduce(ms.x > kNegInf ? ms.y * rel_exp(ms.x, M, c) : 0.f, OpAddF());
  const float lnS = logf(S);
  auto put = [&](int place, unsigned long long key) {
    const float v = f32_from_key((uint32_t)(key >> 32));
    ids[place] = argmax_index(key);
    lp[place] = (v == M ? 0.f : (v - M) / a.temperature) - lnS;
  };
  if (n <= kRankMost) {
    for (int q = tid; q < n; q += kSliceThreads) {
      const unsigned long long key = all[q];
      int place = 0;
      for (int o = 0; o < n; ++o) place += all[o] > key;
      if (place < k) put(place, key);
    }
  } else {
    int size = 1;
    while (size < n) size <<= 1;
    for (int q = n + tid; q < size; q += kSliceThreads) all[q] = 0ull;  // below every key
    sort_keys(all, size);
    for (int q = tid; q < min(n, k); q += kSliceThreads) put(q, all[q]);
  }
  for (int q = n + tid; q < k; q += kSliceThreads) {
    ids[q] = -1;
    lp[q] = kNegInf;
  }
  if (tid == 0) {
    if (a.out_lse) a.out_lse[i] = M / a.temperature + lnS;
  }
  if (stalled && a.error_word) atomicOr(a.error_word, LS_ROW_ERR_STALLED);
}

template <typename TIn>
static ls_status launch_top(const TopArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const SlicePlan plan = plan_slices(n, a.vocab, dtype);
  // the first CTA takes every CTA's keys, padded to a power of two
  const size_t keys = (size_t)plan.ctas * kLocal * sizeof(unsigned long long);
  return launch_slices(top_kernel<TIn>, a, plan, plan.smem > keys ? plan.smem : keys, n, st, done);
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
