// ls_top.cu -- the k best entries of each logits row, their log-probs and the
// row's log-sum-exp (ls_top_log_probs).
//
// One CTA per row.  After the maximum and the sum of exponentials, the k-th
// largest value is found bit by bit from the top of its order-preserving key
// (a count over the row per bit), then, where more entries tie with it than
// are left to take, the highest index taken, the same way.  The at most k
// entries are collected and each is placed by the number of entries before it.
#include "ls_row_ops.cuh"

namespace lsg {
namespace ops {

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

struct OpMaxF {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpAddI {
  __device__ __forceinline__ int operator()(int a, int b) const { return a + b; }
};

template <typename TIn>
__global__ void __launch_bounds__(kThreads) top_kernel(const TopArgs a) {
  using E = Elem<TIn>;
  __shared__ float red_f[kWarps];
  __shared__ int red_i[kWarps];
  __shared__ unsigned long long list[LS_MAX_TOP];
  __shared__ int count;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x, V = a.vocab;
  const int64_t src = a.gather ? a.gather[i] : i;
  int32_t* ids = a.out_ids + i * a.k;
  float* lp = a.out_lp + i * a.k;
  auto fail = [&](int32_t bit) {
    for (int q = tid; q < a.k; q += kThreads) {
      ids[q] = -1;
      lp[q] = quiet_nan();
    }
    if (tid == 0) {
      if (a.out_lse) a.out_lse[i] = quiet_nan();
      if (a.error_word) atomicOr(a.error_word, bit);
    }
  };
  if (src < 0 || src >= a.logits_rows) {
    fail(LS_ROW_ERR_BAD_GATHER);
    return;
  }
  const typename E::Raw* row = static_cast<const typename E::Raw*>(a.logits) + src * a.row_stride;
  float m = kNegInf;
  int live = 0;  // entries above -inf
  for (int64_t j = tid; j < V; j += kThreads) {
    const float v = guard(E::get(row[j]));
    m = fmaxf(m, v);
    live += v > kNegInf;
  }
  const float M = block_reduce(m, OpMaxF(), red_f);
  live = block_reduce(live, OpAddI(), red_i);
  if (M == kNegInf) {
    fail(LS_ROW_ERR_NO_FINITE);
    return;
  }
  const float c = kLog2e / a.temperature;
  float s = 0.f;
  for (int64_t j = tid; j < V; j += kThreads) {
    const float v = guard(E::get(row[j]));
    s += v == M ? 1.f : ex2((v - M) * c);
  }
  const float S = block_reduce(s, OpAddF(), red_f);
  const float lnS = logf(S);
  const int K = min(a.k, live);
  // the largest key with at least K entries at or above it
  uint32_t cut = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t t = cut | (1u << bit);
    int n = 0;
    for (int64_t j = tid; j < V; j += kThreads) n += f32_key(guard(E::get(row[j]))) >= t;
    if (block_reduce(n, OpAddI(), red_i) >= K) cut = t;
  }
  int above = 0;
  for (int64_t j = tid; j < V; j += kThreads) above += f32_key(guard(E::get(row[j]))) > cut;
  const int ties = K - block_reduce(above, OpAddI(), red_i);
  // the lowest index with `ties` entries equal to the cut at or below it
  int64_t lo = 0, hi = V - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    int n = 0;
    for (int64_t j = tid; j <= mid; j += kThreads) n += f32_key(guard(E::get(row[j]))) == cut;
    if (block_reduce(n, OpAddI(), red_i) >= ties)
      hi = mid;
    else
      lo = mid + 1;
  }
  if (tid == 0) count = 0;
  __syncthreads();
  for (int64_t j = tid; j < V; j += kThreads) {
    const float v = guard(E::get(row[j]));
    const uint32_t key = f32_key(v);
    if (key > cut || (key == cut && j <= hi)) list[atomicAdd(&count, 1)] = argmax_key(v, j);
  }
  __syncthreads();
  for (int q = tid; q < a.k; q += kThreads) {
    if (q < K) {
      const unsigned long long key = list[q];
      int rank = 0;
      for (int o = 0; o < K; ++o) rank += list[o] > key;
      const float v = f32_from_key((uint32_t)(key >> 32));
      ids[rank] = argmax_index(key);
      lp[rank] = (v == M ? 0.f : (v - M) / a.temperature) - lnS;
    } else {
      ids[q] = -1;
      lp[q] = kNegInf;
    }
  }
  if (tid == 0 && a.out_lse) a.out_lse[i] = M / a.temperature + lnS;
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
  if (dtype == LS_DTYPE_BF16)
    top_kernel<bf16_tag><<<dim3((unsigned)n), dim3(kThreads), 0, st>>>(a);
  else
    top_kernel<float><<<dim3((unsigned)n), dim3(kThreads), 0, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}

extern "C" int64_t ls_row_ops_max_vocab(ls_dtype dtype) {
  if (device_attr<cudaDevAttrMaxSharedMemoryPerBlockOptin>() <= 0) return 0;
  return max_row(dtype);
}
