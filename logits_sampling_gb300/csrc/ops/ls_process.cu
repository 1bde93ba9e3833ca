// ls_process.cu -- penalties, biases and masks of allowed tokens on logits
// rows (ls_process_logits).
//
// A row is cut into tiles of kTile entries, one CTA each.  The CTA keeps one
// word per entry of its tile in shared memory: bit 0 says that the id occurs in
// the request's history, the bits above count its occurrences past the
// prompt.  It reads the whole history once (each tile of the row does), marks
// the ids of its own tile, adds the row's biases and then passes over its
// entries.
#include "ls_row_ops.cuh"

namespace lsg {
namespace ops {

constexpr int kProcThreads = 256;
constexpr int kTile = 4096;

struct ProcessArgs {
  const void* logits;
  int64_t logits_rows, vocab, row_stride;
  const int32_t* gather;
  const int32_t* t2r;
  ls_logits_params p;
  bool has_params;
  const int32_t* row_lens;
  const uint32_t* mask;
  int64_t mask_rows, mask_stride;
  const int32_t* mask_index;
  void* out;
  int64_t out_stride;
  int32_t* error_word;
};

template <typename TIn>
__global__ void __launch_bounds__(kProcThreads) process_kernel(const ProcessArgs a, int tiles) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  __shared__ uint32_t marks[kTile];
  __shared__ float bias[kTile];
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)tiles;
  const int64_t j0 = (int64_t)(blockIdx.x % (unsigned)tiles) * kTile;
  const int len = (int)min((int64_t)kTile, a.vocab - j0);
  Raw* out = static_cast<Raw*>(a.out) + i * a.out_stride + j0;

  int32_t bad = 0;
  const int64_t src = a.gather ? a.gather[i] : i;
  if (src < 0 || src >= a.logits_rows) bad |= LS_ROW_ERR_BAD_GATHER;
  int64_t r = 0;
  if (a.has_params) {
    r = a.t2r ? a.t2r[i] : i;
    if (r < 0 || r >= a.p.num_requests) bad |= LS_ROW_ERR_BAD_REQUEST;
  }
  int64_t mrow = -1;
  if (a.mask) {
    mrow = a.mask_index ? a.mask_index[i] : i;
    if (mrow < -1 || mrow >= a.mask_rows) bad |= LS_ROW_ERR_BAD_MASK;
  }
  if (bad) {
    for (int e = tid; e < len; e += kProcThreads) out[e] = E::put(quiet_nan());
    if (tid == 0 && j0 == 0 && a.error_word) atomicOr(a.error_word, bad);
    return;
  }
  const Raw* in = static_cast<const Raw*>(a.logits) + src * a.row_stride + j0;

  for (int e = tid; e < kTile; e += kProcThreads) {
    marks[e] = 0u;
    bias[e] = 0.f;
  }
  __syncthreads();
  float rho = 1.f, pres = 0.f, freq = 0.f;
  if (a.has_params && a.p.tokens) {
    if (a.p.repetition) rho = a.p.repetition[r];
    if (a.p.presence) pres = a.p.presence[r];
    if (a.p.frequency) freq = a.p.frequency[r];
    const int32_t L = min(max(a.row_lens ? a.row_lens[i] : a.p.seq_lens[r], 0), a.p.token_capacity);
    const int32_t prompt = a.p.prompt_lens ? a.p.prompt_lens[r] : 0;
    const int32_t* t = a.p.tokens + r * a.p.token_stride;
    for (int32_t q = tid; q < L; q += kProcThreads) {
      const int64_t e = (int64_t)t[q] - j0;
      if (e >= 0 && e < len) {
        if (q < prompt)
          atomicOr(&marks[e], 1u);
        else
          atomicAdd(&marks[e], 2u);
      }
    }
  }
  bool biased = false;
  if (a.has_params && a.p.bias_offsets) {
    const int32_t lo = max(a.p.bias_offsets[r], 0), hi = min(a.p.bias_offsets[r + 1], a.p.bias_count);
    biased = lo < hi;
    for (int32_t q = lo + tid; q < hi; q += kProcThreads) {
      const int64_t e = (int64_t)a.p.bias_ids[q] - j0;
      if (e >= 0 && e < len) bias[e] = a.p.bias_values[q];
    }
  }
  __syncthreads();
  const uint32_t* mask = mrow >= 0 ? a.mask + mrow * a.mask_stride : nullptr;
  for (int e = tid; e < len; e += kProcThreads) {
    Raw raw = in[e];
    const uint32_t m = marks[e];
    const float b = biased ? bias[e] : 0.f;
    if (m != 0u || b != 0.f) {
      const float x = E::get(raw);
      const float c = (float)(m >> 1);
      float y = m != 0u ? (x > 0.f ? x / rho : x * rho) : x;
      y = __fsub_rn(y, __fmul_rn(freq, c));
      if (c > 0.f) y -= pres;
      y += b;
      raw = E::put(guard(y));
    }
    if (mask && !((mask[(j0 + e) >> 5] >> ((j0 + e) & 31)) & 1u)) raw = E::neg_inf();
    out[e] = raw;
  }
}

}  // namespace ops
}  // namespace lsg

using namespace lsg;
using namespace lsg::ops;

extern "C" ls_status ls_process_logits(const void* logits, ls_dtype dtype, int64_t logits_rows, int64_t vocab,
                                       int64_t row_stride, int32_t n, const int32_t* gather_indices,
                                       const int32_t* token_to_request_index, const ls_logits_params* params,
                                       const int32_t* row_lens, const int32_t* allowed_mask, int64_t mask_rows,
                                       int64_t mask_stride, const int32_t* mask_index, void* out, int64_t out_stride,
                                       int32_t* error_word, void* stream) {
  if (n < 0) return LS_ERR_INVALID_ARG;
  if (n == 0) return LS_OK;
  if (!matrix_ok(logits, dtype, vocab, row_stride) || !matrix_ok(out, dtype, vocab, out_stride) || logits_rows < 1)
    return LS_ERR_INVALID_ARG;
  if (!gather_indices && (int64_t)n > logits_rows) return LS_ERR_INVALID_ARG;
  if (!overlap_ok(logits, logits_rows, row_stride, out, n, out_stride, vocab, dtype, !gather_indices))
    return LS_ERR_INVALID_ARG;
  ProcessArgs a = {};
  if (params) {
    a.p = *params;
    a.has_params = true;
    if (a.p.num_requests < 1) return LS_ERR_INVALID_ARG;
    if (!token_to_request_index && n > a.p.num_requests) return LS_ERR_INVALID_ARG;
    if (a.p.tokens && (a.p.token_capacity < 0 || a.p.token_stride < a.p.token_capacity || !(a.p.seq_lens || row_lens)))
      return LS_ERR_INVALID_ARG;
    if (a.p.bias_offsets && (a.p.bias_count < 0 || (a.p.bias_count > 0 && (!a.p.bias_ids || !a.p.bias_values))))
      return LS_ERR_INVALID_ARG;
  }
  if (allowed_mask &&
      (mask_rows < 1 || mask_stride < (vocab + 31) / 32 || (!mask_index && (int64_t)n > mask_rows)))
    return LS_ERR_INVALID_ARG;
  const int64_t tiles = (vocab + kTile - 1) / kTile;
  if (tiles * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  a.logits = logits;
  a.logits_rows = logits_rows;
  a.vocab = vocab;
  a.row_stride = row_stride;
  a.gather = gather_indices;
  a.t2r = token_to_request_index;
  a.row_lens = row_lens;
  a.mask = reinterpret_cast<const uint32_t*>(allowed_mask);
  a.mask_rows = mask_rows;
  a.mask_stride = mask_stride;
  a.mask_index = mask_index;
  a.out = out;
  a.out_stride = out_stride;
  a.error_word = error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(tiles * n)), block(kProcThreads);
  if (dtype == LS_DTYPE_BF16)
    process_kernel<bf16_tag><<<grid, block, 0, st>>>(a, (int)tiles);
  else
    process_kernel<float><<<grid, block, 0, st>>>(a, (int)tiles);
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}
