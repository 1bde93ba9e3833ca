// ls_process.cu -- penalties, biases and masks of allowed tokens on logits
// rows (ls_process_logits).
//
// A row is cut into tiles, one CTA each: kUnits 32-byte units per thread,
// loaded to registers at the start and written at the end (four, or one where
// that leaves SMs without a CTA).  In between, the few
// entries that the history or a bias touches are worked out on the side:
//  1. Each unit takes -inf where the mask says so and is written: entries that
//     nothing touches keep their bits.
//  2. Meanwhile the request's history arrives (every tile of the row reads all
//     of it: at the lengths that occur it is small against the row).  The ids of
//     the CTA's own tile go to a table with one slot per entry: bit 0 says that
//     the id occurs, the bits above count its occurrences past the prompt.  An
//     id's first occurrence lists the entry.
//  3. One thread per listed entry, and one per bias, reads the logit and the
//     slot, works out the new value in fp32 and writes it over the copy, unless
//     the mask forbids the id.  (In place the logit is still there: step 1
//     wrote the same bits, or -inf where the mask forbids it.)
// A slot of 16 bits holds the counts of a history of fewer than 2^15 ids.
#include "ls_stream.cuh"

namespace lsg {
namespace ops {

constexpr int kProcThreads = 256;
constexpr int kHistoryBatch = 8;  // history ids of a thread in flight
constexpr int kSettleBatch = 4;   // touched entries of a thread in flight
constexpr int kListed = 4096;     // touched entries listed; past it step 3 walks the table

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

// Marks a table slot and returns whether it was empty.  An atomic update of
// 16-bit slots works on the 32-bit word that holds two (no carry crosses: see
// the widths above).
template <typename Slot>
__device__ __forceinline__ bool mark(Slot* table, int e, bool prompt) {
  uint32_t* word = reinterpret_cast<uint32_t*>(table) + (sizeof(Slot) == 2 ? e >> 1 : e);
  const int shift = sizeof(Slot) == 2 ? (e & 1) * 16 : 0;
  const uint32_t old = prompt ? atomicOr(word, 1u << shift) : atomicAdd(word, 2u << shift);
  return (Slot)(old >> shift) == 0;
}

// Bits [j, j + N) of a mask row, 1 outside [0, vocab) (j may lie before the row).
template <int N>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* mask, int64_t j, int64_t vocab, bool full) {
  const int64_t w = j >> 5;  // arithmetic: -1 for a negative j
  const int shift = (int)(j & 31);
  uint32_t lo, hi = 0xFFFFFFFFu;
  if (full) {  // all N entries lie in the row: so do their words
    lo = __ldg(mask + w);
    if (shift > 32 - N) hi = __ldg(mask + w + 1);
  } else {
    const int64_t last = (vocab - 1) >> 5;
    lo = w >= 0 && w <= last ? __ldg(mask + w) : 0xFFFFFFFFu;
    if (shift > 32 - N && w + 1 <= last) hi = __ldg(mask + w + 1);
  }
  return __funnelshift_r(lo, hi, shift) & ((1u << N) - 1u);
}

template <typename TIn, typename Slot, int kUnits>
__global__ void __launch_bounds__(kProcThreads, 4) process_kernel(const ProcessArgs a, int tiles) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  constexpr int kN = Unit<TIn>::kN;
  constexpr int kTileUnits = kProcThreads * kUnits, kEntries = kTileUnits * kN;
  extern __shared__ uint4 dyn_smem[];
  Slot* table = reinterpret_cast<Slot*>(dyn_smem);
  uint32_t* biased = reinterpret_cast<uint32_t*>(table + kEntries);  // a bit per entry: those of a bias
  uint32_t* settled = biased + kEntries / 32;                        // those whose bias is applied
  __shared__ uint16_t list[kListed];
  __shared__ int listed;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)tiles;
  const int tile = (int)(blockIdx.x % (unsigned)tiles);
  Raw* out = static_cast<Raw*>(a.out) + i * a.out_stride;

  wait_for_previous();
  let_next_start();
  int32_t bad = 0;
  const int64_t src = a.gather ? a.gather[i] : i;
  const int64_t r = a.has_params ? (a.t2r ? a.t2r[i] : i) : 0;
  const int64_t mrow = a.mask ? (a.mask_index ? a.mask_index[i] : i) : -1;
  if (src < 0 || src >= a.logits_rows) bad |= LS_ROW_ERR_BAD_GATHER;
  if (a.has_params && (r < 0 || r >= a.p.num_requests)) bad |= LS_ROW_ERR_BAD_REQUEST;
  if (mrow < -1 || mrow >= a.mask_rows) bad |= a.mask ? LS_ROW_ERR_BAD_MASK : 0;
  Run<TIn, kProcThreads> run;
  run.init(a.logits, bad & LS_ROW_ERR_BAD_GATHER ? 0 : src, a.row_stride, a.vocab, kTileUnits, tile);
  const bool same = run.aligned_with(out);
  uint32_t v[kUnits][8];
  if (bad) {
    const Raw nan = E::put(quiet_nan());
    Raw e[kN];
#pragma unroll
    for (int q = 0; q < kN; ++q) e[q] = nan;
    memcpy(v[0], e, 32);
    for (int u = tid; u < run.n; u += kProcThreads) run.store(out, same, u, v[0]);
    if (tid == 0 && tile == 0 && a.error_word) atomicOr(a.error_word, bad);
    return;
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q)
    if (tid + q * kProcThreads < run.n) run.template load<LOAD_PLAIN>(tid + q * kProcThreads, v[q]);

  // The request's penalties; neutral ones leave the history unread.
  float rho = 1.f, pres = 0.f, freq = 0.f;
  int32_t L = 0, prompt = 0;
  const int32_t* history = nullptr;
  int32_t b_lo = 0, b_hi = 0;
  if (a.has_params) {
    if (a.p.tokens) {
      if (a.p.repetition) rho = a.p.repetition[r];
      if (a.p.presence) pres = a.p.presence[r];
      if (a.p.frequency) freq = a.p.frequency[r];
      L = a.row_lens ? a.row_lens[i] : a.p.seq_lens[r];
      prompt = a.p.prompt_lens ? a.p.prompt_lens[r] : 0;
      L = min(max(L, 0), a.p.token_capacity);
      if (rho == 1.f && pres == 0.f && freq == 0.f) L = 0;
      history = a.p.tokens + r * a.p.token_stride;
    }
    if (a.p.bias_offsets) {
      b_lo = max(a.p.bias_offsets[r], 0);
      b_hi = min(a.p.bias_offsets[r + 1], a.p.bias_count);
    }
  }
  const bool any = L > 0 || b_lo < b_hi;  // the same in every thread
  const uint32_t* mask = mrow >= 0 ? a.mask + mrow * a.mask_stride : nullptr;
  // the first ids of the history, and a bias, on their way while the units are written
  int32_t held[kHistoryBatch];
  auto fetch = [&](int32_t at) {
#pragma unroll
    for (int q = 0; q < kHistoryBatch; ++q) {
      const int32_t t = at + q * kProcThreads;
      held[q] = t < L ? history[t] : -1;
    }
  };
  auto place = [&](int32_t id) { return id >= 0 && id < run.V ? run.place(id) : -1; };
  int bias_e = -1;
  float bias_v = 0.f;
  if (any) {
    fetch(tid);
    if (b_lo + tid < b_hi) {
      bias_e = place(a.p.bias_ids[b_lo + tid]);
      bias_v = a.p.bias_values[b_lo + tid];
    }
    constexpr int kWords = (kEntries * (int)sizeof(Slot) + 2 * (kEntries / 8)) / 16;  // table and bits
    for (int q = tid; q < kWords; q += kProcThreads) dyn_smem[q] = make_uint4(0u, 0u, 0u, 0u);
    if (tid == 0) listed = 0;
  }
#pragma unroll
  for (int q = 0; q < kUnits; ++q) {
    const int u = tid + q * kProcThreads;
    if (u >= run.n) break;
    if (mask) {
      const uint32_t all = (1u << kN) - 1u;
      const uint32_t forbidden = ~mask_bits<kN>(mask, run.index(u), run.V, run.full(u)) & all;
      if (forbidden) Unit<TIn>::drop(v[q], forbidden);
    }
    run.store(out, same, u, v[q]);
  }
  if (!any) return;
  __syncthreads();
  for (int32_t at = tid; at - tid < L; at += kHistoryBatch * kProcThreads) {
    if (at != tid) fetch(at);
#pragma unroll
    for (int q = 0; q < kHistoryBatch; ++q) {
      const int e = place(held[q]);
      const bool first = e >= 0 && mark(table, e, at + q * kProcThreads < prompt);
      const uint32_t firsts = __ballot_sync(0xFFFFFFFFu, first);
      if (firsts == 0u) continue;
      int n = 0;
      if ((tid & 31) == 0) n = atomicAdd(&listed, __popc(firsts));
      n = __shfl_sync(0xFFFFFFFFu, n, 0) + __popc(firsts & ((1u << (tid & 31)) - 1u));
      if (first && n < kListed) list[n] = (uint16_t)e;
    }
  }
  if (bias_e >= 0) atomicOr(&biased[bias_e >> 5], 1u << (bias_e & 31));
  for (int32_t q = b_lo + tid + kProcThreads; q < b_hi; q += kProcThreads) {
    const int e = place(a.p.bias_ids[q]);
    if (e >= 0) atomicOr(&biased[e >> 5], 1u << (e & 31));
  }
  __syncthreads();  // also: the copies are written before their touched entries are
  auto allowed = [&](int e) {
    const int64_t j = run.j0 + e;
    return !mask || (__ldg(mask + (j >> 5)) >> (j & 31) & 1u) != 0u;
  };
  // the new value of entry e from its logit (called by one thread per entry)
  auto settle = [&](int e, float x, float b, bool has_bias) {
    const uint32_t m = table[e];
    const float n = (float)(m >> 1);
    float y = m != 0u ? (x > 0.f ? x / rho : x * rho) : x;
    y = __fsub_rn(y, __fmul_rn(freq, n));
    if (n > 0.f) y -= pres;
    if (has_bias) y += b;
    out[run.j0 + e] = E::put(guard(y));
  };
  auto logit = [&](int e) { return E::get(run.row[run.j0 + e]); };
  auto settle_bias = [&](int e, float b) {
    const uint32_t bit = 1u << (e & 31);
    if (!(atomicOr(&settled[e >> 5], bit) & bit) && allowed(e)) settle(e, logit(e), b, true);
  };
  if (bias_e >= 0) settle_bias(bias_e, bias_v);
  for (int32_t q = b_lo + tid + kProcThreads; q < b_hi; q += kProcThreads) {
    const int e = place(a.p.bias_ids[q]);
    if (e >= 0) settle_bias(e, a.p.bias_values[q]);
  }
  const int n_listed = listed;
  if (n_listed <= kListed) {
    for (int q = tid; q < n_listed; q += kSettleBatch * kProcThreads) {
      int e[kSettleBatch];
      float x[kSettleBatch];
#pragma unroll
      for (int k = 0; k < kSettleBatch; ++k) {
        e[k] = -1;
        if (q + k * kProcThreads < n_listed) e[k] = list[q + k * kProcThreads];
        if (e[k] >= 0 && (biased[e[k] >> 5] >> (e[k] & 31) & 1u)) e[k] = -1;
        if (e[k] >= 0) x[k] = logit(e[k]);
        if (e[k] >= 0 && !allowed(e[k])) e[k] = -1;
      }
#pragma unroll
      for (int k = 0; k < kSettleBatch; ++k)
        if (e[k] >= 0) settle(e[k], x[k], 0.f, false);
    }
  } else {
    for (int e = tid; e < kEntries; e += kProcThreads)
      if (table[e] != 0 && !(biased[e >> 5] >> (e & 31) & 1u) && allowed(e)) settle(e, logit(e), 0.f, false);
  }
}

template <typename TIn, typename Slot, int kUnits>
static ls_status launch(const ProcessArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  constexpr int kTileUnits = kProcThreads * kUnits, kEntries = kTileUnits * Unit<TIn>::kN;
  const int64_t tiles = (row_units(a.vocab, dtype) + kTileUnits - 1) / kTileUnits;
  if (tiles * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  const bool side = a.has_params && (a.p.tokens || a.p.bias_offsets);
  const size_t smem = side ? (size_t)kEntries * sizeof(Slot) + 2 * (kEntries / 8) : 0;
  if (!open_limits(process_kernel<TIn, Slot, kUnits>, done)) return LS_ERR_CUDA;
  return launch_kernel(process_kernel<TIn, Slot, kUnits>, dim3((unsigned)(tiles * n)), kProcThreads, 1, smem, st, a,
                       (int)tiles);
}

template <typename TIn, typename Slot>
static ls_status launch(const ProcessArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  const int64_t wide = (row_units(a.vocab, dtype) + 4 * kProcThreads - 1) / (4 * kProcThreads) * n;
  return wide < 2 * device_attr<cudaDevAttrMultiProcessorCount>() ? launch<TIn, Slot, 1>(a, dtype, n, st)
                                                                  : launch<TIn, Slot, 4>(a, dtype, n, st);
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
  const bool narrow = !a.has_params || !a.p.tokens || a.p.token_capacity < (1 << 15);
  if (dtype == LS_DTYPE_F32) return narrow ? launch<float, uint16_t>(a, dtype, n, st) : launch<float, uint32_t>(a, dtype, n, st);
  return narrow ? launch<bf16_tag, uint16_t>(a, dtype, n, st) : launch<bf16_tag, uint32_t>(a, dtype, n, st);
}
