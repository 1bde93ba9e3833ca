// ls_process.cu -- penalties, biases and masks of allowed tokens on logits
// rows (ls_process_logits).
//
// Most entries are copied bit for bit, or replaced by -inf where the mask
// forbids them; the few that the history or a bias touches are worked out on
// the side, in fp32 with one rounding to the type of the logits:
//     y = (x > 0 ? x / rho : x rho) - freq n - pres [n > 0] + bias
// (the quotient for ids that occur at all, n the occurrences past the prompt).
// Two forms, chosen in launch():
//
// One kernel (process_kernel).  A row is cut into tiles, one CTA each: kUnits
// 32-byte units per thread (four, or one where that leaves SMs without a CTA),
// loaded to registers, masked and written.  Meanwhile the request's history
// arrives: every tile of the row reads all of it and marks the ids of its own
// entries in a table in shared memory.  Then one thread per touched entry, and
// one per bias, works out the new value and writes it over the copy.
//
// A pair for batches that fill the GPU.  copy_kernel does the masked copy at
// the speed of memory; settle_kernel, one CTA per row, builds a hash table of
// the row's ids while the copies are still being written, and then writes the
// touched entries' new values over them.
#include "ls_stream.cuh"

namespace lsg {
namespace ops {

constexpr int kProcThreads = 256;
constexpr int kHistoryBatch = 4;  // history ids of a thread in flight (8: 2.9 -> 3.3 us for one row, 358 -> 370 for 1 GB)
constexpr int kSettleBatch = 4;   // touched entries of a thread in flight
constexpr int kListed = 4096;     // touched entries listed; past it step 3 walks the table

constexpr int32_t kMostListed = 1 << 30;  // ids of a history, or biases: counts and strides stay within 32 bits

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
  bool keep;  // the output fits in L2 until its touched entries are settled
};

// Marks a table slot and returns whether it was empty.  An atomic update of
// 16-bit slots works on the 32-bit word that holds two (no carry crosses: they
// are used where a history has fewer than 2^15 ids, so 2 n + 1 stays below 2^16).
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

// The row that an output row reads, its request and its mask row.
struct RowSource {
  int64_t src, request, mask_row;
  int32_t bad;  // LS_ROW_ERR_* bits
  __device__ __forceinline__ RowSource(const ProcessArgs& a, int64_t i) {
    src = a.gather ? a.gather[i] : i;
    request = a.has_params ? (a.t2r ? a.t2r[i] : i) : 0;
    mask_row = a.mask ? (a.mask_index ? a.mask_index[i] : i) : -1;
    bad = 0;
    if (src < 0 || src >= a.logits_rows) bad |= LS_ROW_ERR_BAD_GATHER;
    if (a.has_params && (request < 0 || request >= a.p.num_requests)) bad |= LS_ROW_ERR_BAD_REQUEST;
    if (a.mask && (mask_row < -1 || mask_row >= a.mask_rows)) bad |= LS_ROW_ERR_BAD_MASK;
  }
};

// A request's penalties and biases for a row.  Neutral penalties leave the
// history unread (L = 0).
struct RowPenalties {
  float rho = 1.f, pres = 0.f, freq = 0.f;
  int32_t L = 0, prompt = 0;
  const int32_t* history = nullptr;
  int32_t b_lo = 0, b_hi = 0;
  __device__ __forceinline__ RowPenalties(const ProcessArgs& a, int64_t i, int64_t r) {
    if (!a.has_params) return;
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
      b_lo = min(max(a.p.bias_offsets[r], 0), a.p.bias_count);
      b_hi = min(a.p.bias_offsets[r + 1], a.p.bias_count);
    }
  }
  __device__ __forceinline__ bool any() const { return L > 0 || b_lo < b_hi; }
  // The new value of a logit: `marks` bit 0: the id occurs; above: occurrences past the prompt.
  __device__ __forceinline__ float value(float x, uint32_t marks, float b, bool has_bias) const {
    const float n = (float)(marks >> 1);
    float y = marks != 0u ? (x > 0.f ? x / rho : x * rho) : x;
    y = __fsub_rn(y, __fmul_rn(freq, n));
    if (n > 0.f) y -= pres;
    if (has_bias) y += b;
    return guard(y);
  }
};

// Fills this CTA's run of a bad output row with NaN and notes its error.
template <typename TIn, int T>
__device__ __forceinline__ void fail_run(const ProcessArgs& a, const Run<TIn, T>& run, typename Elem<TIn>::Raw* out,
                                         bool same, bool first, int32_t bad) {
  const uint32_t nan = Elem<TIn>::kBytes == 2 ? 0x7FC07FC0u : 0x7FC00000u;
  const uint32_t v[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
  for (int u = threadIdx.x; u < run.n; u += T) run.store(out, same, u, v);
  if (threadIdx.x == 0 && first && a.error_word) atomicOr(a.error_word, bad);
}

// One tile:
//  1. Each unit takes -inf where the mask says so and is written: entries that
//     nothing touches keep their bits.
//  2. The ids of the CTA's own tile go to a table with one slot per entry: bit 0
//     says that the id occurs, the bits above count its occurrences past the
//     prompt (16-bit slots for histories of fewer than 2^15 ids).  An id's first
//     occurrence lists the entry.
//  3. One thread per listed entry, and one per bias, reads the logit and the
//     slot and writes the new value over the copy, unless the mask forbids the
//     id.  (In place the logit is still there: step 1 wrote the same bits, or -inf
//     where the mask forbids it.)
// Bound by latency: a tile's life is a chain of reads (row, request, history,
// logits again) beside 2 x 32 KB of copying, four tiles to an SM, and every tile
// reads the row's whole history in batches of 1024 ids, one after another with
// none in flight between them.  1 x 32000 bf16 2.9 us with 256 ids; with biases
// and masks 63 x 32003 9.0 us with 2048 ids in every row; 256 x 128256 32 / 40 / 78
// us with 512 / 2048 / 8192 ids in every row, and 31 / 33 / 44 us (3.1 TB/s) with
// lengths spread over their logarithm from 16 up to those (130, 366 and 1170 ids a
// row: the longest rows decide).
// Measured against it on lengths up to 8192: tiles of 512 threads 42 us (but 36
// against 34 on lengths up to 2048); the tile's logits in shared memory and settled
// there 49 us (72 KB of it per CTA leaves L1 too small for the loads in flight); a
// hash table in place of a slot per entry 52 us.
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
  const RowSource from(a, i);
  Run<TIn, kProcThreads> run;
  run.init(a.logits, from.bad & LS_ROW_ERR_BAD_GATHER ? 0 : from.src, a.row_stride, a.vocab, kTileUnits, tile);
  const bool same = run.aligned_with(out);
  if (from.bad) {
    fail_run(a, run, out, same, tile == 0, from.bad);
    return;
  }
  uint32_t v[kUnits][8];
#pragma unroll
  for (int q = 0; q < kUnits; ++q)
    if (tid + q * kProcThreads < run.n) run.template load<LOAD_NORMAL>(tid + q * kProcThreads, v[q]);

  const RowPenalties pen(a, i, from.request);
  const int32_t L = pen.L, prompt = pen.prompt, b_lo = pen.b_lo, b_hi = pen.b_hi;
  const int32_t* history = pen.history;
  const bool any = pen.any();  // the same in every thread
  const uint32_t* mask = from.mask_row >= 0 ? a.mask + from.mask_row * a.mask_stride : nullptr;
  // the first ids of the history, and a bias, on their way while the units are written
  int32_t held[kHistoryBatch];
  auto fetch = [&](int32_t at) {
#pragma unroll
    for (int q = 0; q < kHistoryBatch; ++q) {
      const int32_t t = at + q * kProcThreads;
      held[q] = t < L ? history[t] : -1;
    }
  };
  // the tile's entry of an id, -1 for an id of another tile or of none
  const uint32_t least = (uint32_t)max(run.j0, (int64_t)0);
  const uint32_t span = run.n > 0 ? (uint32_t)(min(run.index(run.n), run.V) - (int64_t)least) : 0u;
  auto place = [&](int32_t id) {
    const uint32_t e = (uint32_t)id - least;
    return e < span ? (int)e : -1;
  };
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
    const uint32_t j = least + e;
    return !mask || (__ldg(mask + (j >> 5)) >> (j & 31) & 1u) != 0u;
  };
  // the new value of entry e from its logit (called by one thread per entry)
  auto settle = [&](int e, float x, float b, bool has_bias) {
    out[least + e] = E::put(pen.value(x, table[e], b, has_bias));
  };
  auto logit = [&](int e) { return E::get(run.row[least + e]); };
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

// ---------------------------------------------------------------------------
// The pair of kernels for batches that fill the GPU
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 2048;  // units of a CTA's run

// The masked copy.  The run's lines that the mask leaves something of are called
// into L2 first, one per thread: they keep DRAM busy without registers to hold
// them, and a unit that the mask forbids entirely is not read.  Bound by DRAM:
// with the kernel below 302 us on 1024 x 262144 fp32 under masks (7.2 TB/s of
// logits, mask and output, some of which the mask spares), 346 us without.
template <typename TIn>
__global__ void __launch_bounds__(kCopyThreads, 4) copy_kernel(const ProcessArgs a, int runs, int upc) {
  using Raw = typename Elem<TIn>::Raw;
  using R = Run<TIn, kCopyThreads>;
  constexpr int kN = Unit<TIn>::kN;
  constexpr uint32_t kAll = (1u << kN) - 1u;
  const int tid = threadIdx.x;
  const int64_t i = blockIdx.x / (unsigned)runs;
  const int rank = (int)(blockIdx.x % (unsigned)runs);
  Raw* out = static_cast<Raw*>(a.out) + i * a.out_stride;
  wait_for_previous();
  let_next_start();
  const RowSource from(a, i);
  R run;
  run.init(a.logits, from.bad & LS_ROW_ERR_BAD_GATHER ? 0 : from.src, a.row_stride, a.vocab, upc, rank);
  const bool same = run.aligned_with(out);
  if (from.bad) {
    fail_run(a, run, out, same, rank == 0, from.bad);
    return;
  }
  const uint32_t* mask = from.mask_row >= 0 ? a.mask + from.mask_row * a.mask_stride : nullptr;
  for (int u = tid * 4; u < run.n; u += 4 * kCopyThreads) {  // four units: a line
    uint32_t kept = 1u;
    if (mask) {
      kept = 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (u + k < run.n) kept |= mask_bits<kN>(mask, run.index(u + k), run.V, run.full(u + k));
    }
    if (kept && run.full(u)) asm volatile("prefetch.global.L2 [%0];" ::"l"(run.base + (int64_t)u * 32));
  }
  // Bits of the entries that a unit may keep, a stage ahead of its logits.
  typedef uint32_t Bits[kStage];
  auto keep_bits = [&](int u, Bits& b) {
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const int uk = u + k * kCopyThreads;
      b[k] = mask && uk < run.n ? mask_bits<kN>(mask, run.index(uk), run.V, run.full(uk)) : kAll;
    }
  };
  auto load = [&](int u, const Bits& b, typename R::Stage& v) {
#pragma unroll
    for (int k = 0; k < kStage; ++k)
      if (u + k * kCopyThreads < run.n && b[k] != 0u) run.template load<LOAD_PLAIN>(u + k * kCopyThreads, v[k]);
  };
  typename R::Stage cur = {}, next = {};
  Bits b0, b1, b2;
  keep_bits(tid, b0);
  keep_bits(tid + R::kStep, b1);
  load(tid, b0, cur);
#pragma unroll 1
  for (int u = tid; u < run.n; u += R::kStep) {
    keep_bits(u + 2 * R::kStep, b2);
    load(u + R::kStep, b1, next);
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      if (u + k * kCopyThreads >= run.n) break;
      if (b0[k] != kAll) Unit<TIn>::drop(cur[k], ~b0[k] & kAll);
      run.store(out, same, u + k * kCopyThreads, cur[k], a.keep);
    }
    R::move(next, cur);
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      b0[k] = b1[k];
      b1[k] = b2[k];
    }
  }
}

// The touched entries of a row, one CTA per row.  While the copies are being
// written it builds a hash table of the history's ids and the biases' in shared
// memory; then it reads the copies of those that the mask allows, which are the
// logits themselves, and writes the new values over them.  Bound by latency, two
// CTAs to an SM: a chain of dependent reads (row, request, length, ids) and then
// barriers and scattered accesses to the table and the copies.  Alone it takes 24
// us on 300 rows of 395 ids on average (16 to 2048) and 34 us with 2048 in each.
constexpr int kSettleThreads = 512;
constexpr int kSettleSlots = 11776;               // two CTAs to an SM
constexpr int kSettleIds = kSettleSlots / 4 * 3;  // ids that it takes, repeated ones and biases counted
constexpr int kSettleHistory = 8;                 // history ids of a thread in flight

struct SettleShared {
  uint32_t id[kSettleSlots];     // id + 1, 0: free
  uint32_t marks[kSettleSlots];  // as RowPenalties::value; bit 31: a bias settles it
  uint16_t list[kSettleIds];     // the slots in use
  int listed;
};

__device__ __forceinline__ int home_of(uint32_t id) { return (int)__umulhi(id * 0x9E3779B1u, (uint32_t)kSettleSlots); }
__device__ __forceinline__ int slot_after(int at) { return at + 1 == kSettleSlots ? 0 : at + 1; }

// The slot of an id, taken if it has none, from slot `at` on.
__device__ __forceinline__ int slot_of(SettleShared& sh, uint32_t id, int at) {
  for (int t = 0; t < kSettleSlots; ++t) {
    const uint32_t met = atomicCAS(&sh.id[at], 0u, id + 1u);
    if (met == 0u || met == id + 1u) break;
    at = slot_after(at);
  }
  return at;
}

template <typename TIn>
__global__ void __launch_bounds__(kSettleThreads, 2) settle_kernel(const ProcessArgs a) {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  extern __shared__ uint4 dyn_smem[];
  SettleShared& sh = *reinterpret_cast<SettleShared*>(dyn_smem);
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t i = blockIdx.x;
  // Inputs may be read before the copies are complete: the copying kernel has
  // itself waited for everything before it.  Every CTA waits for the copies
  // before it exits, so whoever waits for this kernel waits for them too.
  const RowSource from(a, i);
  if (from.bad) {
    wait_for_previous();
    return;
  }
  const RowPenalties pen(a, i, from.request);
  if (!pen.any()) {
    wait_for_previous();
    return;
  }
  const uint32_t V = (uint32_t)a.vocab;
  Raw* out = static_cast<Raw*>(a.out) + i * a.out_stride;
  const uint32_t* mask = from.mask_row >= 0 ? a.mask + from.mask_row * a.mask_stride : nullptr;
  auto allowed = [&](uint32_t j) { return !mask || (__ldg(mask + (j >> 5)) >> (j & 31) & 1u) != 0u; };
  const int32_t L = pen.L, biases = max(pen.b_hi - pen.b_lo, 0);
  if ((int64_t)L + biases > kSettleIds) {
    // A longer history: the row in parts of as many entries as fit, a count each.
    wait_for_previous();
    uint32_t* count = sh.id;
    constexpr int kPart = 2 * kSettleSlots;  // over id and marks
    for (uint32_t part = 0; part < V; part += kPart) {
      __syncthreads();
      for (int q = tid; q < kPart; q += kSettleThreads) count[q] = 0u;
      __syncthreads();
#pragma unroll 8
      for (int32_t at = tid; at < L; at += kSettleThreads) {
        const uint32_t j = (uint32_t)pen.history[at], e = j - part;
        if (j < V && e < (uint32_t)kPart) {
          if (at < pen.prompt)
            atomicOr(&count[e], 1u);
          else
            atomicAdd(&count[e], 2u);
        }
      }
      __syncthreads();
      for (int32_t q = pen.b_lo + tid; q < pen.b_hi; q += kSettleThreads) {
        const uint32_t j = (uint32_t)a.p.bias_ids[q], e = j - part;
        if (j >= V || e >= (uint32_t)kPart) continue;
        const uint32_t marks = atomicOr(&count[e], 0x80000000u);
        if (!(marks & 0x80000000u) && allowed(j))
          out[j] = E::put(pen.value(E::get(out[j]), marks, a.p.bias_values[q], true));
      }
      __syncthreads();
      for (uint32_t e = tid; e < (uint32_t)kPart && part + e < V; e += kSettleThreads) {
        const uint32_t marks = count[e], j = part + e;
        if (marks != 0u && !(marks & 0x80000000u) && allowed(j))
          out[j] = E::put(pen.value(E::get(out[j]), marks, 0.f, false));
      }
    }
    return;
  }
  // A batch of ids at a time.  Compare-and-swap takes the lanes of a warp one by
  // one, so most ids are placed without it: each pending one that finds its slot
  // free writes itself there and sees after a barrier whether it, or an equal
  // one, is what stayed; else it moves a slot on.  At a load of 60% three
  // quarters are placed in each of the two rounds; what is left is swapped in
  // (the table is never full, so that ends).  A batch begins when every warp has
  // swapped in what it had left of the one before: the rounds' test and store
  // are two accesses, and a swap between them would be overwritten.
  uint32_t id[kSettleHistory];
  auto insert = [&](uint32_t pending, uint32_t output) {  // bits: ids to insert, occurrences past the prompt
    int at[kSettleHistory];
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q) at[q] = home_of(id[q]);
    const uint32_t all = pending;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
#pragma unroll
      for (int q = 0; q < kSettleHistory; ++q)
        if ((pending >> q & 1u) && sh.id[at[q]] == 0u) sh.id[at[q]] = id[q] + 1u;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kSettleHistory; ++q)
        if (pending >> q & 1u) {
          if (sh.id[at[q]] == id[q] + 1u)
            pending &= ~(1u << q);
          else
            at[q] = slot_after(at[q]);
        }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q)
      if (pending >> q & 1u) at[q] = slot_of(sh, id[q], at[q]);
    uint32_t fresh = 0u;
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q)
      if (all >> q & 1u) {
        const uint32_t was = output >> q & 1u ? atomicAdd(&sh.marks[at[q]], 2u) : atomicOr(&sh.marks[at[q]], 1u);
        if (was == 0u) fresh |= 1u << q;
      }
    if (!__any_sync(0xFFFFFFFFu, fresh != 0u)) return;
    const int mine = __popc(fresh);
    int upto = mine;  // with this lane
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += t;
    }
    int n = 0;
    if (lane == 31) n = atomicAdd(&sh.listed, upto);
    n = __shfl_sync(0xFFFFFFFFu, n, 31) + upto - mine;
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q)
      if (fresh >> q & 1u) sh.list[n++] = (uint16_t)at[q];
  };
  auto fetch = [&](int32_t at) {
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q)
      id[q] = at + q * kSettleThreads < L ? (uint32_t)pen.history[at + q * kSettleThreads] : 0xFFFFFFFFu;
  };
  fetch(tid);
  for (int q = tid; q < 2 * kSettleSlots / 4; q += kSettleThreads) dyn_smem[q] = make_uint4(0u, 0u, 0u, 0u);
  if (tid == 0) sh.listed = 0;
  __syncthreads();
  for (int32_t at = tid; at - tid < L; at += kSettleHistory * kSettleThreads) {
    if (at != tid) {
      fetch(at);
      __syncthreads();
    }
    uint32_t pending = 0u, output = 0u;
#pragma unroll
    for (int q = 0; q < kSettleHistory; ++q) {
      if (id[q] < V) pending |= 1u << q;
      if (at + q * kSettleThreads >= pen.prompt) output |= 1u << q;
    }
    insert(pending, output);
  }
  __syncthreads();
  // biased entries belong to the thread of their bias
  auto claim = [&](uint32_t j, uint32_t* marks) {  // whether this bias is its id's first; *marks as before
    const int at = slot_of(sh, j, home_of(j));
    const uint32_t was = atomicOr(&sh.marks[at], 0x80000000u);
    *marks = was;
    return !(was & 0x80000000u);
  };
  uint32_t bias_j = V, bias_marks = 0u;
  float bias_v = 0.f;
  if (tid < biases) {
    const uint32_t j = (uint32_t)a.p.bias_ids[pen.b_lo + tid];
    bias_v = a.p.bias_values[pen.b_lo + tid];
    if (j < V && claim(j, &bias_marks) && allowed(j)) bias_j = j;
  }
  const int listed = sh.listed;
  if (biases > kSettleThreads) {  // the remaining biases, one after another
    wait_for_previous();
    for (int32_t q = pen.b_lo + tid + kSettleThreads; q < pen.b_hi; q += kSettleThreads) {
      const uint32_t j = (uint32_t)a.p.bias_ids[q];
      uint32_t marks;
      if (j < V && claim(j, &marks) && allowed(j))
        out[j] = E::put(pen.value(E::get(out[j]), marks, a.p.bias_values[q], true));
    }
  }
  if (biases > 0) __syncthreads();
  wait_for_previous();
  Raw bias_x = bias_j < V ? out[bias_j] : E::neg_inf();
  for (int q = tid; q < listed; q += kSettleBatch * kSettleThreads) {
    uint32_t j[kSettleBatch], marks[kSettleBatch];
    float x[kSettleBatch];
#pragma unroll
    for (int k = 0; k < kSettleBatch; ++k) {
      j[k] = V;
      if (q + k * kSettleThreads < listed) {
        const int slot = sh.list[q + k * kSettleThreads];
        marks[k] = sh.marks[slot];
        if (!(marks[k] & 0x80000000u)) {
          j[k] = sh.id[slot] - 1u;
          x[k] = E::get(out[j[k]]);
          if (!allowed(j[k])) j[k] = V;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kSettleBatch; ++k)
      if (j[k] < V) out[j[k]] = E::put(pen.value(x[k], marks[k], 0.f, false));
  }
  if (bias_j < V) out[bias_j] = E::put(pen.value(E::get(bias_x), bias_marks, bias_v, true));
}

constexpr int64_t kPairBytesPerId = 64 * 1024;  // of logits per id that a history may hold

// ls_set_process_policy: 0 = chosen from the batch; 1 = one kernel; 2 = the pair.
static std::atomic<int> g_policy{0};

template <typename TIn>
static ls_status launch_pair(ProcessArgs a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  static std::atomic<int> done[kMaxDevices];
  const int64_t units = row_units(a.vocab, dtype), runs = (units + kCopyUnits - 1) / kCopyUnits;
  if (runs * n > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  a.keep = (int64_t)n * a.vocab * Elem<TIn>::kBytes * 5 <= (int64_t)device_attr<cudaDevAttrL2CacheSize>() * 3;
  const ls_status rc = launch_kernel(copy_kernel<TIn>, dim3((unsigned)(runs * n)), kCopyThreads, 1, 0, st, a, (int)runs, kCopyUnits);
  if (rc != LS_OK || !(a.has_params && (a.p.tokens || a.p.bias_offsets))) return rc;
  if (!open_limits(settle_kernel<TIn>, done)) return LS_ERR_CUDA;
  return launch_kernel(settle_kernel<TIn>, dim3((unsigned)n), kSettleThreads, 1, sizeof(SettleShared), st, a);
}

template <typename TIn, typename Slot>
static ls_status launch(const ProcessArgs& a, ls_dtype dtype, int32_t n, cudaStream_t st) {
  const int64_t wide = (row_units(a.vocab, dtype) + 4 * kProcThreads - 1) / (4 * kProcThreads) * n;
  const int sms = device_attr<cudaDevAttrMultiProcessorCount>();
  // The pair copies at the speed of memory and spares what a mask forbids, but
  // settles a row on one SM; the one kernel spreads a row's touched entries over its
  // tiles.  Measured in us, one kernel / pair, with lengths spread over their
  // logarithm up to the buffer's, and with every row that long:
  //   1024 x 262144 fp32, masks, buffers of 2048    358 / 302   414 / 369
  //   the same, no masks                            303 / 346   351 / 407
  //   1024 x 262144 fp32, masks, buffers of 8192    396 / 368   703 / 618
  //   256 x 128256 bf16, masks, buffers of 512       31 /  29    32 /  30
  //   the same, buffers of 2048                      33 /  35    40 /  41
  //   the same, buffers of 8192                      44 /  62    78 /  90
  // Lengths lie on the device, so the rule goes by the buffer's; it does not look
  // for a mask, without which the one kernel would be the faster one.
  const bool light = !a.has_params || !a.p.tokens ||
                     (int64_t)n * a.vocab * Elem<TIn>::kBytes >= (int64_t)a.p.token_capacity * kPairBytesPerId;
  const int policy = g_policy.load(std::memory_order_relaxed);
  if (policy == 2 || (policy == 0 && wide >= 8 * sms && light)) return launch_pair<TIn>(a, dtype, n, st);
  return wide < 2 * sms ? launch<TIn, Slot, 1>(a, dtype, n, st) : launch<TIn, Slot, 4>(a, dtype, n, st);
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
    if (a.p.token_capacity >= kMostListed || a.p.bias_count >= kMostListed) return LS_ERR_UNSUPPORTED;
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

extern "C" int ls_set_process_policy(int policy) {
  if (policy < 0 || policy > 2) return (int)LS_ERR_INVALID_ARG;
  g_policy.store(policy, std::memory_order_relaxed);
  return (int)LS_OK;
}
