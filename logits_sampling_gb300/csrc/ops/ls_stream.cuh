// ls_stream.cuh -- a logits row streamed through registers, split over the
// CTAs of a cluster where one CTA would be too slow or its share too large.
//
// The row is seen as 32-byte units aligned in global memory (16 bf16 or 8 fp32
// entries).  CTA q of C owns a contiguous run of units; its threads take them in
// turn, a few (a stage) at a time, with the next stage's loads in flight while
// one is computed.  The units that lie wholly in the row are one 256-bit load,
// the row's first and last partial unit are read entry by entry, with -inf in
// the places outside the row.
//
// Registers rather than shared memory hold what is in flight: the same kernels
// with a row's share copied to the shared memory of a cluster took 173 us
// against 44 (20 best of 672 x 151936 bf16) and 96 against 32 (the loss there);
// a stream alone reaches the measured copy rate this way.
#pragma once

#include "ls_row_ops.cuh"

namespace lsg {
namespace ops {

constexpr int kStage = 2;  // units of a thread per stage
constexpr int kMaxCluster = 8;

// ---------------------------------------------------------------------------
// Cluster primitives
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(rank));
  return d;
}
__device__ __forceinline__ void peer_store(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void peer_store2(uint32_t a, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_add(uint32_t a, uint32_t v) {
  uint32_t o;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(a), "r"(v) : "memory");
  return o;
}

// Programmatic dependent launch, as the sampling kernels do it: a kernel may be
// scheduled while the one before it on the stream drains; every CTA waits for
// that one's completion before it touches memory, and lets the next kernel be
// scheduled once its own stream is done.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------------------
// 32-byte units by type
// ---------------------------------------------------------------------------
// A streamed line leaves L2 first: what every CTA reuses (the kernel's code among
// it) stays.
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t pol;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.nc.L1::no_allocate.L2::cache_hint.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p), "l"(stream_policy()));
}
// The same as an ordinary load, for memory that the kernel itself may write
// later (an output over its input).
__device__ __forceinline__ void load32_plain(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p), "l"(stream_policy())
               : "memory");
}
// And with no wish about L2.
__device__ __forceinline__ void load32_normal(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
// And where the line is read again soon: it leaves L2 last.
__device__ __forceinline__ void load32_keep(const void* p, uint32_t (&w)[8]) {
  uint64_t pol;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p), "l"(pol)
               : "memory");
}
__device__ __forceinline__ void store32_normal(void* p, const uint32_t (&w)[8]) {  // may be read again from L2
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
enum { LOAD_ONCE, LOAD_PLAIN, LOAD_KEEP, LOAD_NORMAL };
template <int kHow>
__device__ __forceinline__ void load_as(const void* p, uint32_t (&w)[8]) {
  if (kHow == LOAD_ONCE)
    load32(p, w);
  else if (kHow == LOAD_PLAIN)
    load32_plain(p, w);
  else if (kHow == LOAD_KEEP)
    load32_keep(p, w);
  else
    load32_normal(p, w);
}
// A store whose line leaves L2 first.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.cs.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <typename TIn>
struct Unit;

template <>
struct Unit<bf16_tag> {
  static constexpr int kN = 16;
  // NaNs become -inf (max with -inf drops a NaN).
  __device__ __forceinline__ static void clean(uint32_t (&w)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = bmax2(w[q], 0xFF80FF80u);
  }
  // Maximum of a unit, NaNs ignored (NaN where there is nothing else).
  __device__ __forceinline__ static float max(const uint32_t (&w)[8]) {
    const uint32_t m = bmax2(bmax2(bmax2(w[0], w[1]), bmax2(w[2], w[3])), bmax2(bmax2(w[4], w[5]), bmax2(w[6], w[7])));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  __device__ __forceinline__ static f32x2 pair(const uint32_t (&w)[8], int q) {
    return pack2(__uint_as_float(w[q] << 16), __uint_as_float(w[q] & 0xFFFF0000u));
  }
  __device__ __forceinline__ static void set_pair(uint32_t (&w)[8], int q, float lo, float hi) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[q]) : "f"(hi), "f"(lo));
  }
  // -inf in the entries whose bit is set.
  __device__ __forceinline__ static void drop(uint32_t (&w)[8], uint32_t bits) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {  // bytes 0-1 and 2-3 of the word, or of the replacement
      const uint32_t two = bits >> (2 * q) & 3u;
      w[q] = __byte_perm(w[q], 0xFF80FF80u, 0x3210u | (two & 1u) * 0x44u | (two & 2u) * 0x2200u);
    }
  }
};

template <>
struct Unit<float> {
  static constexpr int kN = 8;
  __device__ __forceinline__ static void clean(uint32_t (&w)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(fmaxf(__uint_as_float(w[q]), kNegInf));
  }
  __device__ __forceinline__ static float max(const uint32_t (&w)[8]) {
    return fmax3(fmax3(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2])),
                 fmax3(__uint_as_float(w[3]), __uint_as_float(w[4]), __uint_as_float(w[5])),
                 fmaxf(__uint_as_float(w[6]), __uint_as_float(w[7])));
  }
  __device__ __forceinline__ static f32x2 pair(const uint32_t (&w)[8], int q) {
    return pack2(__uint_as_float(w[2 * q]), __uint_as_float(w[2 * q + 1]));
  }
  __device__ __forceinline__ static void set_pair(uint32_t (&w)[8], int q, float lo, float hi) {
    w[2 * q] = __float_as_uint(lo);
    w[2 * q + 1] = __float_as_uint(hi);
  }
  __device__ __forceinline__ static void drop(uint32_t (&w)[8], uint32_t bits) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (bits & (1u << q)) w[q] = 0xFF800000u;
  }
};

// Entry e of a unit for an index that is not known beforehand.
template <typename TIn>
__device__ __forceinline__ float entry_at(const uint32_t (&w)[8], int e) {
  const int at = Unit<TIn>::kN == 8 ? e : e >> 1;
  uint32_t word = w[0];
#pragma unroll
  for (int q = 1; q < 8; ++q) word = select_word(word, w[q], at == q);
  if (Unit<TIn>::kN == 8) return __uint_as_float(word);
  return __uint_as_float(e & 1 ? word & 0xFFFF0000u : word << 16);
}

// exp((v - M) / T), c = log2(e) / T, for v <= M; entries at an infinite
// maximum share it.
__device__ __forceinline__ float rel_exp(float v, float M, float c) { return v == M ? 1.f : ex2((v - M) * c); }

// exp((v - m) / T) for many v against one m.  fma(v, c, -r) with r = RN(m c)
// is one instruction for two entries and exact up to its last rounding; the
// common factor 2^(m c - r) that r's rounding leaves is known (`scale` takes
// it out).  For |m c| of 2^16 and above that factor would matter, and for an
// infinite m the difference is undefined: there each entry is subtracted first.
struct ExpAgainst {
  float m, c, r, scale;
  bool fast;
  __device__ __forceinline__ void init(float m_, float c_) {
    m = m_;
    c = c_;
    r = m * c;
    fast = fabsf(r) < 65536.f;
    scale = fast ? ex2(-fmaf(m, c, -r)) : 1.f;
  }
  // The exponentials of a pair over `scale`.
  __device__ __forceinline__ f32x2 pair_fast(f32x2 v) const {
    float a, b;
    unpack2(fma2(v, pack2(c, c), pack2(-r, -r)), a, b);
    return pack2(ex2(a), ex2(b));
  }
  __device__ __forceinline__ f32x2 pair_slow(f32x2 v) const {
    float a, b;
    unpack2(v, a, b);
    return pack2(rel_exp(a, m, c), rel_exp(b, m, c));
  }
};

// A warp's running maximum m and each thread's sum of exp((v - m) / T).  The
// maximum is the warp's, so raising it is one branch for all lanes and rare
// after the first stages.
struct OnlineSum {
  ExpAgainst x;
  f32x2 s0, s1;
  __device__ __forceinline__ void init(float c) {
    x.init(kNegInf, c);
    s0 = s1 = 0ull;
  }
  // Before units of maximum um in this lane are added (all lanes call).
  __device__ __forceinline__ void raise(float um) {
    um = warp_max(um);  // NaN compares false below
    if (um > x.m) {
      const float f = x.m > kNegInf ? x.scale * rel_exp(x.m, um, x.c) : 0.f;
      x.init(um, x.c);
      const float g = f / x.scale;
      s0 = mul2(s0, pack2(g, g));
      s1 = mul2(s1, pack2(g, g));
    }
  }
  template <typename TIn>
  __device__ __forceinline__ void add(const uint32_t (&w)[8]) {
    if (x.fast) {
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; q += 2) {
        s0 = add2(s0, x.pair_fast(Unit<TIn>::pair(w, q)));
        s1 = add2(s1, x.pair_fast(Unit<TIn>::pair(w, q + 1)));
      }
    } else if (x.m > kNegInf) {
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) s0 = add2(s0, x.pair_slow(Unit<TIn>::pair(w, q)));
    } else {  // nothing yet but -inf and NaN: the sum shall show a NaN
      uint32_t other = 0u;
#pragma unroll
      for (int q = 0; q < 8; ++q) other |= w[q] ^ (Unit<TIn>::kN == 16 ? 0xFF80FF80u : 0xFF800000u);
      if (other) s0 = pack2(quiet_nan(), quiet_nan());
    }
  }
  __device__ __forceinline__ float sum() const {
    float a, b;
    unpack2(add2(s0, s1), a, b);
    return (a + b) * x.scale;
  }
};

// ---------------------------------------------------------------------------
// One CTA's run of a row's units
// ---------------------------------------------------------------------------
// A unit that is not wholly in the row, whose entry 0 has index j: once or twice
// per row, so out of the loops' code.
template <typename TIn>
__device__ __noinline__ void load_edge(const typename Elem<TIn>::Raw* row, int64_t j, int64_t V, uint32_t* w) {
  constexpr int kN = Unit<TIn>::kN;
  typename Elem<TIn>::Raw* e = reinterpret_cast<typename Elem<TIn>::Raw*>(w);
#pragma unroll 1
  for (int q = 0; q < kN; ++q) e[q] = j + q >= 0 && j + q < V ? row[j + q] : Elem<TIn>::neg_inf();
}

// T: threads of the CTA.
template <typename TIn, int T>
struct Run {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  static constexpr int kN = Unit<TIn>::kN;
  const Raw* row;
  const char* base;  // unit 0 of the run
  int64_t V;
  int64_t j0;        // vocabulary index of the run's first place (negative in the row's first unit)
  int n;             // units
  int f, l;          // units [f, l) lie wholly in the row

  __device__ __forceinline__ void init(const void* matrix, int64_t src, int64_t stride, int64_t vocab, int upc, int rank) {
    row = static_cast<const Raw*>(matrix) + src * stride;
    V = vocab;
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 31u) / E::kBytes);
    const int units = (int)((off + V + kN - 1) / kN), u0 = rank * upc;
    j0 = (int64_t)u0 * kN - off;
    base = reinterpret_cast<const char*>(row) + j0 * E::kBytes;
    n = max(min(upc, units - u0), 0);
    f = u0 == 0 && off > 0 ? 1 : 0;
    l = min(n, (int)((off + V) / kN) - u0);
  }
  __device__ __forceinline__ int64_t index(int u) const { return j0 + (int64_t)u * kN; }
  __device__ __forceinline__ bool full(int u) const { return u >= f && u < l; }
  // Place of a vocabulary index in the run, -1 when another CTA holds it.
  __device__ __forceinline__ int place(int64_t j) const {
    const int64_t e = j - j0;
    return e >= 0 && e < (int64_t)n * kN ? (int)e : -1;
  }
  // A unit's words (u < n); kHow: LOAD_*.
  template <int kHow = LOAD_ONCE>
  __device__ __forceinline__ void load(int u, uint32_t (&w)[8]) const {
    if (full(u)) {
      load_as<kHow>(base + (int64_t)u * 32, w);
    } else {
      uint32_t edge[8];
      load_edge<TIn>(row, index(u), V, edge);
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = edge[q];
    }
  }
  // Writes unit u of an output row with this row's indices (`same`: and its alignment).
  __device__ __forceinline__ void store(Raw* out, bool same, int u, const uint32_t (&w)[8], bool keep = false) const {
    const int64_t j = index(u);
    if (same && full(u)) {
      if (keep)
        store32_normal(out + j, w);
      else
        store32(out + j, w);
    } else {
      Raw e[kN];
      memcpy(e, w, 32);
#pragma unroll
      for (int q = 0; q < kN; ++q)
        if (j + q >= 0 && j + q < V) out[j + q] = e[q];
    }
  }
  __device__ __forceinline__ bool aligned_with(const Raw* out) const {
    return ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(row)) & 31u) == 0;
  }
  // Visits this thread's units in order, kStage at a time: visit(u, w) with the
  // words of units u and u + T (units past n as -inf); the first stage has been
  // loaded by prefetch().  A stage whose units all lie wholly in the row and the
  // run (for the whole CTA: one branch) is loaded without further checks.
  typedef uint32_t Stage[kStage][8];
  static constexpr int kStep = kStage * T;
  __device__ __forceinline__ bool whole(int u) const {
    const int first = u - (int)threadIdx.x;
    return first >= f && first + kStep <= l;
  }
  template <int kHow = LOAD_ONCE>
  __device__ __forceinline__ void prefetch(int u, Stage& w) const {
    if (whole(u)) {
      const char* p = base + (int64_t)u * 32;
#pragma unroll
      for (int k = 0; k < kStage; ++k) {
        load_as<kHow>(p + k * T * 32, w[k]);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const int uk = u + k * T;
      if (uk < n) {
        load<kHow>(uk, w[k]);
      } else {
        const uint32_t none = E::kBytes == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (int q = 0; q < 8; ++q) w[k][q] = none;
      }
    }
  }
  // The trip count is the warp's: every lane of a warp visits the same stages.
  template <int kHow = LOAD_ONCE, typename F>
  __device__ __forceinline__ void stream(Stage& cur, F visit) const {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int u = threadIdx.x; u - lane < n; u += kStep) {
      Stage next;
      prefetch<kHow>(u + kStep, next);
      visit(u, cur);
      move(next, cur);
    }
  }
  __device__ __forceinline__ static void move(const Stage& from, Stage& to) {
#pragma unroll
    for (int k = 0; k < kStage; ++k)
#pragma unroll
      for (int q = 0; q < 8; ++q) to[k][q] = from[k][q];
  }
  // The same from the run's last stage to its first.
  __device__ __forceinline__ int last_stage() const { return (n - 1) / kStep * kStep + (int)threadIdx.x; }
  template <int kHow = LOAD_ONCE, typename F>
  __device__ __forceinline__ void stream_back(Stage& cur, F visit) const {
#pragma unroll 1
    for (int u = last_stage(); u >= 0; u -= kStep) {
      Stage next;
      if (u >= kStep) prefetch<kHow>(u - kStep, next);
      visit(u, cur);
      move(next, cur);
    }
  }
};

// (maximum, sum) of the block from each warp's maximum and thread's sum, in
// every thread; the sum's order is fixed.  `red` holds a pair per warp.
template <int kWarps>
__device__ __forceinline__ float2 block_lse(float wm, float s, float c, float2* red) {
  const float ws = warp_reduce(s, OpAddF());
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(wm, ws);
  __syncthreads();
  const float2 r = red[threadIdx.x & (kWarps - 1)];
  const float bm = warp_max(r.x);
  float bs = r.y * (r.x > kNegInf ? rel_exp(r.x, bm, c) : 0.f);  // a NaN stays one
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) bs += __shfl_xor_sync(0xFFFFFFFFu, bs, o);
  return make_float2(bm, bs);
}

// ---------------------------------------------------------------------------
// Host: cluster size and launch
// ---------------------------------------------------------------------------
struct StreamPlan {
  int ctas;  // per row
  int upc;   // units per CTA
};

static inline int64_t row_units(int64_t vocab, ls_dtype dtype) {  // at the worst alignment
  const int64_t e = dtype == LS_DTYPE_F32 ? 4 : 2;
  return (vocab * e + 31 - e) / 32 + 1;
}

// The fewest CTAs per row that keep a CTA's run within `most` bytes and, while
// runs stay above kRunLeast bytes, give each SM `per_sm` CTAs (half of what it
// holds).  Measured on 128256 bf16 entries a row, us with 1 / 2 / 4 / 8 CTAs per
// row: the 20 best of 8 rows 16.1 / 12.7 / 9.7 / 8.4, of 150 26.3 / 18.2 / 16.4 /
// 20.7, of 600 36.9 / 34.6 / 48.4, of 672 40.1 / 48.4 / 52.4; the distillation
// loss of 8 rows 12.8 / 9.4 / 7.2 / 5.9, of 150 16.3 / 13.1 / 11.5 / 15.0, of 304
// 20.5 / 17.3 / 23.7, of 400 22.0 / 24.9 / 27.8.
constexpr int64_t kRunLeast = 16 * 1024;

static inline StreamPlan plan_stream(int32_t n, int64_t vocab, ls_dtype dtype, int64_t most, int per_sm) {
  const int64_t units = row_units(vocab, dtype), sms = device_attr<cudaDevAttrMultiProcessorCount>();
  int c = 1;
  while (c < kMaxCluster && (units + c - 1) / c * 32 > most) c *= 2;
  while (c < kMaxCluster && (int64_t)n * c <= per_sm * sms && units * 32 / (2 * c) >= kRunLeast) c *= 2;
  return StreamPlan{c, (int)((units + c - 1) / c)};
}

// Lets a kernel use the device's whole shared memory per CTA (once per device; `done` belongs to the kernel).
template <typename Kernel>
static bool open_limits(Kernel kernel, std::atomic<int>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_relaxed)) return true;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return false;
  const int most = device_attr<cudaDevAttrMaxSharedMemoryPerBlockOptin>() - (int)fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
    return false;
  if (dev >= 0 && dev < kMaxDevices) done[dev].store(1, std::memory_order_relaxed);
  return true;
}

// Launches a kernel in clusters of `cluster` CTAs, dependent on its predecessor.
template <typename... Params, typename... Args>
static ls_status launch_kernel(void (*kernel)(Params...), dim3 grid, int threads, int cluster, size_t smem,
                               cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return LS_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}

// Launches one cluster of p.ctas CTAs per row.
template <typename Kernel, typename Args>
static ls_status launch_rows(Kernel kernel, const Args& a, const StreamPlan& p, int threads, size_t smem, int32_t n,
                             cudaStream_t stream, std::atomic<int>* done) {
  if ((int64_t)n * p.ctas > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  if (!open_limits(kernel, done)) return LS_ERR_CUDA;
  return launch_kernel(kernel, dim3((unsigned)((int64_t)n * p.ctas)), threads, p.ctas, smem, stream, a, p.upc);
}

}  // namespace ops
}  // namespace lsg
