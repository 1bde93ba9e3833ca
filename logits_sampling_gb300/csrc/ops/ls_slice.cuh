// ls_slice.cuh -- a logits row held in shared memory, over the CTAs of a
// cluster where one CTA's share would be too large.
//
// The row is seen as 16-byte units aligned in global memory.  CTA q of C owns
// a contiguous run of units: the units that lie wholly in the row arrive by
// bulk copies (both addresses 16-byte aligned by construction), the row's
// first and last partial unit by plain loads with -inf in the places outside
// the row.  The row is read from global memory once; every later pass reads
// shared memory.
#pragma once

#include "ls_row_ops.cuh"

namespace lsg {
namespace ops {

constexpr int kSliceThreads = 512;
constexpr int kSliceWarps = kSliceThreads / 32;
constexpr int kChunks = 4;         // bulk copies (and barriers) per slice: the first pass starts on the first chunk
constexpr int kMaxCluster = 16;
constexpr uint32_t kWaitTries = 1u << 20;  // of a barrier wait, of kWaitNs each: about two seconds
constexpr uint32_t kWaitNs = 2000;

// ---------------------------------------------------------------------------
// Cluster and barrier primitives
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

__device__ __forceinline__ void mbar_init(uint64_t* bar) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// Waits for the barrier's first phase.  False when the tries ran out.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar) {
  const uint32_t a = smem_addr(bar);
  for (uint32_t t = 0; t < kWaitTries; ++t) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0, %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(a), "r"(kWaitNs)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// ---------------------------------------------------------------------------
// 16-byte units by type
// ---------------------------------------------------------------------------
template <typename TIn>
struct Unit;

template <>
struct Unit<bf16_tag> {
  static constexpr int kN = 8;
  // The unit with its NaNs read as -inf (max with -inf drops a NaN).
  __device__ __forceinline__ static uint4 clean(uint4 u) {
    const uint32_t low = 0xFF80FF80u;
    return make_uint4(bmax2(u.x, low), bmax2(u.y, low), bmax2(u.z, low), bmax2(u.w, low));
  }
  __device__ __forceinline__ static float max(uint4 u) {
    const uint32_t m = bmax2(bmax2(u.x, u.y), bmax2(u.z, u.w));
    return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), kNegInf);
  }
  __device__ __forceinline__ static f32x2 pair(uint4 u, int q) {
    const uint32_t w = q == 0 ? u.x : q == 1 ? u.y : q == 2 ? u.z : u.w;
    return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ __forceinline__ static uint4 make(const float (&v)[kN]) {
    return make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
  }
};

template <>
struct Unit<float> {
  static constexpr int kN = 4;
  __device__ __forceinline__ static uint4 clean(uint4 u) {
    return make_uint4(__float_as_uint(fmaxf(__uint_as_float(u.x), kNegInf)),
                      __float_as_uint(fmaxf(__uint_as_float(u.y), kNegInf)),
                      __float_as_uint(fmaxf(__uint_as_float(u.z), kNegInf)),
                      __float_as_uint(fmaxf(__uint_as_float(u.w), kNegInf)));
  }
  __device__ __forceinline__ static float max(uint4 u) {
    return fmaxf(fmax3(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)),
                 fmaxf(__uint_as_float(u.w), kNegInf));
  }
  __device__ __forceinline__ static f32x2 pair(uint4 u, int q) {
    return q == 0 ? pack2(__uint_as_float(u.x), __uint_as_float(u.y))
                  : pack2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  __device__ __forceinline__ static uint4 make(const float (&v)[kN]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};

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

// ---------------------------------------------------------------------------
// One CTA's slice of a row
// ---------------------------------------------------------------------------
template <typename TIn>
struct Slice {
  using E = Elem<TIn>;
  using Raw = typename E::Raw;
  static constexpr int kN = Unit<TIn>::kN;
  uint4* buf;      // the units in shared memory
  const Raw* row;  // the row in global memory
  int64_t V;
  int off;         // entries of the first unit that lie before the row
  int u0, n;       // first unit of the slice, units in it
  int chunk;       // units per chunk

  __device__ __forceinline__ void init(uint4* smem, const void* matrix, int64_t src, int64_t stride, int64_t vocab,
                                       int upc, int rank) {
    buf = smem;
    row = static_cast<const Raw*>(matrix) + src * stride;
    V = vocab;
    off = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / E::kBytes);
    const int units = (int)((off + V + kN - 1) / kN);
    u0 = rank * upc;
    n = max(min(upc, units - u0), 0);
    chunk = (n + kChunks - 1) / kChunks;
  }
  // Units [first, last) of the slice lie wholly in the row.
  __device__ __forceinline__ int full_first() const { return u0 == 0 && off > 0 ? 1 : 0; }
  __device__ __forceinline__ int full_last() const { return min(n, (int)((off + V) / kN) - u0); }
  // Vocabulary index of entry e of the slice (outside [0, V) in an edge unit's padding).
  __device__ __forceinline__ int64_t index(int e) const { return (int64_t)u0 * kN + e - off; }
  // Slice entry of a vocabulary index, -1 when another CTA holds it.
  __device__ __forceinline__ int entry(int64_t j) const {
    const int64_t e = j + off - (int64_t)u0 * kN;
    return e >= 0 && e < (int64_t)n * kN ? (int)e : -1;
  }
  __device__ __forceinline__ Raw* raw() const { return reinterpret_cast<Raw*>(buf); }

  // Starts the copies (thread 0) and fills the edge units; all threads call.
  // Ends with a block barrier: nobody waits on a barrier that is not yet
  // initialised, or reads an edge unit before it is filled.
  __device__ __forceinline__ void start(uint64_t* bars) const {
    if (threadIdx.x == 0) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) mbar_init(&bars[k]);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      const char* base = reinterpret_cast<const char*>(row) - off * E::kBytes + (int64_t)u0 * 16;
      const int f = full_first(), l = full_last();
      for (int k = 0; k < kChunks; ++k) {
        const int a = max(k * chunk, f), b = min((k + 1) * chunk, l);
        const uint32_t bytes = b > a ? (uint32_t)(b - a) * 16u : 0u;
        mbar_expect(&bars[k], bytes);
        if (bytes) bulk_load(buf + a, base + (int64_t)a * 16, bytes, &bars[k]);
      }
    }
    if (threadIdx.x < 2 * 32 && (threadIdx.x & 31) < kN) {  // the two possible edge units, an entry per lane
      const int u = threadIdx.x < 32 ? 0 : n - 1;
      const bool edge = threadIdx.x < 32 ? full_first() == 1 : (n > 0 && full_last() < n);
      if (edge && n > 0) {
        const int e = u * kN + (int)(threadIdx.x & 31);
        const int64_t j = index(e);
        raw()[e] = j >= 0 && j < V ? row[j] : E::neg_inf();
      }
    }
    __syncthreads();
  }
};

// Block-wide maximum of 16 warps (all threads call; `red` holds kSliceWarps floats).
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_max(red[threadIdx.x & (kSliceWarps - 1)]);
}
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_reduce(v, OpAddF());
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kSliceWarps; ++w) s += red[w];
  return s;
}

// This thread's maximum over the slice, chunk by chunk as it arrives.
template <typename TIn>
__device__ __forceinline__ float slice_max(const Slice<TIn>& s, uint64_t* bars, bool* stalled) {
  float m = kNegInf;
  for (int k = 0; k < kChunks; ++k) {
    if (!mbar_wait(&bars[k])) *stalled = true;
    const int b = min((k + 1) * s.chunk, s.n);
    for (int u = k * s.chunk + (int)threadIdx.x; u < b; u += kSliceThreads) m = fmaxf(m, Unit<TIn>::max(s.buf[u]));
  }
  return m;
}

// This thread's sum of exp((v - m) / T) over the slice.
template <typename TIn>
__device__ __forceinline__ float slice_sum(const Slice<TIn>& s, const ExpAgainst& x) {
  f32x2 s0 = 0ull, s1 = 0ull;
  if (x.fast) {
    for (int u = threadIdx.x; u < s.n; u += kSliceThreads) {
      const uint4 w = Unit<TIn>::clean(s.buf[u]);
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; q += 2) {
        s0 = add2(s0, x.pair_fast(Unit<TIn>::pair(w, q)));
        s1 = add2(s1, x.pair_fast(Unit<TIn>::pair(w, q + 1)));
      }
    }
  } else if (x.m > kNegInf) {
    for (int u = threadIdx.x; u < s.n; u += kSliceThreads) {
      const uint4 w = Unit<TIn>::clean(s.buf[u]);
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) s0 = add2(s0, x.pair_slow(Unit<TIn>::pair(w, q)));
    }
  }
  float a, b;
  unpack2(add2(s0, s1), a, b);
  return (a + b) * x.scale;
}

// ---------------------------------------------------------------------------
// Host: cluster size and launch
// ---------------------------------------------------------------------------
struct SlicePlan {
  int ctas;     // per row
  int upc;      // units per CTA
  size_t smem;  // bytes of the slice
};

// Slices of at most kSliceTarget bytes leave three CTAs of a row or of
// different rows on an SM, so that one loads while another computes and a
// third writes.  A batch too small to give every SM a CTA is split further,
// down to slices of kSliceLeast bytes.
constexpr int64_t kSliceTarget = 68 * 1024;
constexpr int64_t kSliceLeast = 8 * 1024;

static inline SlicePlan plan_slices(int32_t n, int64_t vocab, ls_dtype dtype) {
  const int64_t e = dtype == LS_DTYPE_F32 ? 4 : 2;
  const int64_t units = (vocab * e + 15 - e) / 16 + 1;  // at the worst alignment
  const int64_t sms = device_attr<cudaDevAttrMultiProcessorCount>();
  int c = 1;
  while (c < kMaxCluster && (units + c - 1) / c * 16 > kSliceTarget) c *= 2;
  while (c < 8 && (int64_t)n * c < 2 * sms && units * 16 / (2 * c) >= kSliceLeast) c *= 2;
  SlicePlan p;
  p.ctas = c;
  p.upc = (int)((units + c - 1) / c);
  p.smem = (size_t)p.upc * 16;
  return p;
}

// Lets a kernel use the device's whole shared memory per CTA and clusters of
// 16 CTAs (once per device; `done` belongs to the kernel).
template <typename Kernel>
static bool open_limits(Kernel kernel, std::atomic<int>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_relaxed)) return true;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return false;
  const int most = device_attr<cudaDevAttrMaxSharedMemoryPerBlockOptin>() - (int)fa.sharedSizeBytes;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return false;
  if (dev >= 0 && dev < kMaxDevices) done[dev].store(1, std::memory_order_relaxed);
  return true;
}

// Launches one cluster of p.ctas CTAs per row.
template <typename Kernel, typename Args>
static ls_status launch_slices(Kernel kernel, const Args& a, const SlicePlan& p, size_t smem, int32_t n,
                               cudaStream_t stream, std::atomic<int>* done) {
  if ((int64_t)n * p.ctas > 0x7FFFFFFFll) return LS_ERR_UNSUPPORTED;
  if (!open_limits(kernel, done)) return LS_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)n * p.ctas));
  cfg.blockDim = dim3(kSliceThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)p.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, a, p.upc) != cudaSuccess) return LS_ERR_CUDA;
  return cudaPeekAtLastError() == cudaSuccess ? LS_OK : LS_ERR_CUDA;
}

}  // namespace ops
}  // namespace lsg
