// ls_row_ops.cuh -- what the kernels of include/ls_row_ops.h share: element
// access by type, the row an output row reads, argument checks, and the
// device limits they are launched under.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ls_device.cuh"
#include "ls_row_ops.h"

namespace lsg {
namespace ops {

// Storage of one logit: bf16 as its bits, fp32 as itself.
template <typename TIn>
struct Elem;

template <>
struct Elem<float> {
  typedef float Raw;
  static constexpr int kBytes = 4;
  __device__ __forceinline__ static float get(Raw r) { return r; }
  __device__ __forceinline__ static Raw put(float v) { return v; }
  __device__ __forceinline__ static Raw neg_inf() { return kNegInf; }
};

template <>
struct Elem<bf16_tag> {
  typedef uint16_t Raw;
  static constexpr int kBytes = 2;
  __device__ __forceinline__ static float get(Raw r) { return __uint_as_float((uint32_t)r << 16); }
  // round to nearest even, NaN kept
  __device__ __forceinline__ static Raw put(float v) {
    Raw r;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(v));
    return r;
  }
  __device__ __forceinline__ static Raw neg_inf() { return (Raw)0xFF80u; }
};

__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// NaN logits are read as -inf.
__device__ __forceinline__ float guard(float v) { return v == v ? v : kNegInf; }

constexpr int kMaxDevices = 64;

// One device attribute, looked up once per device (0 when unknown).
template <cudaDeviceAttr A>
static int device_attr() {
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < kMaxDevices && (v = cache[dev].load(std::memory_order_relaxed)) > 0) return v;
  if (cudaDeviceGetAttribute(&v, A, dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < kMaxDevices) cache[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Largest vocab of the calls that keep a few bits per entry in shared memory.
static inline int64_t max_row(ls_dtype) { return int64_t(1) << 22; }

static inline bool matrix_ok(const void* p, ls_dtype dtype, int64_t vocab, int64_t row_stride) {
  if (!p || (dtype != LS_DTYPE_F32 && dtype != LS_DTYPE_BF16)) return false;
  if ((reinterpret_cast<uintptr_t>(p) & (dtype == LS_DTYPE_F32 ? 3u : 1u)) != 0) return false;
  return vocab >= 1 && vocab < 0x7FFFFFFFll && row_stride >= vocab;
}

// Whether `out` (n x out_stride) may be written while `in` (rows x in_stride)
// is read: apart, or the same matrix where the caller works in place.
static inline bool overlap_ok(const void* in, int64_t rows, int64_t in_stride, const void* out, int64_t n,
                              int64_t out_stride, int64_t vocab, ls_dtype dtype, bool in_place) {
  const uintptr_t e = dtype == LS_DTYPE_F32 ? 4u : 2u;
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  const uintptr_t a_end = a + ((uintptr_t)(rows - 1) * (uintptr_t)in_stride + (uintptr_t)vocab) * e;
  const uintptr_t b_end = b + ((uintptr_t)(n - 1) * (uintptr_t)out_stride + (uintptr_t)vocab) * e;
  if (a == b) return in_place && in_stride == out_stride;
  return a_end <= b || b_end <= a;
}

}  // namespace ops
}  // namespace lsg
