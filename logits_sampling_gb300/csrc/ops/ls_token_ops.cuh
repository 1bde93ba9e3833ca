// ls_token_ops.cuh -- what the kernels of include/ls_token_ops.h share: one pass
// over a row for its maximum, sum and entropy term, the scalars of each
// operator, and the gradient of a unit of entries.
//
// Every operator is a function of lp and H of its rows, so every gradient is
//     d_j = 1 / T (g_lp [j = id] - q_j (g_lp + g_H (ln q_j + H)))
// with two numbers per row, g_lp and g_H: one kernel computes all of them.
#pragma once

#include "ls_stream.cuh"
#include "ls_token_ops.h"

namespace lsg {
namespace ops {

constexpr float kLn2 = 0.6931471805599453f;

// What a forward call leaves of a row (LS_TOKEN_STATS floats).
struct alignas(16) TokenStats {
  float M, over;          // reference of the sum, 1 / (S T)
  float id_lp, id_H;      // the token's gradient: g_lp * id_lp - g_H * id_H
  float g_lp;             // the loss's slopes g_lp and g_H; both 0: the row does not count
  int32_t up;             // the entry of the gradient from above that belongs to the row (kNoPair: none yet)
  float g_H;
  float mean;             // H - ln S
  float dirty;            // not 0: the row may hold NaNs
  float term, w;          // preference: weight * (lp - ref), the weight of a row that counts
  float term_lo;          // what `term` has lost to its rounding
};
constexpr int32_t kNoPair = 0x7FFFFFFF;
static_assert(sizeof(TokenStats) == sizeof(float) * LS_TOKEN_STATS, "the header's size of a row's stats");

enum TokenKind { KIND_SCORE, KIND_POLICY, KIND_PREFERENCE };

struct TokenArgs {
  const void* logits;
  int64_t vocab, row_stride;
  int32_t n;
  const int32_t* ids;
  float temperature, c, inv_T;  // c = log2(e) / T
  int kind;
  ls_policy policy;            // of a preference loss: weights and ref_log_probs only
  const int32_t* offsets;      // preference
  int32_t pairs;
  float* out_loss;             // score: the log-probs
  float* out_entropy;          // score
  float4* out_metrics;         // policy
  TokenStats* out_stats;
  void* out_grad;
  int64_t grad_stride;
  int32_t* error_word;
};

// ---------------------------------------------------------------------------
// One pass: maximum, sum and entropy term
// ---------------------------------------------------------------------------
// (M, S, E) of a set of entries: S = sum 2^y, E = sum y 2^y, y = (x - M) c, c =
// log2(e) / T, against a reference M (their maximum, or what is used in its place).
// H = ln S - ln 2 * E / S.
struct Moments {
  float m, s, e;
};

// 2^(d c) for what a whole sum is multiplied by: the product's rounding, up to 2^-24
// of an exponent of 20 or 30, is taken into account, and the exponential is e^z's
// series for |z| <= ln 2 / 2 (z^8 / 8! is 5e-9), because the instruction is low on
// average: 5.05e-8 of its result over 16.8 million exponents in [-20, 0], 1.42e-7 at
// most.
constexpr float kExpLow = 5.05e-8f;
__device__ __forceinline__ float factor(float d, float c) {
  const float y = d * c;
  if (!(y > -126.f)) return 0.f;
  const float n = rintf(y), z = ((y - n) + fmaf(d, c, -y)) * kLn2;
  float e = 1.f / 5040.f;
  e = fmaf(e, z, 1.f / 720.f);
  e = fmaf(e, z, 1.f / 120.f);
  e = fmaf(e, z, 1.f / 24.f);
  e = fmaf(e, z, 1.f / 6.f);
  e = fmaf(e, z, 0.5f);
  e = fmaf(e, z, 1.f);
  e = fmaf(e, z, 1.f);
  return e * __int_as_float(((int)n + 127) << 23);
}

// The same set against a maximum m >= a.m.  A NaN in a.s stays one.
__device__ __forceinline__ Moments rebase(const Moments& a, float m, float c) {
  if (!(a.m > kNegInf)) return Moments{m, a.s, a.e};
  const float f = a.m == m ? 1.f : factor(a.m - m, c);
  const float d = a.m == m ? 0.f : (a.m - m) * c;
  return Moments{m, a.s * f, f > 0.f ? f * (a.e + d * a.s) : 0.f};
}

// Below every entry that matters, above what overflows on the way to an
// exponent: what -inf, the type's lowest values and NaN are read as where 0 *
// inf would make a NaN of y 2^y.  Only where ExpAgainst is fast and c lies within
// [2^-64, 2^24]: there |m| < 2^80, so 2^((-2^100 - m) c) is 0 and the product finite.
constexpr float kFloor = -1.2676506e30f;        // -2^100, a bf16 value
constexpr uint32_t kFloorPair = 0xF180F180u;    // two of them as bf16
constexpr float kFloorExp = -300.f;             // 2^-300 is 0 in fp32

template <typename TIn>
__device__ __forceinline__ void lift(uint32_t (&w)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if (Unit<TIn>::kN == 16)
      w[q] = bmax2(w[q], kFloorPair);
    else
      w[q] = __float_as_uint(fmaxf(__uint_as_float(w[q]), kFloor));
  }
}
__device__ __forceinline__ bool lift_ok(float c) { return c >= 5.4210109e-20f && c <= 16777216.f; }
// y of one entry by subtraction, NaN and -inf at kFloorExp.
__device__ __forceinline__ float rel_log(float v, float m, float c) { return v == m ? 0.f : fmaxf((v - m) * c, kFloorExp); }

// ExpAgainst with its `scale`, 2^-delta, from a series: delta, what m c lost to its
// rounding, is below 2^-8, and the instruction is off by 2^-23 at 0 where all rows
// with the same maximum would share it.  While there is no reference (m = -inf) r is 0:
// what has been seen by then is -inf, which adds 0, or NaN, which shows.
struct Reference : ExpAgainst {
  float delta;
  __device__ __forceinline__ void none(float c_, bool lift) {
    m = kNegInf;
    c = c_;
    r = delta = 0.f;
    scale = 1.f;
    fast = !lift || lift_ok(c);
  }
  __device__ __forceinline__ void at(float m_, float c_, bool lift) {
    m = m_;
    c = c_;
    r = m * c;
    fast = fabsf(r) < 65536.f && (!lift || lift_ok(c));
    delta = fast ? fmaf(m, c, -r) : 0.f;
    const float t = -delta * kLn2;
    scale = fmaf(t, fmaf(t, fmaf(t, 0.16666667f, 0.5f), 1.f), 1.f);
  }
};

// The sum of a unit's pairs, in a tree, before it meets what has been added up so
// far: term by term a row's many small entries were lost to a large sum's rounding
// (2e-7 of S on average, the same in every row).
template <int kN>
__device__ __forceinline__ f32x2 sum_pairs(f32x2 (&t)[kN]) {
#pragma unroll
  for (int d = kN / 2; d > 0; d /= 2)
#pragma unroll
    for (int q = 0; q < d; ++q) t[q] = add2(t[q], t[q + d]);
  return t[0];
}

// A warp's reference and each thread's S and E.
template <bool kEntropy>
struct RowSum;

template <>
struct RowSum<false> {
  Reference x;
  f32x2 s0;
  __device__ __forceinline__ void init(float c) {
    x.none(c, false);
    s0 = 0ull;
  }
  // Before units of maximum um in this lane are added (all lanes call).
  __device__ __forceinline__ void raise(float um) {
    um = warp_max(um);  // NaN compares false below
    if (um > x.m) {
      const float was = x.m, d0 = x.scale;
      x.at(um, x.c, false);
      const float g = was > kNegInf ? d0 * factor(was - um, x.c) / x.scale : 0.f;
      s0 = mul2(s0, pack2(g, g));
    }
  }
  template <typename TIn>
  __device__ __forceinline__ void add_fast(uint32_t (&w)[8]) {  // against a reference that is `fast`
    f32x2 t[Unit<TIn>::kN / 2];
#pragma unroll
    for (int q = 0; q < Unit<TIn>::kN / 2; ++q) t[q] = x.pair_fast(Unit<TIn>::pair(w, q));
    s0 = add2(s0, sum_pairs(t));
  }
  template <typename TIn>
  __device__ __forceinline__ void add(uint32_t (&w)[8]) {
    if (x.fast) {
      add_fast<TIn>(w);
    } else if (x.m > kNegInf) {
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) s0 = add2(s0, x.pair_slow(Unit<TIn>::pair(w, q)));
    }
  }
  __device__ __forceinline__ Moments moments() const {
    float a, b;
    unpack2(s0, a, b);
    return Moments{x.m, (a + b) * x.scale, 0.f};
  }
};

// E counts y = v c - r, short of the true exponent by delta.
template <>
struct RowSum<true> {
  Reference x;
  f32x2 s0, e0;
  __device__ __forceinline__ void init(float c) {
    x.none(c, true);
    s0 = e0 = 0ull;
  }
  __device__ __forceinline__ void raise(float um) {
    um = warp_max(um);
    if (um > x.m) {
      const float was = x.m, d0 = x.delta, z0 = x.scale;
      x.at(um, x.c, true);
      const float g = was > kNegInf ? z0 * factor(was - um, x.c) / x.scale : 0.f;
      if (g > 0.f) {
        const float k = (was - um) * x.c - d0 + x.delta;
        e0 = fma2(s0, pack2(k, k), e0);
      }
      s0 = mul2(s0, pack2(g, g));
      e0 = g > 0.f ? mul2(e0, pack2(g, g)) : 0ull;
    }
  }
  template <typename TIn>
  __device__ __forceinline__ void add_fast(uint32_t (&w)[8]) {
    lift<TIn>(w);
    const f32x2 c2 = pack2(x.c, x.c), r2 = pack2(-x.r, -x.r);
    f32x2 t[Unit<TIn>::kN / 2], e = 0ull;
#pragma unroll
    for (int q = 0; q < Unit<TIn>::kN / 2; ++q) {
      const f32x2 y = fma2(Unit<TIn>::pair(w, q), c2, r2);
      float a, b;
      unpack2(y, a, b);
      t[q] = pack2(ex2(a), ex2(b));
      e = fma2(t[q], y, e);
    }
    s0 = add2(s0, sum_pairs(t));
    e0 = add2(e0, e);
  }
  template <typename TIn>
  __device__ __forceinline__ void add(uint32_t (&w)[8]) {
    if (x.fast) {
      add_fast<TIn>(w);
    } else if (x.m > kNegInf) {
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) {
        float a, b;
        unpack2(Unit<TIn>::pair(w, q), a, b);
        a = rel_log(a, x.m, x.c);
        b = rel_log(b, x.m, x.c);
        const f32x2 t = pack2(ex2(a), ex2(b));
        s0 = add2(s0, t);
        e0 = fma2(t, pack2(a, b), e0);
      }
    }
  }
  __device__ __forceinline__ Moments moments() const {
    float a, b, p, q;
    unpack2(s0, a, b);
    unpack2(e0, p, q);
    const float s = a + b;
    return Moments{x.m, s * x.scale, (p + q - x.delta * s) * x.scale};
  }
};

// A run's stages.  They begin at its first whole unit, so that [0, whole) of them
// lie wholly in the row however it is aligned; what is left (units at the run's
// end, and the row's first unit where it is not whole) makes up the stages [whole,
// all): one, seldom two.
template <typename TIn, int T>
struct Stages {
  typedef Run<TIn, T> R;
  typedef typename R::Stage Stage;
  static constexpr int kBytes = R::kStep * 32;
  int all, whole;
  const char* base;  // this thread's first unit of stage 0
  __device__ __forceinline__ void init(const R& run) {
    all = (run.n + R::kStep - 1) / R::kStep;
    whole = max(run.l - run.f, 0) / R::kStep;
    base = run.base + (run.f + (int)threadIdx.x) * 32;
  }
  // A whole stage.
  template <int kHow>
  __device__ __forceinline__ void load(int s, Stage& w) const {
    const char* p = base + (int64_t)s * kBytes;
#pragma unroll
    for (int k = 0; k < kStage; ++k) load_as<kHow>(p + k * T * 32, w[k]);
  }
  // Unit k of this thread in any stage, -1: none.
  __device__ __forceinline__ static int unit(const R& run, int s, int k) {
    const int v = s * R::kStep + k * T + (int)threadIdx.x;
    return v >= run.n ? -1 : v + run.f < run.n ? v + run.f : 0;
  }
  // The thread that visits a place of the run (Run::place).
  __device__ __forceinline__ static int owner(const R& run, int place) {
    const int v = place / R::kN - run.f;
    return (v >= 0 ? v : run.n - 1) % T;
  }
  // Any stage; units past the run as -inf.
  __device__ __forceinline__ static void load_any(const R& run, int s, Stage& w) {
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const int u = unit(run, s, k);
      if (u >= 0) {
        run.template load<LOAD_PLAIN>(u, w[k]);
      } else {
        const uint32_t none = Elem<TIn>::kBytes == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
        for (int q = 0; q < 8; ++q) w[k][q] = none;
      }
    }
  }
};

// Stages that stay in shared memory between two passes: the last `n` whole ones of
// a run.  A thread reads back what it wrote: [stage][unit][half][thread].
template <int T>
struct Kept {
  uint4* mine;  // this thread's first 16 bytes
  int n;
  typedef uint32_t Stage[kStage][8];
  __device__ __forceinline__ void put(int s, const Stage& v) const {
    uint4* const at = mine + (size_t)s * (kStage * 2 * T);
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      at[2 * k * T] = make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
      at[(2 * k + 1) * T] = make_uint4(v[k][4], v[k][5], v[k][6], v[k][7]);
    }
  }
  __device__ __forceinline__ void get(int s, Stage& v) const {
    const uint4* const at = mine + (size_t)s * (kStage * 2 * T);
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      const uint4 lo = at[2 * k * T], hi = at[(2 * k + 1) * T];
      v[k][0] = lo.x, v[k][1] = lo.y, v[k][2] = lo.z, v[k][3] = lo.w;
      v[k][4] = hi.x, v[k][5] = hi.y, v[k][6] = hi.z, v[k][7] = hi.w;
    }
  }
};

// Adds a run up; `a` holds its first whole stage.  A warp takes the maximum of
// that stage (of the first that holds an entry above -inf) as its reference and adds
// up all that follow against it, without looking for larger ones: for two entries two
// conversions, one multiplication, two exponentials and one addition, and no branch
// but one per stage for a warp that has found no entry yet.  A reference is always an
// entry of the row, so a sum against the largest of them is at least 1.  A sum does
// against a reference below the maximum as long as it stays within kMostSum, and each
// thread's within kThreadSum (an exponent below 64 is rounded to 2^-18, so its term is
// off by up to 1.3e-6; and past 2^126 a sum would count 0 beside a warp whose reference
// lies that far above).  Where it does not, or where there is a NaN, the row is taken
// again, `careful`: with a reference that rises with the maximum and NaNs read as -inf,
// as the row's ends are always taken.  An entropy's E / S is a mean of exponents and
// loses digits to a distant reference (1.4e-6 of H in 1024 x 262144 fp32 with a head at
// 20, 1e-7 with the maximum; 149.6 and 150.2 us): there the reference follows the
// maximum.
constexpr float kMostSum = 1.0995116e12f;    // 2^40
constexpr float kThreadSum = 4.6116860e18f;  // 2^62: with 2^40, 2048 x 128256 at T = 0.3 took 88 us instead of 76
constexpr float kLeastSum = 0.5f;            // below any sum that holds its reference's own 1

template <int kHow, bool kKeep, bool kEntropy, typename TIn, int T>
__device__ __forceinline__ void sum_run(const Run<TIn, T>& run, const Stages<TIn, T>& st, typename Run<TIn, T>::Stage& a,
                                        RowSum<kEntropy>& acc, float c, bool careful, const Kept<T>& kept) {
  typedef typename Run<TIn, T>::Stage Stage;
  acc.init(c);
  Stage b;
#pragma unroll 1
  for (int s = careful ? 0 : st.whole; s < st.all; ++s) {
    st.load_any(run, s, b);
    float um = kNegInf;
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      if (kEntropy || careful) Unit<TIn>::clean(b[k]);  // else a NaN shows: the backward pass has to know of it
      um = fmaxf(um, Unit<TIn>::max(b[k]));
    }
    acc.raise(um);
#pragma unroll
    for (int k = 0; k < kStage; ++k) acc.template add<TIn>(b[k]);
  }
  if (careful || st.whole == 0) return;
  {
    float um = kNegInf;
#pragma unroll
    for (int k = 0; k < kStage; ++k) um = fmaxf(um, Unit<TIn>::max(a[k]));
    acc.raise(um);
  }
  bool fast = acc.x.fast;
  auto add = [&](Stage& v) {
#pragma unroll
    for (int k = 0; k < kStage; ++k) acc.template add_fast<TIn>(v[k]);
  };
  const char* in = st.base;
  int left = st.whole;
  auto step = [&](Stage& v, Stage& w) {
    in += Stages<TIn, T>::kBytes;
    if (left > 1) {
      if (kKeep && left - 1 <= kept.n) {
#pragma unroll
        for (int k = 0; k < kStage; ++k) load_as<LOAD_PLAIN>(in + k * T * 32, w[k]);
      } else {
#pragma unroll
        for (int k = 0; k < kStage; ++k) load_as<kHow>(in + k * T * 32, w[k]);
      }
    }
    if (kKeep && left <= kept.n) kept.put(left - 1, v);
    if (kEntropy || !(acc.x.m > kNegInf)) {
      float um = kNegInf;
#pragma unroll
      for (int k = 0; k < kStage; ++k) um = fmaxf(um, Unit<TIn>::max(v[k]));
      acc.raise(um);
      fast = fast && acc.x.fast;
    }
    add(v);
    return --left > 0;
  };
#pragma unroll 1
  for (;;) {
    if (!step(a, b)) break;
    if (!step(b, a)) break;
  }
  bool most = true;
  if (!kEntropy) {  // each thread's: another warp's reference may hide what is past it
    float lo, hi;
    unpack2(acc.s0, lo, hi);
    most = lo + hi < kThreadSum;
  }
  if (!fast || !most) acc.s0 = pack2(quiet_nan(), quiet_nan());  // asks for a careful pass
}
// Whether a share's sum stands (NaN compares false); one of nothing but -inf does.
__device__ __forceinline__ bool sum_ok(const Moments& r) {
  return (r.s < kMostSum && r.s > kLeastSum) || (r.m == kNegInf && r.s == 0.f);
}

// The block's moments from each warp's maximum and thread's sums, in every
// thread; the order of the sums is fixed.  `red` holds one per warp.
template <int kWarps, bool kEntropy>
__device__ __forceinline__ Moments block_moments(Moments t, float c, Moments* red) {
  t.s = warp_reduce(t.s, OpAddF());
  if (kEntropy) t.e = warp_reduce(t.e, OpAddF());
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  constexpr int kLanes = kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : 16;  // that hold one, again and again over the warp
  static_assert(kWarps <= 16, "");
  const int at = threadIdx.x & (kLanes - 1);
  Moments r = at < kWarps ? red[at] : Moments{kNegInf, 0.f, 0.f};
  r = rebase(r, warp_max(r.m), c);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
    if (kEntropy) r.e += __shfl_xor_sync(0xFFFFFFFFu, r.e, o);
  }
  return r;
}

// The moments of a row whose CTAs have theirs, in the first warp of each; `parts`
// belongs to this CTA, careful becomes whether any of them was.  All threads call.
struct alignas(16) Part {
  Moments m;
  float careful;
};
template <bool kEntropy>
__device__ __forceinline__ void cluster_moments(Moments& r, bool& careful, float c, Part* parts, int C, int rank) {
  const int tid = threadIdx.x, lane = tid & 31;
  cluster_wait();  // every CTA of the cluster runs
  if (tid < C) {
    const uint32_t to = peer_addr(smem_addr(parts + rank), tid);
    peer_store2(to, r.m, r.s);
    peer_store2(to + 8, r.e, careful ? 1.f : 0.f);
  }
  cluster_arrive();
  cluster_wait();
  if (tid >= 32) return;
  const Part p = lane < C ? parts[lane] : Part{{kNegInf, 0.f, 0.f}, 0.f};
  r = rebase(p.m, warp_max(p.m.m), c);
  r.s = warp_reduce(r.s, OpAddF());
  if (kEntropy) r.e = warp_reduce(r.e, OpAddF());
  careful = __any_sync(0xFFFFFFFFu, p.careful != 0.f);
}

// ---------------------------------------------------------------------------
// A row's scalars
// ---------------------------------------------------------------------------
// Whether row i counts, and its token and weight.
__device__ __forceinline__ bool counts(const TokenArgs& a, int64_t i, int32_t& id, float& w) {
  id = a.ids[i];
  w = a.policy.weights ? a.policy.weights[i] : 1.f;
  bool in = id >= 0 && (int64_t)id < a.vocab && w != 0.f;
  if (a.kind == KIND_PREFERENCE) in = in && i >= a.offsets[0] && i < a.offsets[2 * (int64_t)a.pairs];
  return in;
}

__device__ __forceinline__ void skip_row(const TokenArgs& a, int64_t i) {
  if (a.kind != KIND_PREFERENCE) a.out_loss[i] = 0.f;
  if (a.out_entropy) a.out_entropy[i] = 0.f;
  if (a.out_metrics) a.out_metrics[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.out_stats) {
    float4* st = reinterpret_cast<float4*>(a.out_stats + i);
#pragma unroll
    for (int q = 0; q < 3; ++q) st[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// What a row's scalars need beside its moments, loaded before the row is streamed.
struct RowInputs {
  int32_t id;
  float w, x;        // weight, the token's logit (NaN as -inf)
  float A, old, ref; // where the operator has them
};
template <typename TIn>
__device__ __forceinline__ void load_inputs(const TokenArgs& a, int64_t i, RowInputs& in) {  // id and w are known
  const typename Elem<TIn>::Raw* row = static_cast<const typename Elem<TIn>::Raw*>(a.logits) + i * a.row_stride;
  in.x = guard(Elem<TIn>::get(row[in.id]));
  in.A = a.kind == KIND_POLICY ? a.policy.advantages[i] : 0.f;
  in.old = a.policy.old_log_probs ? a.policy.old_log_probs[i] : 0.f;
  in.ref = a.policy.ref_log_probs ? a.policy.ref_log_probs[i] : 0.f;
}

// a - b of two log-probs, 0 where both are -inf.
__device__ __forceinline__ float log_ratio(float a, float b) { return a == kNegInf && b == kNegInf ? 0.f : a - b; }
// RN(a + b); what the rounding lost is added to `lost` (Knuth's two-sum).
__device__ __forceinline__ float two_sum(float a, float b, float& lost) {
  const float s = a + b, v = s - a;
  lost += (a - (s - v)) + (b - v);
  return s;
}

// The loss's slopes and outputs of row i from its moments (one thread; `write`:
// this one stores the outputs).  kKind: the operator where a kernel has only one.
template <bool kEntropy, int kKind = -1>
__device__ __forceinline__ TokenStats finish_row(const TokenArgs& a, int64_t i, const Moments& r, const RowInputs& in,
                                                 bool dirty, bool write = true) {
  const float x = in.x, w = in.w;
  const int kind = kKind >= 0 ? kKind : a.kind;
  TokenStats st;
  float lp, H;
  st.M = r.m;
  // In base-2 exponents, S = 2^k s: lp = ln 2 ((x - M) c - k - log2 s), c the factor
  // that the sum was made with, so that its rounding moves x and S alike (against
  // (x - M) / T it would be a bias of every row).  With what each step loses kept
  // (two-sums, products' remainders): an answer's ratio is a sum of differences of
  // log-probs, in which the rounding of lp itself, up to 1e-6, would be the largest
  // error.  A sum's terms but the maximum's own, 1, are low by kExpLow on average; S
  // holds that 1, but for what it is short of it by rounding.
  const int k = (int)(__float_as_uint(r.s) >> 23 & 255u) - 127;
  const float log2s = log2f(__uint_as_float((__float_as_uint(r.s) & 0x7FFFFFu) | 0x3F800000u));
  const float c = a.c, p = x * c, q = r.m * c;
  float rest = 0.f;  // of lp
  if (fabsf(p) < 1e30f && fabsf(q) < 1e30f) {
    float lo = fmaf(x, c, -p) - fmaf(r.m, c, -q) - kExpLow * kLog2e * fmaxf(1.f - 1.f / r.s, 0.f);
    const float y = two_sum(p, -q, lo), z = two_sum(y, -(float)k, lo), t = two_sum(z, -log2s, lo);
    const float v = kLn2 * t;
    lo = fmaf(kLn2, t, -v) + fmaf(-1.9046543e-9f, t, kLn2 * lo);  // ln 2 less kLn2
    lp = v + lo;
    rest = (v - lp) + lo;
  } else {
    lp = (x == r.m ? 0.f : (x - r.m) / a.temperature) - kLn2 * ((float)k + log2s);
  }
  st.mean = H = quiet_nan();  // a gradient of what was not computed shows
  if (kEntropy) {  // ln 2 (k + log2 s - E / S), put together likewise; E's terms are all low, S's but the 1
    const float over = 1.f / r.s, y = r.e * over;
    float lo = kExpLow * (kLog2e * fmaxf(1.f - over, 0.f) - y * over) - fmaf(-y, r.s, r.e) * over;
    const float z = two_sum((float)k, log2s, lo), t = two_sum(z, -y, lo), v = kLn2 * t;
    st.mean = -kLn2 * y;
    H = v + (fmaf(kLn2, t, -v) + fmaf(-1.9046543e-9f, t, kLn2 * lo));
  }
  if (r.m == kNegInf) {
    lp = H = quiet_nan();
    if (write && a.error_word) atomicOr(a.error_word, LS_ROW_ERR_NO_FINITE);
  }
  st.over = r.m == kNegInf ? quiet_nan() : __frcp_rn(r.s * a.temperature);
  st.id_lp = -expm1f(lp) * a.inv_T;  // 1 - q
  st.id_H = quiet_nan();
  if (kEntropy) st.id_H = lp == kNegInf ? 0.f : expf(lp) * (lp + H) * a.inv_T;
  st.dirty = dirty || kEntropy ? 1.f : 0.f;  // with entropies NaNs go unseen
  st.g_lp = st.g_H = st.term = st.w = st.term_lo = 0.f;
  st.up = kind == KIND_PREFERENCE ? kNoPair : (int32_t)i;
  if (kind == KIND_SCORE) {
    st.g_lp = st.g_H = 1.f;
    a.out_loss[i] = lp;
    if (a.out_entropy) a.out_entropy[i] = H;
  } else if (kind == KIND_POLICY) {
    const ls_policy& p = a.policy;
    const float A = in.A;
    // from lp as it is returned: a policy that has not moved has ratio 1 and KL 0
    const float ratio = p.old_log_probs ? expf(log_ratio(lp, in.old)) : lp == lp ? 1.f : lp;
    float s = 0.f, slope = 0.f;
    if (A != 0.f) {
      const float u = ratio * A, v = fminf(fmaxf(ratio, 1.f - p.clip_low), 1.f + p.clip_high) * A;
      s = u <= v || u != u ? u : v;
      slope = u <= v || u != u ? -u : 0.f;
      if (A < 0.f && p.dual_clip > 0.f && s < p.dual_clip * A) {
        s = p.dual_clip * A;
        slope = 0.f;
      }
    }
    float kl = 0.f, kl_slope = 0.f;
    if (p.ref_log_probs) {
      const float d = -log_ratio(lp, in.ref);
      if (p.kl == LS_KL_K1) {
        kl = -d;
        kl_slope = 1.f;
      } else if (p.kl == LS_KL_K2) {
        kl = 0.5f * d * d;
        kl_slope = -d;
      } else {
        const float g = expm1f(d);
        kl = g < kPosInf ? g - d : g;
        kl_slope = -g;
      }
    }
    float loss = -s;
    if (p.kl_coef != 0.f) {
      loss += p.kl_coef * kl;
      slope += p.kl_coef * kl_slope;
    }
    if (p.entropy_coef != 0.f) loss -= p.entropy_coef * H;
    if (r.m == kNegInf) loss = slope = quiet_nan();  // also where A is 0
    if (write) a.out_loss[i] = w * loss;
    st.g_lp = w * slope;
    st.g_H = p.entropy_coef != 0.f ? -w * p.entropy_coef : 0.f;
    if (write && a.out_metrics) a.out_metrics[i] = make_float4(lp, kEntropy ? H : 0.f, kl, ratio);
  } else if (!kEntropy) {  // a preference loss has no entropies
    st.w = w;
    // w (lp + rest - ref); in.ref is 0 where there is none
    const bool both = a.policy.ref_log_probs && lp == kNegInf && in.ref == kNegInf;
    const float d = both ? 0.f : two_sum(lp, -in.ref, rest);
    st.term = w * d;
    st.term_lo = fabsf(st.term) < kPosInf ? fmaf(w, d, -st.term) + w * rest : 0.f;
  }
  if (write && a.out_stats) {
    float4* out = reinterpret_cast<float4*>(a.out_stats + i);
    out[0] = make_float4(st.M, st.over, st.id_lp, st.id_H);
    out[1] = make_float4(st.g_lp, __int_as_float(st.up), st.g_H, st.mean);
    out[2] = make_float4(st.dirty, st.term, st.w, st.term_lo);
  }
  return st;
}

// ---------------------------------------------------------------------------
// The gradient
// ---------------------------------------------------------------------------
template <bool kV>
struct Bool {
  static constexpr bool value = kV;
};

// d_j = e_j (k0 + k1 y_j), e_j = 2^y_j over x.scale where x is fast, for every
// entry but the token's, which is at_id.
struct RowGradient {
  Reference x;
  float k0, k1;
  float at_id;
  bool lifted;  // with an entropy term, or where the row may hold NaNs: exponents end at kFloorExp
  // g_lp, g_H: the row's slopes times the gradient from above; c = log2(e) / T.
  __device__ __forceinline__ void init(const TokenStats& st, float g_lp, float g_H, float c) {
    lifted = g_H != 0.f || st.dirty != 0.f;
    x.at(st.M, c, false);
    const float over = st.over * x.scale;
    k1 = 0.f;
    k0 = -g_lp * over;
    at_id = g_lp * st.id_lp;
    if (g_H != 0.f) {
      k1 = -g_H * kLn2 * over;
      k0 = -(g_lp + g_H * st.mean) * over - k1 * x.delta;  // pair_fast's y is short of the true one by delta
      at_id -= g_H * st.id_H;
      x.fast = x.fast && fabsf(k1) < 1e30f;  // k1 times any exponent is finite
    }
  }
  // The unit's entries become their gradients, x being fast.
  template <typename TIn, bool kLift>
  __device__ __forceinline__ void apply_fast(uint32_t (&w)[8]) const {
    const f32x2 a0 = pack2(k0, k0), a1 = pack2(k1, k1), c2 = pack2(x.c, x.c), r2 = pack2(-x.r, -x.r);
    uint32_t o[8];
#pragma unroll
    for (int q = 0; q < Unit<TIn>::kN / 2; ++q) {
      float a, b;
      unpack2(fma2(Unit<TIn>::pair(w, q), c2, r2), a, b);
      if (kLift) {
        a = fmaxf(a, kFloorExp);
        b = fmaxf(b, kFloorExp);
      }
      unpack2(mul2(pack2(ex2(a), ex2(b)), kLift ? fma2(pack2(a, b), a1, a0) : a0), a, b);
      Unit<TIn>::set_pair(o, q, a, b);
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = o[q];
  }
  // Any unit.
  template <typename TIn>
  __device__ __forceinline__ void apply(uint32_t (&w)[8]) const {
    Unit<TIn>::clean(w);
    if (x.fast && !lifted) {
      apply_fast<TIn, false>(w);
    } else if (x.fast) {
      apply_fast<TIn, true>(w);
    } else {
      uint32_t o[8];
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) {
        float a, b;
        unpack2(Unit<TIn>::pair(w, q), a, b);
        a = rel_log(a, x.m, x.c);
        b = rel_log(b, x.m, x.c);
        const f32x2 e = pack2(ex2(a), ex2(b));  // first: k1 may be too large for an entry without mass
        unpack2(fma2(mul2(e, pack2(k1, k1)), pack2(a, b), mul2(e, pack2(k0, k0))), a, b);
        Unit<TIn>::set_pair(o, q, a, b);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q] = o[q];
    }
  }
};

// Writes a run's gradients but the token's, from its first stage to its last or
// (kBack) the other way; `a` holds the first of the whole ones that are not kept.
template <bool kBack, bool kLift, typename TIn, int T>
__device__ __forceinline__ void gradient_sweep(const Stages<TIn, T>& st, typename Run<TIn, T>::Stage& a,
                                               const RowGradient& g, char* out, const Kept<T>& kept) {
  typedef typename Run<TIn, T>::Stage Stage;
  constexpr int kBytes = kBack ? -Stages<TIn, T>::kBytes : Stages<TIn, T>::kBytes;
  const int64_t first = (int64_t)(kBack ? st.whole - 1 : 0) * Stages<TIn, T>::kBytes;
  out += first;
  Stage b;
  int held = 0;
  if (kBack) {
    held = min(kept.n, st.whole);
#pragma unroll 1
    for (int s = 0; s < held; ++s) {
      kept.get(s, b);
#pragma unroll
      for (int k = 0; k < kStage; ++k) {
        g.template apply_fast<TIn, kLift>(b[k]);
        store32(out + k * T * 32, b[k]);
      }
      out += kBytes;
    }
  }
  const char* in = st.base + (first + (int64_t)held * kBytes);
  int left = st.whole - held;
  auto step = [&](Stage& v, Stage& w) {
    in += kBytes;
    if (left > 1) {
#pragma unroll
      for (int k = 0; k < kStage; ++k) load_as<LOAD_PLAIN>(in + k * T * 32, w[k]);
    }
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      g.template apply_fast<TIn, kLift>(v[k]);
      store32(out + k * T * 32, v[k]);
    }
    out += kBytes;
    return --left > 0;
  };
#pragma unroll 1
  while (left > 0) {
    if (!step(a, b)) break;
    step(b, a);
  }
}
template <bool kBack, typename TIn, int T>
__device__ __forceinline__ void gradient_run(const Run<TIn, T>& run, const Stages<TIn, T>& st,
                                             typename Run<TIn, T>::Stage& a, const RowGradient& shared,
                                             typename Elem<TIn>::Raw* grad, const Kept<T>& kept) {
  const RowGradient g = shared;
  const bool same = run.aligned_with(grad), slow = !g.x.fast || !same;
  // what the whole stages leave; all of a row that is not aligned with its gradient or far from fp32's range
#pragma unroll 1
  for (int s = slow ? 0 : st.whole; s < st.all; ++s) {
    typename Run<TIn, T>::Stage v;
    st.load_any(run, s, v);
#pragma unroll
    for (int k = 0; k < kStage; ++k) {
      g.template apply<TIn>(v[k]);
      const int u = st.unit(run, s, k);
      if (u >= 0) run.store(grad, same, u, v[k]);
    }
  }
  if (slow) return;
  char* const out = reinterpret_cast<char*>(grad + run.j0) + (run.f + (int)threadIdx.x) * 32;
  if (g.lifted)
    gradient_sweep<kBack, true>(st, a, g, out, kept);
  else
    gradient_sweep<kBack, false>(st, a, g, out, kept);
}

// ls_token_grad.cu: loss and gradient from one call.
ls_status token_grad(const TokenArgs& a, ls_dtype dtype, bool entropy, cudaStream_t st);

}  // namespace ops
}  // namespace lsg
