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
  float M, S, H, lp;      // maximum, sum exp((x - M) / T), entropy, log-prob of the token
  float g_lp, g_H;        // the loss's slopes; both 0: the row does not count
  int32_t up;             // the entry of the gradient from above that belongs to the row
  float term;             // preference: weight * (lp - ref)
  float w;                // preference: the weight of a row that counts
  float pad[23];
};
static_assert(sizeof(TokenStats) == sizeof(float) * LS_TOKEN_STATS, "the header's size of a row's stats");

enum TokenKind { KIND_SCORE, KIND_POLICY, KIND_PREFERENCE };

struct TokenArgs {
  const void* logits;
  int64_t vocab, row_stride;
  int32_t n;
  const int32_t* ids;
  float temperature;
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
// (M, S, E) of a set of entries: S = sum 2^y, E = sum y 2^y, y = (x - M) c <= 0,
// c = log2(e) / T.  H = ln S - ln 2 * E / S.
struct Moments {
  float m, s, e;
};

// The same set against a maximum m >= a.m.  A NaN in a.s stays one.
__device__ __forceinline__ Moments rebase(const Moments& a, float m, float c) {
  if (!(a.m > kNegInf)) return Moments{m, a.s, a.e};
  const float f = rel_exp(a.m, m, c);
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

// A warp's running maximum and each thread's S and E (as OnlineSum; the E of a
// fast maximum counts y = v c - r, short of the true one by delta = m c - r).
template <bool kEntropy>
struct RowSum;

template <>
struct RowSum<false> : OnlineSum {
  __device__ __forceinline__ Moments moments() const { return Moments{x.m, sum(), 0.f}; }
};

template <>
struct RowSum<true> {
  ExpAgainst x;
  float delta;
  f32x2 s0, s1, e0;
  __device__ __forceinline__ void against(float m, float c) {
    x.init(m, c);
    x.fast = x.fast && lift_ok(c);
    if (!x.fast) x.scale = 1.f;
    delta = x.fast ? fmaf(m, c, -x.r) : 0.f;
  }
  __device__ __forceinline__ void init(float c) {
    against(kNegInf, c);
    s0 = s1 = e0 = 0ull;
  }
  __device__ __forceinline__ void raise(float um) {
    um = warp_max(um);
    if (um > x.m) {
      const float was = x.m, d0 = delta, f = was > kNegInf ? x.scale * rel_exp(was, um, x.c) : 0.f;
      against(um, x.c);
      const float g = f / x.scale;
      if (g > 0.f) {
        const float k = (was - um) * x.c - d0 + delta;
        e0 = fma2(add2(s0, s1), pack2(k, k), e0);
      }
      s0 = mul2(s0, pack2(g, g));
      s1 = mul2(s1, pack2(g, g));
      e0 = g > 0.f ? mul2(e0, pack2(g, g)) : 0ull;
    }
  }
  template <typename TIn>
  __device__ __forceinline__ void add(uint32_t (&w)[8]) {
    if (x.fast) {
      lift<TIn>(w);
      const f32x2 c2 = pack2(x.c, x.c), r2 = pack2(-x.r, -x.r);
#pragma unroll
      for (int q = 0; q < Unit<TIn>::kN / 2; ++q) {
        const f32x2 y = fma2(Unit<TIn>::pair(w, q), c2, r2);
        float a, b;
        unpack2(y, a, b);
        const f32x2 t = pack2(ex2(a), ex2(b));
        if (q & 1)
          s1 = add2(s1, t);
        else
          s0 = add2(s0, t);
        e0 = fma2(t, y, e0);
      }
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
    unpack2(add2(s0, s1), a, b);
    unpack2(e0, p, q);
    const float s = a + b;
    return Moments{x.m, s * x.scale, (p + q - delta * s) * x.scale};
  }
};

// The block's moments from each warp's maximum and thread's sums, in every
// thread; the order of the sums is fixed.  `red` holds one per warp.
template <int kWarps, bool kEntropy>
__device__ __forceinline__ Moments block_moments(Moments t, float c, Moments* red) {
  t.s = warp_reduce(t.s, OpAddF());
  if (kEntropy) t.e = warp_reduce(t.e, OpAddF());
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = t;
  __syncthreads();
  Moments r = red[threadIdx.x & (kWarps - 1)];
  r = rebase(r, warp_max(r.m), c);
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
    if (kEntropy) r.e += __shfl_xor_sync(0xFFFFFFFFu, r.e, o);
  }
  return r;
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

// a - b of two log-probs, 0 where both are -inf.
__device__ __forceinline__ float log_ratio(float a, float b) { return a == kNegInf && b == kNegInf ? 0.f : a - b; }

// The loss's slopes and outputs of row i from its moments and its token's logit
// (one thread).
__device__ __forceinline__ TokenStats finish_row(const TokenArgs& a, int64_t i, const Moments& r, float x, float w,
                                                 bool entropy) {
  TokenStats st;
  st.M = r.m;
  st.S = r.s;
  const float lnS = logf(r.s);
  st.H = entropy ? lnS - kLn2 * (r.e / r.s) : quiet_nan();  // a gradient of what was not computed shows
  st.lp = (x == r.m ? 0.f : (x - r.m) / a.temperature) - lnS;
  if (r.m == kNegInf) {
    st.lp = quiet_nan();
    st.H = quiet_nan();
    if (a.error_word) atomicOr(a.error_word, LS_ROW_ERR_NO_FINITE);
  }
  st.g_lp = st.g_H = st.term = st.w = 0.f;
  st.up = (int32_t)i;
  if (a.kind == KIND_SCORE) {
    st.g_lp = st.g_H = 1.f;
    a.out_loss[i] = st.lp;
    if (a.out_entropy) a.out_entropy[i] = st.H;
  } else if (a.kind == KIND_POLICY) {
    const ls_policy& p = a.policy;
    const float A = p.advantages[i];
    const float ratio = p.old_log_probs ? expf(log_ratio(st.lp, p.old_log_probs[i])) : st.lp == st.lp ? 1.f : st.lp;
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
      const float d = log_ratio(p.ref_log_probs[i], st.lp);
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
    if (p.entropy_coef != 0.f) loss -= p.entropy_coef * st.H;
    if (r.m == kNegInf) loss = slope = quiet_nan();  // also where A is 0
    a.out_loss[i] = w * loss;
    st.g_lp = w * slope;
    st.g_H = p.entropy_coef != 0.f ? -w * p.entropy_coef : 0.f;
    if (a.out_metrics) a.out_metrics[i] = make_float4(st.lp, entropy ? st.H : 0.f, kl, ratio);
  } else {
    st.w = w;
    st.term = w * (a.policy.ref_log_probs ? log_ratio(st.lp, a.policy.ref_log_probs[i]) : st.lp);
  }
  if (a.out_stats) {
    float4* out = reinterpret_cast<float4*>(a.out_stats + i);
    out[0] = make_float4(st.M, st.S, st.H, st.lp);
    out[1] = make_float4(st.g_lp, st.g_H, __int_as_float(st.up), st.term);
    out[2] = make_float4(st.w, 0.f, 0.f, 0.f);
  }
  return st;
}

// ---------------------------------------------------------------------------
// The gradient of a unit
// ---------------------------------------------------------------------------
// d_j = e_j (k0 + k1 y_j), e_j = 2^y_j over x.scale where x is fast.
struct RowGradient {
  ExpAgainst x;
  float k0, k1;
  float at_id;  // the token's entry
  bool entropy;
  // g_lp, g_H: the row's slopes times the gradient from above.
  __device__ __forceinline__ void init(const TokenStats& st, float g_lp, float g_H, float T) {
    const float c = kLog2e / T;
    x.init(st.M, c);
    entropy = g_H != 0.f;
    if (entropy && !lift_ok(c)) {
      x.fast = false;
      x.scale = 1.f;
    }
    const float lnS = logf(st.S), over = x.scale / (st.S * T);
    k1 = entropy ? -g_H * kLn2 * over : 0.f;
    k0 = -(g_lp + (entropy ? g_H * (st.H - lnS) : 0.f)) * over;
    if (entropy && x.fast) k0 -= k1 * fmaf(st.M, c, -x.r);  // pair_fast's y is short of the true one by this
    const float q = expf(st.lp);
    at_id = g_lp * -expm1f(st.lp);  // 1 - q
    if (entropy && q > 0.f) at_id -= g_H * q * (st.lp + st.H);
    at_id /= T;
    if (st.M == kNegInf) k0 = quiet_nan();
  }
  // The unit's entries become their gradients; `at`: the token's place in it, kN and above: none.
  template <typename TIn>
  __device__ __forceinline__ void apply(uint32_t (&w)[8], uint32_t at) const {
    constexpr int kN = Unit<TIn>::kN;
    const f32x2 a0 = pack2(k0, k0);
    uint32_t o[8];
    if (x.fast && !entropy) {
      Unit<TIn>::clean(w);
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) {
        float a, b;
        unpack2(mul2(x.pair_fast(Unit<TIn>::pair(w, q)), a0), a, b);
        Unit<TIn>::set_pair(o, q, a, b);
      }
    } else if (x.fast) {
      lift<TIn>(w);
      const f32x2 a1 = pack2(k1, k1), c2 = pack2(x.c, x.c), r2 = pack2(-x.r, -x.r);
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) {
        const f32x2 y = fma2(Unit<TIn>::pair(w, q), c2, r2);
        float a, b;
        unpack2(y, a, b);
        unpack2(mul2(pack2(ex2(a), ex2(b)), fma2(y, a1, a0)), a, b);
        Unit<TIn>::set_pair(o, q, a, b);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) {
        float a, b;
        unpack2(Unit<TIn>::pair(w, q), a, b);
        a = rel_log(a, x.m, x.c);
        b = rel_log(b, x.m, x.c);
        Unit<TIn>::set_pair(o, q, ex2(a) * fmaf(a, k1, k0), ex2(b) * fmaf(b, k1, k0));
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = o[q];
    if (at < (uint32_t)kN) {
#pragma unroll
      for (int q = 0; q < kN / 2; ++q) {
        float a = Unit<TIn>::kN == 16 ? __uint_as_float(w[q] << 16) : __uint_as_float(w[2 * q & 7]);
        float b = Unit<TIn>::kN == 16 ? __uint_as_float(w[q] & 0xFFFF0000u) : __uint_as_float(w[(2 * q + 1) & 7]);
        if ((int)(at >> 1) == q) {
          if (at & 1)
            b = at_id;
          else
            a = at_id;
        }
        Unit<TIn>::set_pair(w, q, a, b);
      }
    }
  }
};

}  // namespace ops
}  // namespace lsg
