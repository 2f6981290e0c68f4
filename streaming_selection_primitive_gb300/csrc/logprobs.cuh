// A row of logits under the softmax: running maximum and sums of one pass (logprobs.cu),
// their joins, and what the losses make of a row.
#pragma once

#include "lm.cuh"
#include "lm.h"

namespace profk {

using Pair = unsigned long long;  // two floats, low half first

__device__ __forceinline__ Pair pair(float a, float b) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void split(Pair p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Below this, 2^x is zero in float32 whatever it is; as the smallest exponent it keeps
// x 2^x from becoming inf * 0 where a logit is -inf.
constexpr float NO_MASS = -300.f;

// The exponents of a row: x = (l - m) c for a largest logit m, c = log2(e) / T.  Where m c is of
// ordinary size they are taken as one fused product, l c - (m c rounded): off the definition
// by the same r = m c - (m c rounded) for every l of the row, |r| <= 2^-5, which the row's sums are
// freed of at the end (centred).  Otherwise, where r could be anything or m c overflow, as the difference first.
struct Centre {
  float m, c, by;  // by: -(m c rounded), or -m
  bool fused;
  __device__ __forceinline__ Centre(float largest, float c_) : m(largest), c(c_) {
    if (m == -INFINITY) m = 0.f;  // (any finite number while there is nothing)
    const float mc = m * c;
    fused = fabsf(mc) < 1048576.f;
    by = fused ? -mc : -m;
  }
  __device__ __forceinline__ float operator()(float l) const { return fused ? fmaf(l, c, by) : (l + by) * c; }
  // r: what the fused exponents are too large by.
  __device__ __forceinline__ float off() const { return fused ? fmaf(m, c, by) : 0.f; }
};

// What has been seen of a row: its largest logit m, s = sum 2^x and t = sum x 2^x by
// m's centre.  A NaN or +inf logit makes s NaN (inf - inf), and it stays so; s = 0 says that
// nothing but -inf came.  The sums of a long row have millions of terms a thread: what an
// addition loses is carried along in a second float.
struct Running {
  float m, s, t, s_lost, t_lost;
};

// sum + v exactly, as a float and what it lost.
__device__ __forceinline__ void add_exact(float& sum, float& lost, float v) {
  const float r = sum + v, back = r - sum;
  lost += (sum - (r - back)) + (v - back);
  sum = r;
}

// The exponent by which sums by the centre of `from` shrink when taken by that of `to`: what each has besides (m c
// exactly) counts too, where only one of them is fused.
// (fmaxf gives NO_MASS where it is NaN, at infinite ones: what is NaN already stays it, what is zero too.)
__device__ __forceinline__ float shrink(float from, float to, float c) {
  const Centre a(from, c), b(to, c);
  return fmaxf(from == -INFINITY ? NO_MASS : a.fused && b.fused ? b.by - a.by : (a.m - b.m) * c + (b.off() - a.off()), NO_MASS);
}

// Row results that the kernels exchange (and the logit of the row's token with them, where they do).
struct alignas(16) RowSum {
  float m, s, t, logit;
};

__device__ __forceinline__ RowSum total(const Running& r) { return {r.m, r.s + r.s_lost, r.t + r.t_lost, 0.f}; }

// Sums by the centre of m as sums by m itself (to which m's own logit gives 1, whatever was rounded).
__device__ __forceinline__ RowSum centred(const RowSum& y, float c) {
  const float r = Centre(y.m, c).off(), f = lm_exp2(-r);
  const float s = f * y.s;
  return {y.m, s > 0.f && s < 1.f ? 1.f : s, f * (y.t - r * y.s), 0.f};
}

// Joins over the warp: all lanes get the same, in the same order every time.
template <bool ENTROPY>
__device__ __forceinline__ RowSum warp_join(RowSum r, float c) {
  const float m = warp_max(r.m);
  const float d = shrink(r.m, m, c), f = lm_exp2(d);
  const float s = warp_sum(r.s * f);
  const float t = ENTROPY ? warp_sum(f * (r.t + d * r.s)) : 0.f;
  return {m, s, t, 0.f};
}

// Two parts of a row as one.
__device__ __forceinline__ RowSum joined(const RowSum& y, const RowSum& z, float c) {
  const float m = fmaxf(y.m, z.m), dy = shrink(y.m, m, c), dz = shrink(z.m, m, c);
  const float fy = lm_exp2(dy), fz = lm_exp2(dz);
  return {m, fy * y.s + fz * z.s, fy * (y.t + dy * y.s) + fz * (z.t + dz * z.s), 0.f};
}

// ln s as a float and what it lacks, for s >= 1: from s = 2^k f with f in [1, 2), whose logarithm is off by less
// than that of s (2^-25 of at most 0.7, not of 20).  ln 2 is split as Cody and Waite do (Software Manual for the
// Elementary Functions, 1980): k times its head, 15 bits, is exact.
__device__ __forceinline__ float log_exactly(float s, float& lacks) {
  const int bits = __float_as_int(s), k = (bits >> 23) - 127;
  const float f = __int_as_float((bits & 0x7fffff) | 0x3f800000);
  constexpr float HEAD = 0.693145751953125f, REST = 1.42860682030941723e-6f;  // ln 2 = HEAD + REST
  const float a = k * HEAD, b = logf(f), y = a + b, back = y - a;
  lacks = ((a - (y - back)) + (b - back)) + k * REST;
  return y;
}

// A token's log-probability from its logit and the row's sums, and what the float lacks (sums over a
// sequence take it along): -inf where the row holds nothing, NaN where it holds a NaN or +inf.
__device__ __forceinline__ float row_logprob(const RowSum& r, float logit, float T, float& lacks) {
  lacks = 0.f;
  if (r.s == 0.f) return -INFINITY;
  if (!(r.s < INFINITY)) return NAN;
  float of_log;
  const float a = logit - r.m, x = a / T, L = log_exactly(r.s, of_log);
  const float y = x - L;
  if (!(fabsf(y) < INFINITY)) return y;
  const float back = y - x;
  const float of_x = fabsf(x) > 0x1p-100f ? fmaf(-x, T, a) / T : 0.f;
  lacks = ((x - (y - back)) + (-L - back)) + (of_x - of_log);
  const float z = y + lacks;
  lacks += y - z;
  return z;
}
__device__ __forceinline__ float row_logprob(const RowSum& r, float logit, float T) {
  float lacks;
  return row_logprob(r, logit, T, lacks);
}

// log s - (sum x exp x) / s; 0 for a row that holds nothing.
__device__ __forceinline__ float row_entropy(const RowSum& r) {
  const float H = logf(r.s) - r.t * LN2 / r.s;
  return r.s == 0.f || H < 0.f ? 0.f : H;  // (below it only by rounding)
}

// log2(e) / T; NaN where T is no positive number, or so near to zero (or infinity) that
// this is none.
__device__ __forceinline__ float inverse_temperature(float T) {
  const float c = LOG2E / T;
  return c > 0.f && c < INFINITY ? c : NAN;
}

// exp(q) - 1 - q, e = expm1(q): never below 0.  Near 0, where the difference is e's rounding (and of either sign), by its series:
// the first term left out is 2^-26 of it at the border, where the difference is off by 2^-20 of itself at most.
__device__ __forceinline__ float exp_beyond_line(float q, float e) {
  if (fabsf(q) < 0.25f)
    return q * q * fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, 1.f / 5040, 1.f / 720), 1.f / 120), 1.f / 24), 1.f / 6), 0.5f);
  return e == INFINITY ? e : e - q;
}

// One token's part of the clipped policy loss, by its log-probability.
struct PolicyTerm {
  float loss;     // without the entropy
  float kl;       // exp(q) - 1 - q, q = reference - log-probability
  bool clipped;   // the clipped ratio is what counts: no gradient of the ratio
  float slope;    // d loss / d log-probability
};

__device__ __forceinline__ PolicyTerm policy_term(float lp, float old_lp, float A, bool with_ref, float ref_lp,
                                                  const PolicyHow& how) {
  PolicyTerm y;
  const float ratio = expf(lp - old_lp), low = 1.f - how.clip_low, high = 1.f + how.clip_high;
  y.clipped = (A > 0.f && ratio > high) || (A < 0.f && ratio < low);
  // A ratio that is not a number, or an infinite one times nothing, shows in the loss.
  y.loss = y.clipped ? -A * (A > 0.f ? high : low) : -A * ratio;
  y.slope = y.clipped ? 0.f : -A * ratio;
  y.kl = 0.f;
  if (with_ref) {
    const float q = ref_lp - lp, e = expm1f(q);
    y.kl = exp_beyond_line(q, e);
    if (how.kl != 0.f) {
      y.loss += how.kl * y.kl;
      y.slope -= how.kl * e;
    }
  }
  return y;
}

}  // namespace profk
