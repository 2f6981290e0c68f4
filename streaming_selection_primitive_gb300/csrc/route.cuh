// Choice of each token's experts, and its gradient: the kernels, for route.cu (bias
// added to the logits, and the gradient) and route_scores.cu (bias added to the
// scores), which are compiled side by side.
//
// A token t has one logit z_e per expert.  With y = z (softmax scores) or
// y = log sigmoid(z) (sigmoid scores), p = softmax(y) over the experts.  The
// choice is the first k experts in the library order of c = z + bias, or of
// c = score + bias (SCORES; the score is p or sigmoid z), descending, ties by
// lower index, -inf and NaN never.  Gates: over the
// chosen, softmax(y) when normalized, else p (softmax) or sigmoid(z).  Balance
// loss:
//   loss = E sum_e (counts_e / N) P_e,  P_e = sum_t n_t p_te / N,
// counts_e the slots given to expert e, n_t those token t filled, N = sum n_t.
//
// One warp takes a token: R = E / 32 logits a lane (rounded up to a power of
// two), in registers, read once.  The choice runs on 32-bit keys that end in
// the expert's index (sort_key), so that a round is one warp-wide maximum.
//
// What bounds it (several sets of inputs in turn, beyond L2):
//   256 experts of float32: a token's instructions, 551 forward and 438 backward, of
//     which the SMs issue 3.2 and 2.8 a cycle of 4.  131072 tokens, k = 8: 79 us
//     forward (147 MB, 1.9 TB/s) and 69 backward (281 MB, 4.1 TB/s);
//   128 of bfloat16: 344 and 271 instructions, 2.5 and 2.0 a cycle (2.8 and 2.6 with
//     the inputs in L2): a token begins with its load, which the other warps do not
//     hide in full, and the backward pass with its choice and gates too.  32768
//     tokens: 20 and 16 us, 12 for a backward pass that finds the logits in L2;
//   few tokens: the launches, one token's chain of rounds and exchanges, and the
//     join of the CTAs' sums.  4096 of 64 take 7.7 and 3.5 us, 16 of 128 take 4.4
//     with the loss, 3.4 without, and 3.2 backward.
#pragma once

#include <type_traits>

#include <cooperative_groups.h>

#include "../../include/profk.h"
#include "lm.cuh"
#include "lm.h"

namespace cg = cooperative_groups;

namespace profk {
namespace {

constexpr int CLUSTER = 8;  // CTAs of the one-launch form and of the join

// Warps of a CTA, and resident CTAs per SM of the forms for many tokens (which
// size their grids): what the registers of R values a lane allow.  (131072 x 256
// float32, forward and backward: 79 and 69 us; with one CTA an SM 86 and 97, with
// eight warps a CTA 90 and 97.)
template <int R>
constexpr int WARPS = R <= 16 ? 16 : 8;
template <int R>
constexpr int PER_SM = R <= 8 ? 2 : 1;

// ---------------------------------------------------------------------------
// A lane's part of a token: R values, VEC consecutive ones at a time.
template <typename T, int R>
struct Part {
  static constexpr int VEC = R < 16 / int(sizeof(T)) ? R : 16 / int(sizeof(T));
  static __device__ __forceinline__ int expert(int r) { return ((r / VEC) * 32 + (threadIdx.x & 31)) * VEC + r % VEC; }
};

template <int BYTES>
struct Bits;
template <>
struct Bits<2> { using type = unsigned short; };
template <>
struct Bits<4> { using type = unsigned; };
template <>
struct Bits<8> { using type = uint2; };
template <>
struct Bits<16> { using type = uint4; };

// The lane's logits of one token, -inf beyond E.  vec: the row starts on a
// boundary of VEC values, so a whole group is one load.
template <typename T, int R>
__device__ __forceinline__ void load_part(const T* row, int E, bool vec, float (&z)[R]) {
  using P = Part<T, R>;
#pragma unroll
  for (int g = 0; g < R; g += P::VEC) {
    const int e = P::expert(g);
    if (vec && e + P::VEC <= E) {
      union {
        typename Bits<P::VEC * sizeof(T)>::type bits;
        T v[P::VEC];
      } u;
      u.bits = *reinterpret_cast<const decltype(u.bits)*>(row + e);
#pragma unroll
      for (int j = 0; j < P::VEC; ++j) z[g + j] = lm_float(u.v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < P::VEC; ++j) z[g + j] = e + j < E ? lm_float(row[e + j]) : -INFINITY;
    }
  }
}

// The lane's part, laid out as for T, of 32 R floats in shared memory.
template <typename T, int R>
__device__ __forceinline__ void load_shared(const float* from, float (&z)[R]) {
  using P = Part<T, R>;
  constexpr int V = P::VEC < 4 ? P::VEC : 4;
#pragma unroll
  for (int g = 0; g < R; g += V) {
    union {
      typename Bits<4 * V>::type bits;
      float v[V];
    } u;
    u.bits = *reinterpret_cast<const decltype(u.bits)*>(from + P::expert(g));
#pragma unroll
    for (int j = 0; j < V; ++j) z[g + j] = u.v[j];
  }
}

template <typename T, int R>
__device__ __forceinline__ void store_part(T* row, int E, bool vec, const float (&d)[R]) {
  using P = Part<T, R>;
#pragma unroll
  for (int g = 0; g < R; g += P::VEC) {
    const int e = P::expert(g);
    if (vec && e + P::VEC <= E) {
      union {
        typename Bits<P::VEC * sizeof(T)>::type bits;
        T v[P::VEC];
      } u;
#pragma unroll
      for (int j = 0; j < P::VEC; ++j) u.v[j] = lm_cast<T>(d[g + j]);
      *reinterpret_cast<decltype(u.bits)*>(row + e) = u.bits;
    } else {
#pragma unroll
      for (int j = 0; j < P::VEC; ++j)
        if (e + j < E) row[e + j] = lm_cast<T>(d[g + j]);
    }
  }
}

// A warp's ring of STAGES token rows in shared memory, filled by asynchronous
// copies: each lane copies what it reads itself, so that the next tokens'
// rows are on their way while one is worked on, without holding registers.
// Taken for rows of 1 to 2 KB whose groups of VEC values are whole and aligned
// (32768 x 512 bfloat16: 45.5 us forward and 32.8 backward, against 49.5 and 41.3
// with plain loads; 131072 x 256 float32 79.0 and 69.1, against 77.0 and 69.5).
// Shorter ones are loaded when their turn comes (32768 x 128 bfloat16: 20.0 and 16.4
// us, against 21.3 and 15.5 through a ring); longer ones would need more shared
// memory than there is.
template <typename T, int R>
struct Ring {
  using P = Part<T, R>;
  static constexpr int CHUNK = P::VEC * int(sizeof(T));
  static constexpr int ROW = 32 * R * int(sizeof(T));
  static constexpr int STAGES = ROW < 1024 || ROW > 2048 ? 0 : ROW > 1024 ? 2 : 4;
  static constexpr int BYTES = STAGES * ROW;  // per warp
  unsigned char* base;  // this warp's
  bool on;

  __device__ __forceinline__ Ring(unsigned char* smem, bool vec, int E) {
    base = smem + (threadIdx.x >> 5) * BYTES;
    on = STAGES > 0 && vec && E % P::VEC == 0;
  }
  // Starts the copy of a row (none: an empty group) into stage `at`.
  __device__ __forceinline__ void fetch(const T* row, int E, bool some, int at) const {
    if constexpr (STAGES > 0) {
      if (!on) return;
      if (some) {
#pragma unroll
        for (int g = 0; g < R; g += P::VEC) {
          const int e = P::expert(g);
          if (e < E) {
            const unsigned to = static_cast<unsigned>(__cvta_generic_to_shared(base + at * ROW + e * int(sizeof(T))));
            if constexpr (CHUNK == 16)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row + e) : "memory");
            else
              asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(row + e), "n"(CHUNK) : "memory");
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  // Waits until the oldest of the rows under way has arrived.
  __device__ __forceinline__ void wait() const {
    if constexpr (STAGES > 0)
      if (on) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();
      }
  }
  // Where the token's row can be read now.
  __device__ __forceinline__ const T* row(const T* global, int at) const {
    return on ? reinterpret_cast<const T*>(base + at * ROW) : global;
  }
};

// ---------------------------------------------------------------------------
// Scores.

// log sigmoid(z), exact for large |z|.
__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

__device__ __forceinline__ float sigmoid(float z) { return lm_rcp(1.f + lm_exp2(-LOG2E * z)); }

// The token's p, unnormalized, into s; returns the sum over the warp.  `ref`
// is the largest logit for softmax, any logit of the token for sigmoid.
// Softmax: s = exp(z - ref).  Sigmoid: s = sigmoid(z), or, where that could
// underflow for every expert (ref below -60) or a value is not finite, the
// careful form: s = sigmoid(z) exp(-c) with c = min(max z, 0).
template <bool SIG, int R>
__device__ __forceinline__ float token_scores(const float (&z)[R], float (&s)[R], float ref) {
  float sum = 0.f;
  if (SIG && ref > -60.f) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = sigmoid(z[r]);
  } else if (!SIG && fabsf(ref) < INFINITY) {
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = lm_exp2((z[r] - ref) * LOG2E);
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < R; ++r) m = fmaxf(m, z[r]);
    m = warp_max(m);
    const float c = fminf(m, 0.f), ec = expf(c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if constexpr (SIG) {
        const bool pos = z[r] >= 0.f;
        const float u = z[r] == -INFINITY ? 0.f : expf(pos ? -z[r] : z[r] - c);
        s[r] = (pos ? 1.f : u) / (1.f + (pos ? u : u * ec));
      } else {
        s[r] = z[r] == m ? 1.f : expf(z[r] - m);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) sum += s[r];
  return warp_sum(sum);
}

// Sum over lanes 0 .. width - 1 (a power of two; the others hold 0), in each of them.
__device__ __forceinline__ float slots_sum(float v, int width) {
  for (int d = width >> 1; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

// The gate of the lane's slot (logit zc; ok: the slot is filled).  ref: the
// token's largest logit (sigmoid: unused); sum: of its experts' scores.  width: the power of two not
// below k.
template <bool SIG>
__device__ __forceinline__ float slot_gate(float zc, bool ok, int width, bool normalize, float ref, float sum) {
  float e = SIG ? sigmoid(zc) : zc == ref ? 1.f : lm_exp2((zc - ref) * LOG2E);
  e = ok ? e : 0.f;
  if (!normalize) return SIG ? e : e * lm_rcp(sum);
  float all = slots_sum(e, width);
  const float first = __shfl_sync(FULL_MASK, all, 0);
  if (!(first > 1e-20f)) {
    // The chosen are far below the largest (a bias chose them), or underflow:
    // by their logarithms.
    const float y = ok ? (SIG ? log_sigmoid(zc) : zc) : -INFINITY;
    const float top = key_to_float(__reduce_max_sync(FULL_MASK, ord_key(y)));
    e = ok ? (y == top ? 1.f : lm_exp2((y - top) * LOG2E)) : 0.f;
    all = slots_sum(e, width);
  }
  return ok ? e * lm_rcp(all) : 0.f;
}

// ---------------------------------------------------------------------------
// The choice.

// Key of an expert that sorts like (c descending, index ascending): ord(c)
// with its low bits (as many as index the 32 R experts) replaced by the
// inverted index.  For bf16 and f16 logits without a bias those bits carry
// nothing, so the order is exact; for float32 sums two experts whose c agree
// in the remaining 22 to 27 bits may come in the wrong order, which the
// caller checks.  c is a sum, so it is no -0 (the bias is +0 where there is
// none) and a NaN is the positive one, whose key is above that of +inf.
// Below AVAILABLE: -inf, also where there is no expert.
constexpr uint32_t AVAILABLE = 0x00800000u;  // ord of the lowest finite value

template <int R>
__device__ __forceinline__ uint32_t sort_key(float c, int e) {
  const int b = __float_as_int(c);
  const uint32_t ord = static_cast<uint32_t>(b ^ ((b >> 31) | int(0x80000000)));
  return (ord | (32u * R - 1u)) ^ static_cast<uint32_t>(e);
}

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// What the choice is made by: z + bias, or score + bias for every expert whose
// logit is above -inf (SCORES).  A NaN logit's is NaN, and the others' scores are
// those of a token without it.  (131072 x 256 float32, k = 8, sigmoid, without the
// loss: 69 us by logits and 75 by scores; 32768 x 128 bfloat16, softmax: 19.3 and
// 21.8.  Kernels of their own, so that the choice by logits does not pay for it.)
template <bool SIG, bool SCORES, int R>
__device__ __forceinline__ void choose_by(const float (&z)[R], const float (&bias)[R], float (&c)[R]) {
  if constexpr (!SCORES) {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = z[r] + bias[r];
  } else if constexpr (SIG) {
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = z[r] == -INFINITY ? z[r] : sigmoid(z[r]) + bias[r];
  } else {
    float m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) m = fmaxf(m, z[r]);
    m = warp_max(m);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c[r] = z[r] == m ? 1.f : lm_exp2((z[r] - m) * LOG2E);
      sum += c[r] == c[r] ? c[r] : 0.f;
    }
    const float inv = lm_rcp(warp_sum(sum));
#pragma unroll
    for (int r = 0; r < R; ++r) c[r] = z[r] == -INFINITY ? z[r] : fmaf(c[r], inv, bias[r]);
  }
}

// Descending sort of a lane's keys (odd-even merge networks).
template <int R>
__device__ __forceinline__ void sort_lane(uint32_t (&v)[R]) {
  if constexpr (R == 2) order2(v[0], v[1]);
  if constexpr (R >= 4) {
#pragma unroll
    for (int p = 1; p < R; p <<= 1)
#pragma unroll
      for (int q = p; q >= 1; q >>= 1)
#pragma unroll
        for (int j = q % p; j + q < R; j += 2 * q)
#pragma unroll
          for (int i = 0; i < q; ++i)
            if (i + j + q < R && (i + j) / (2 * p) == (i + j + q) / (2 * p)) order2(v[i + j], v[i + j + q]);
  }
}

// Lane j < k gets the j-th largest key, lane k (k < 32) the next one.  The
// lanes' keys are consumed.  Up to eight keys a lane are sorted first, so that
// a round looks at one key a lane and the lane that gave it moves up; more
// are scanned each round.
template <int R>
__device__ __forceinline__ uint32_t pick(uint32_t (&v)[R], int rounds) {
  const int lane = threadIdx.x & 31;
  uint32_t mine = 0u;
  if constexpr (R <= 8) sort_lane<R>(v);
  for (int j = 0; j < rounds; ++j) {
    uint32_t head = v[0];
    if constexpr (R > 8) {
#pragma unroll
      for (int r = 1; r < R; ++r) head = max(head, v[r]);
    }
    const uint32_t top = __reduce_max_sync(FULL_MASK, head);
    if (lane == j) mine = top;
    if constexpr (R <= 8) {
      if (head == top) {
#pragma unroll
        for (int r = 0; r + 1 < R; ++r) v[r] = v[r + 1];
        v[R - 1] = 0u;
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = v[r] == top ? 0u : v[r];
    }
  }
  return mine;
}

// The choice by full order keys, one round of two reductions per slot: for
// tokens whose sort_keys cannot tell.  Lane j gets slot j's expert or -1.
template <typename T, int R>
__device__ __noinline__ int pick_exact(const float (&c)[R], int k) {
  const int lane = threadIdx.x & 31;
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = choice_key(c[r]);
  int mine = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (key[r] > best) {
        best = key[r];
        at = Part<T, R>::expert(r);
      }
    const uint32_t top = __reduce_max_sync(FULL_MASK, best);
    if (top == 0u) break;
    const int e = static_cast<int>(__reduce_min_sync(FULL_MASK, best == top ? unsigned(at) : 0xFFFFFFFFu));
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (Part<T, R>::expert(r) == e) key[r] = 0u;
    if (lane == j) mine = e;
  }
  return mine;
}

// ---------------------------------------------------------------------------
// Forward.

// The tokens of this CTA.  Leaves the CTA's slots per expert in cnt and the
// sums of n_t p_te in psum (both E entries of shared memory; psum through
// `stage`, WARPS x E), complete after the block barrier that ends it.
template <typename T, int R, bool SIG, bool SCORES>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, unsigned* cnt, float* psum, float* stage,
                                             unsigned char* ring_smem) {
  using P = Part<T, R>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts, k = a.k;
  const bool exact = sizeof(T) == 2 && !a.bias;
  const bool need_p = a.loss || (!a.normalize && !SIG);
  int width = 1;
  while (width < k) width <<= 1;
  const T* logits = static_cast<const T*>(a.logits);
  const bool vec = reinterpret_cast<uintptr_t>(logits) % (P::VEC * sizeof(T)) == 0 && a.ld % P::VEC == 0;
  const int rounds = exact || k == E || k == 32 ? k : k + 1;
  float acc[R], bias[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    acc[r] = 0.f;
    bias[r] = a.bias && P::expert(r) < E ? a.bias[P::expert(r)] + 0.f : 0.f;
  }
  const int64_t step = int64_t(gridDim.x) * WARPS<R>;
  int64_t t = int64_t(blockIdx.x) * WARPS<R> + warp;
  const Ring<T, R> ring(ring_smem, vec, E);
  constexpr int S = Ring<T, R>::STAGES;
#pragma unroll
  for (int i = 0; i + 1 < S; ++i) ring.fetch(logits + (t + i * step) * a.ld, E, t + i * step < a.tokens, i);
  bool used = t < a.tokens && (!a.mask || a.mask[t]);
  // Where this token's row, the row to fetch and the outputs are; each moves by a step.
  const T* here = logits + t * a.ld;
  const T* ahead = here + (S - 1) * step * a.ld;
  const int64_t row_step = step * a.ld, slot_step = step * k;
  float* gate_at = a.gates + t * k + lane;
  int64_t* chosen_at = a.chosen + t * k + lane;
  for (int at = 0; t < a.tokens; t += step, at = at + 1 < S ? at + 1 : 0) {
    int mine = -1;  // lane j: the expert of slot j
    float gate = 0.f;
    if constexpr (S > 0) ring.fetch(ahead, E, t + (S - 1) * step < a.tokens, at > 0 ? at - 1 : S - 1);
    const bool use_next = !a.mask || (t + step < a.tokens && a.mask[t + step]);
    ring.wait();
    if (used) {
      const T* row = ring.row(here, at);
      float z[R], by[R];
      load_part<T, R>(row, E, vec, z);
      choose_by<SIG, SCORES, R>(z, bias, by);
      uint32_t key[R];
#pragma unroll
      for (int r = 0; r < R; ++r) key[r] = sort_key<R>(by[r], P::expert(r));
      const uint32_t got = pick<R>(key, rounds);
      constexpr uint32_t INDEX = 32u * R - 1u;
      if (lane < k && got >= AVAILABLE) mine = static_cast<int>(INDEX ^ (got & INDEX));
      float zc = mine >= 0 ? lm_float(row[mine]) : -INFINITY;
      // Unsure: a key above that of +inf (a NaN), keys of different c that
      // share their leading bits, or no next key to compare the last with.
      bool unsure = got > (0xff800000u | INDEX);
      if (!exact) {
        const uint32_t next = __shfl_down_sync(FULL_MASK, got, 1);
        unsure |= mine >= 0 && (lane + 1 < k || k < E) && (lane == 31 || (got ^ next) <= INDEX);
      }
      bool nan = false;
      if (__any_sync(FULL_MASK, unsure)) {
        float c[R];
#pragma unroll
        for (int r = 0; r < R; ++r) nan |= z[r] != z[r];
        choose_by<SIG, SCORES, R>(z, bias, c);
        nan = __any_sync(FULL_MASK, nan);
        mine = pick_exact<T, R>(c, k);
        zc = mine >= 0 ? lm_float(row[mine]) : -INFINITY;
      }
      const bool ok = mine >= 0;
      // The largest logit: that of the first slot, unless a bias chose it.
      float ref = __shfl_sync(FULL_MASK, zc, 0), sum = 1.f;
      if (!SIG && a.bias) {
        ref = z[0];
#pragma unroll
        for (int r = 1; r < R; ++r) ref = fmaxf(ref, z[r]);
        ref = key_to_float(__reduce_max_sync(FULL_MASK, ord_key(ref)));
      }
      if (need_p) {
        const int filled = __popc(__ballot_sync(FULL_MASK, ok));
        if (filled) {
          float s[R];
          sum = token_scores<SIG, R>(z, s, ref);
          const float scale = __fdividef(static_cast<float>(filled), sum);
#pragma unroll
          for (int r = 0; r < R; ++r) acc[r] = fmaf(s[r], scale, acc[r]);
        }
      }
      gate = slot_gate<SIG>(zc, ok, width, a.normalize, ref, sum);
      if (ok) {
        if (nan) gate = __int_as_float(0x7fc00000);
        atomicAdd(cnt + mine, 1u);
      }
    }
    if (lane < k) {
      *gate_at = gate;
      *chosen_at = mine;
    }
    here += row_step;
    ahead += row_step;
    gate_at += slot_step;
    chosen_at += slot_step;
    used = use_next;
    __syncwarp();  // the stage is free to be filled
  }
  if (a.loss) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (P::expert(r) < E) stage[warp * E + P::expert(r)] = acc[r];
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += WARPS<R> * 32) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS<R>; ++w) sum += stage[w * E + e];
      psum[e] = sum;
    }
  }
  __syncthreads();
}

// counts, and the terms of the loss, of the experts of one CTA of a cluster;
// rank 0 joins them: loss = E / N^2 sum_e counts_e (N P_e).
__device__ __forceinline__ void finish_loss(int E, unsigned long long c, float term, float* loss) {
  __shared__ float sf[32];
  __shared__ unsigned long long sn[32];
  __shared__ float cf[CLUSTER];
  __shared__ unsigned long long cn[CLUSTER];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  term = warp_sum(term);
#pragma unroll
  for (int d = 16; d; d >>= 1) c += __shfl_xor_sync(FULL_MASK, c, d);
  if (lane == 0) {
    sf[warp] = term;
    sn[warp] = c;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < warps; ++w) {
      term += sf[w];
      c += sn[w];
    }
    *cluster.map_shared_rank(&cf[cluster.block_rank()], 0) = term;
    *cluster.map_shared_rank(&cn[cluster.block_rank()], 0) = c;
  }
  cluster.sync();
  if (cluster.block_rank() == 0 && threadIdx.x == 0) {
    float sum = 0.f;
    unsigned long long n = 0;
    for (int i = 0; i < CLUSTER; ++i) {
      sum += cf[i];
      n += cn[i];
    }
    const float N = n ? static_cast<float>(n) : 1.f;
    *loss = static_cast<float>(E) * (sum / N) / N;
  }
}

// Shared memory of a CTA: the ring, counts, sums, the warps' sums.
template <typename T, int R>
constexpr size_t route_smem(int E) {
  return size_t(WARPS<R>) * Ring<T, R>::BYTES + size_t(2 + WARPS<R>) * E * 4;
}

// Few tokens: one cluster, the CTAs' sums joined through distributed shared
// memory; one launch and no workspace.
template <typename T, int R, bool SIG, bool SCORES>
__global__ void __launch_bounds__(WARPS<R> * 32) __cluster_dims__(CLUSTER, 1, 1) k_route_one(RouteArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NW = WARPS<R>;
  const int E = a.experts;
  unsigned* cnt = reinterpret_cast<unsigned*>(smem + NW * Ring<T, R>::BYTES);
  float* psum = reinterpret_cast<float*>(cnt + E);
  float* stage = psum + E;
  for (int e = threadIdx.x; e < E; e += NW * 32) cnt[e] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  route_tokens<T, R, SIG, SCORES>(a, cnt, psum, stage, smem);
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  unsigned long long n = 0;
  float term = 0.f;
  // Thread i of every CTA takes expert CLUSTER i + rank, and so on.
  for (int e = threadIdx.x * CLUSTER + cluster.block_rank(); e < E; e += CLUSTER * NW * 32) {
    unsigned long long c = 0;
    float p = 0.f;
#pragma unroll
    for (int i = 0; i < CLUSTER; ++i) {
      c += *cluster.map_shared_rank(cnt + e, i);
      if (a.loss) p += *cluster.map_shared_rank(psum + e, i);
    }
    a.counts[e] = static_cast<int64_t>(c);
    n += c;
    term += static_cast<float>(c) * p;
  }
  if (a.loss) finish_loss(E, n, term, a.loss);
  cluster.sync();  // every CTA's shared memory has been read
}

// Many tokens: each CTA writes its sums, and k_route_join adds them up.
template <typename T, int R, bool SIG, bool SCORES>
__global__ void __launch_bounds__(WARPS<R> * 32, PER_SM<R>) k_route(RouteArgs a, float* part_p, unsigned* part_c) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NW = WARPS<R>;
  const int E = a.experts;
  unsigned* cnt = reinterpret_cast<unsigned*>(smem + NW * Ring<T, R>::BYTES);
  float* psum = reinterpret_cast<float*>(cnt + E);
  float* stage = psum + E;
  for (int e = threadIdx.x; e < E; e += NW * 32) cnt[e] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  route_tokens<T, R, SIG, SCORES>(a, cnt, psum, stage, smem);
  for (int e = threadIdx.x; e < E; e += NW * 32) {
    part_c[int64_t(blockIdx.x) * E + e] = cnt[e];
    if (a.loss) part_p[int64_t(blockIdx.x) * E + e] = psum[e];
  }
}

// Adds the CTAs' sums in a fixed order: one cluster, 32 experts at a time a
// CTA, the parts shared out over its warps.
constexpr int JOIN_THREADS = 1024;
__global__ void __launch_bounds__(JOIN_THREADS) __cluster_dims__(CLUSTER, 1, 1)
    k_route_join(int parts, int E, const float* part_p, const unsigned* part_c, int64_t* counts, float* loss) {
  __shared__ float sp[32][33];
  __shared__ unsigned sc[32][33];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cluster.sync();  // every CTA runs before finish_loss writes to rank 0
  pdl_wait();
  pdl_trigger();
  unsigned long long n = 0;
  float term = 0.f;
  for (int base = cluster.block_rank() * 32; base < E; base += CLUSTER * 32) {
    const int e = base + lane;
    unsigned c = 0u;
    float p = 0.f;
    if (e < E)
#pragma unroll 10
      for (int i = warp; i < parts; i += 32) {
        c += __ldg(part_c + int64_t(i) * E + e);
        if (loss) p += __ldg(part_p + int64_t(i) * E + e);
      }
    __syncthreads();
    sc[warp][lane] = c;
    sp[warp][lane] = p;
    __syncthreads();
    // Warp w joins expert base + w over the 32 warps' sums.
    unsigned long long cc = sc[lane][warp];
#pragma unroll
    for (int d = 16; d; d >>= 1) cc += __shfl_xor_sync(FULL_MASK, cc, d);
    const float pp = warp_sum(sp[lane][warp]);
    if (lane == 0 && base + warp < E) {
      counts[base + warp] = static_cast<int64_t>(cc);
      n += cc;
      term += static_cast<float>(cc) * pp;
    }
  }
  if (loss) finish_loss(E, n, term, loss);
}

// ---------------------------------------------------------------------------
// Gradient of the gates and of the balance loss; the choice and the counts
// are constants.  With a_e = dL E counts_e n_t / N^2:
//   dy = p (a - sum_e p_e a_e), and for the chosen
//   + g_j (dg_j - sum g dg)                          normalized
//   + p_i ([i chosen] dg_i - sum_j p_j dg_j)         softmax
//   + g_j dg_j                                       sigmoid
// and dz = dy (softmax) or dy sigmoid(-z).
template <typename T, int R, bool SIG>
__global__ void __launch_bounds__(WARPS<R> * 32, PER_SM<R>) k_route_backward(RouteBackwardArgs a) {
  using P = Part<T, R>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts, k = a.k;
  // The chosen experts' part of dy, this warp's.
  float* extra = reinterpret_cast<float*>(smem + WARPS<R> * Ring<T, R>::BYTES) + warp * 32 * R;
  for (int e = lane; e < 32 * R; e += 32) extra[e] = 0.f;
  __syncwarp();
  pdl_wait();
  pdl_trigger();
  int width = 1;
  while (width < k) width <<= 1;
  const T* logits = static_cast<const T*>(a.logits);
  T* grad = static_cast<T*>(a.grad_logits);
  const bool vec = reinterpret_cast<uintptr_t>(logits) % (P::VEC * sizeof(T)) == 0 && a.ld % P::VEC == 0;
  const bool out_vec = reinterpret_cast<uintptr_t>(grad) % (P::VEC * sizeof(T)) == 0 && a.grad_ld % P::VEC == 0;
  const int64_t step = int64_t(gridDim.x) * WARPS<R>;
  int64_t t = int64_t(blockIdx.x) * WARPS<R> + warp;
  const Ring<T, R> ring(smem, vec, E);
  constexpr int S = Ring<T, R>::STAGES;
#pragma unroll
  for (int i = 0; i + 1 < S; ++i) ring.fetch(logits + (t + i * step) * a.ld, E, t + i * step < a.tokens, i);
  float share[R];  // dL E counts_e / N^2
#pragma unroll
  for (int r = 0; r < R; ++r) share[r] = 0.f;
  if (a.grad_loss) {  // every warp adds the counts up for itself
    long long c[R];
    unsigned long long n = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c[r] = P::expert(r) < E ? a.counts[P::expert(r)] : 0;
      n += static_cast<unsigned long long>(c[r]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(FULL_MASK, n, d);
    const float N = n ? static_cast<float>(n) : 1.f;
    const float f = *a.grad_loss * static_cast<float>(E) / N / N;
#pragma unroll
    for (int r = 0; r < R; ++r) share[r] = f * static_cast<float>(c[r]);
  }
  // A slot's expert as 32 bits, -1 for what is outside [0, E).
  auto slot = [&](int64_t e) { return e >= 0 && e < E ? static_cast<int>(e) : -1; };
  const int64_t* chosen_at = a.chosen + t * k + lane;
  const float* dg_at = a.grad_gates ? a.grad_gates + t * k + lane : nullptr;
  const T* here = logits + t * a.ld;
  const T* ahead = here + (S - 1) * step * a.ld;
  T* out_at = grad + t * a.grad_ld;
  const int64_t row_step = step * a.ld, out_step = step * a.grad_ld, slot_step = step * k;
  int next_mine = t < a.tokens && lane < k ? slot(*chosen_at) : -1;
  float next_dg = dg_at && t < a.tokens && lane < k ? *dg_at : 0.f;
  for (int at = 0; t < a.tokens; t += step, at = at + 1 < S ? at + 1 : 0) {
    const int mine = next_mine;
    const bool ok = mine >= 0;
    const float dg = ok ? next_dg : 0.f;
    const T* const this_row = here;
    T* const out = out_at;
    if constexpr (S > 0) ring.fetch(ahead, E, t + (S - 1) * step < a.tokens, at > 0 ? at - 1 : S - 1);
    here += row_step;
    ahead += row_step;
    out_at += out_step;
    chosen_at += slot_step;
    if (dg_at) dg_at += slot_step;
    if (lane < k && t + step < a.tokens) {
      next_mine = slot(*chosen_at);
      if (dg_at) next_dg = *dg_at;
    }
    const int filled = __popc(__ballot_sync(FULL_MASK, ok));
    float z[R], s[R];
    ring.wait();
    if (!filled) {  // masked, or nothing to choose: no gradient
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = 0.f;
      store_part<T, R>(out, E, out_vec, s);
      __syncwarp();
      continue;
    }
    const T* row = ring.row(this_row, at);
    load_part<T, R>(row, E, vec, z);
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < R; ++r) m = fmaxf(m, z[r]);
    m = key_to_float(__reduce_max_sync(FULL_MASK, ord_key(m)));
    const float sum = token_scores<SIG, R>(z, s, m), inv = lm_rcp(sum);
    const float n_t = static_cast<float>(filled);
    float dot = 0.f;
    if (a.grad_loss) {
#pragma unroll
      for (int r = 0; r < R; ++r) dot = fmaf(s[r], share[r], dot);
      dot = warp_sum(dot) * inv * n_t;
    }
    if (a.grad_gates) {
      const float zc = ok ? lm_float(row[mine]) : -INFINITY;
      const float g = slot_gate<SIG>(zc, ok, width, a.normalize, m, sum);
      float d = g * dg;
      if (a.normalize || !SIG) {
        const float gd = __shfl_sync(FULL_MASK, slots_sum(d, width), 0);
        if (a.normalize)
          d = g * (dg - gd);
        else
          dot += gd;
      }
      if (ok) extra[mine] = d;
      __syncwarp();
    }
    float chosen_part[R];
    load_shared<T, R>(extra, chosen_part);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float dy = fmaf(s[r] * inv, fmaf(share[r], n_t, -dot), chosen_part[r]);
      if constexpr (SIG) dy *= sigmoid(-z[r]);
      s[r] = dy;
    }
    store_part<T, R>(out, E, out_vec, s);
    __syncwarp();
    if (a.grad_gates && ok) extra[mine] = 0.f;
    __syncwarp();
  }
}

template <typename F>
cudaError_t by_score(bool sig, F&& f) {
  return sig ? f(std::true_type{}) : f(std::false_type{});
}

template <typename F>
cudaError_t by_type(int type, F&& f) {
  switch (type) {
    case PROFK_F32: return f(float{});
    case PROFK_BF16: return f(__nv_bfloat16{});
    default: return f(__half{});
  }
}

// The smallest R with 32 R >= E.
template <typename F>
cudaError_t by_width(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

int route_grid(int64_t tokens, int warps, int per_sm) {
  const int64_t need = (tokens + warps - 1) / warps;
  const int64_t most = per_sm * static_cast<int64_t>(sms());
  return static_cast<int>(need < most ? need : most);
}

// Launches a kernel with `smem` bytes of dynamic shared memory, `most` being what any
// call of it asks for.  The limit is the kernel's, for all host threads: it is
// set to the same number whatever the call, so that none of them takes it back
// below what another is about to launch with.
template <typename... KArgs, typename... Args>
cudaError_t launch_with(void (*kernel)(KArgs...), int grid, int threads, size_t smem, size_t most, cudaStream_t stream,
                        Args... args) {
  if (most > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, dim3(grid), dim3(threads), smem, stream, args...);
}

// One launch up to this many tokens (two a warp of the cluster).  (x 128 bfloat16,
// k = 8: 16 tokens take 4.4 us, and 5.5 by the grid and the join; 512 take 6.0 by
// the grid and 8.3 in one launch.)
template <int R>
constexpr int64_t ONE_TOKENS = 2 * CLUSTER * WARPS<R>;

template <bool SCORES>
cudaError_t launch_forward(const RouteArgs& a, cudaStream_t stream) {
  return by_type(a.type, [&](auto type) {
    return by_width(a.experts, [&](auto width) {
      return by_score(a.sigmoid, [&](auto sig) {
        using T = decltype(type);
        constexpr int R = decltype(width)::value;
        constexpr bool SIG = decltype(sig)::value;
        const size_t smem = route_smem<T, R>(a.experts), most = route_smem<T, R>(32 * R);
        if (a.tokens <= ONE_TOKENS<R>)
          return launch_with(k_route_one<T, R, SIG, SCORES>, CLUSTER, WARPS<R> * 32, smem, most, stream, a);
        const int grid = route_grid(a.tokens, WARPS<R>, PER_SM<R>);
        cudaMemPool_t pool;
        cudaError_t err = library_pool(&pool);
        if (err != cudaSuccess) return err;
        void* part = nullptr;
        const size_t each = size_t(grid) * a.experts * 4;
        err = cudaMallocFromPoolAsync(&part, (a.loss ? 2 : 1) * each, pool, stream);
        if (err != cudaSuccess) return err;
        unsigned* part_c = static_cast<unsigned*>(part);
        float* part_p = reinterpret_cast<float*>(static_cast<char*>(part) + each);
        err = launch_with(k_route<T, R, SIG, SCORES>, grid, WARPS<R> * 32, smem, most, stream, a, part_p, part_c);
        if (err == cudaSuccess)
          err = launch_kernel(k_route_join, dim3(CLUSTER), dim3(JOIN_THREADS), 0, stream, grid, a.experts, part_p, part_c,
                              a.counts, a.loss);
        const cudaError_t freed = cudaFreeAsync(part, stream);
        return err != cudaSuccess ? err : freed;
      });
    });
  });
}

}  // namespace
}  // namespace profk
