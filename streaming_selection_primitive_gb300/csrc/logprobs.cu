// Log-probabilities of given tokens from logits, the gradient, and the losses on them:
// the clipped policy loss (perhaps with its gradient in the same launch) and the
// preference loss of pairs.
//
// With c = log2(e) / T, m the row's largest logit, x_i = (l_i - m) c, s = sum 2^x_i and
// t = sum x_i 2^x_i:
//   logprob = ln 2 x_token - ln s,   H = ln s - ln 2 t / s,
//   d(g logprob + h H) / d l_i = [g 1(i = token) - p_i (g + h ln 2 (x_i - t / s))] / T,  p_i = 2^x_i / s.
//
// A row is taken by a cluster of CTAs (k_logprobs) or, where it is short, by a warp
// (k_logprobs_short): one pass with a running maximum and sums, one exchange.  For a
// policy loss with its gradient the same CTAs then go over their part again.
#include <cooperative_groups.h>

#include "../../include/profk.h"
#include "lm.h"
#include "logprobs.cuh"

namespace cg = cooperative_groups;

namespace profk {
namespace {

constexpr int THREADS = 512;    // of a CTA that takes a row or a part of one
constexpr int WARPS = THREADS / 32;
constexpr int SHORT_THREADS = 256;  // of a CTA whose warps take a row each
constexpr int LOADS = 4;        // 16-byte loads of a thread before it looks at what came
constexpr int MAX_CLUSTER = 8;

// ---------------------------------------------------------------------------
// 16 bytes of a row.

template <typename T>
constexpr int PER_VECTOR = 16 / int(sizeof(T));

// Pair i of the elements in v.
template <typename T>
__device__ __forceinline__ Pair element_pair(const uint4& v, int i);
template <>
__device__ __forceinline__ Pair element_pair<float>(const uint4& v, int i) {
  return i == 0 ? pair(__uint_as_float(v.x), __uint_as_float(v.y)) : pair(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
template <>
__device__ __forceinline__ Pair element_pair<__nv_bfloat16>(const uint4& v, int i) {
  const uint32_t w = word(v, i);
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ Pair element_pair<__half>(const uint4& v, int i) {
  const uint32_t w = word(v, i);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

// The largest of all elements (NaN is passed over).
__device__ __forceinline__ float largest(const uint4 (&v)[LOADS], float) {
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < LOADS; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, __uint_as_float(word(v[u], i)));
  return m;
}
template <typename H2, typename T>
__device__ __forceinline__ float largest_half(const uint4 (&v)[LOADS]) {
  H2 m;
#pragma unroll
  for (int u = 0; u < LOADS; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = word(v[u], i);
      const H2 h = *reinterpret_cast<const H2*>(&w);
      m = u + i == 0 ? h : __hmax2(m, h);
    }
  return fmaxf(lm_float(m.x), lm_float(m.y));
}
__device__ __forceinline__ float largest(const uint4 (&v)[LOADS], __nv_bfloat16) {
  return largest_half<__nv_bfloat162, __nv_bfloat16>(v);
}
__device__ __forceinline__ float largest(const uint4 (&v)[LOADS], __half) { return largest_half<__half2, __half>(v); }

template <typename T>
__device__ __forceinline__ uint4 nothing();  // elements of -inf
template <>
__device__ __forceinline__ uint4 nothing<float>() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
template <>
__device__ __forceinline__ uint4 nothing<__nv_bfloat16>() {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}
template <>
__device__ __forceinline__ uint4 nothing<__half>() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }

__device__ __forceinline__ void put_pair(float* out, float a, float b) { *reinterpret_cast<float2*>(out) = make_float2(a, b); }
__device__ __forceinline__ void put_pair(__nv_bfloat16* out, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(out) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void put_pair(__half* out, float a, float b) {
  *reinterpret_cast<__half2*>(out) = __floats2half2_rn(a, b);
}

// ---------------------------------------------------------------------------
// A row's elements in memory: up to the first 16-byte boundary one by one (`head`),
// then `vectors` of 16 bytes, then `tail` one by one.
template <typename T>
struct Layout {
  int head, vectors, tail;
  __device__ __forceinline__ Layout(const T* p, int n) {
    const int to_boundary = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / int(sizeof(T));
    head = min(to_boundary, n);
    vectors = (n - head) / PER_VECTOR<T>;
    tail = n - head - vectors * PER_VECTOR<T>;
  }
  // The element that is this thread's alone, -1 where there is none: the first threads of
  // the first part have the head, the next eight of the last part the tail.
  __device__ __forceinline__ int single(int thread, bool first, bool last) const {
    if (first && thread < head) return thread;
    if (last && thread >= 8 && thread < 8 + tail) return head + vectors * PER_VECTOR<T> + thread - 8;
    return -1;
  }
};

// Part `rank` of `parts` of the vectors.
__device__ __forceinline__ int part_begin(int vectors, int rank, int parts) {
  return static_cast<int>(static_cast<int64_t>(vectors) * rank / parts);
}

// One chunk of elements joins what has been seen.
template <typename T, bool ENTROPY>
__device__ __forceinline__ void take(Running& r, const uint4 (&v)[LOADS], float c) {
  const float m = fmaxf(r.m, largest(v, T{}));
  const float d = shrink(r.m, reference(m), c), f = lm_exp2(d);
  const Pair minus = pair(-reference(m), -reference(m)), cc = pair(c, c);
  Pair s[2] = {0, 0}, t[2] = {0, 0};
#pragma unroll
  for (int u = 0; u < LOADS; ++u)
#pragma unroll
    for (int i = 0; i < PER_VECTOR<T> / 2; ++i) {
      float x0, x1;
      split(mul2(add2(element_pair<T>(v[u], i), minus), cc), x0, x1);
      const Pair e = pair(lm_exp2(x0), lm_exp2(x1));
      s[i & 1] = add2(s[i & 1], e);
      if (ENTROPY) t[i & 1] = fma2(pair(fmaxf(x0, NO_MASS), fmaxf(x1, NO_MASS)), e, t[i & 1]);
    }
  float a, b;
  if (ENTROPY) {
    split(add2(t[0], t[1]), a, b);
    r.t = f * (r.t + d * r.s);
    r.t_lost = f * (r.t_lost + d * r.s_lost);
    add_exact(r.t, r.t_lost, a + b);
  }
  split(add2(s[0], s[1]), a, b);
  r.s *= f;
  r.s_lost *= f;
  add_exact(r.s, r.s_lost, a + b);
  r.m = m;
}

// The pass over vectors [begin, end) and this thread's single element by `STEP` threads.
template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ Running pass(const T* p, const Layout<T>& at, int begin, int end, int thread, int single, float c) {
  const uint4* body = reinterpret_cast<const uint4*>(p + at.head);
  Running r{-INFINITY, 0.f, 0.f, 0.f, 0.f};
  if (single >= 0) {
    const float v = lm_float(p[single]);
    r.m = fmaxf(v, -INFINITY);
    r.s = v == -INFINITY ? 0.f : v - v + 1.f;
  }
  uint4 v[LOADS], next[LOADS];
  const auto load = [&](uint4(&w)[LOADS], int i) {
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + u * STEP + thread;
      w[u] = j < end ? body[j] : nothing<T>();
    }
  };
  int i = begin;
  if (i < end) load(next, i);
  while (i < end) {
#pragma unroll
    for (int u = 0; u < LOADS; ++u) v[u] = next[u];
    i += LOADS * STEP;
    if (i < end) load(next, i);
    take<T, ENTROPY>(r, v, c);
  }
  return r;
}

// What a row's gradient is made of: element i gets e (k0 + k1 x) with x = (l - m) c and
// e = 2^x, and the token's element `one` besides.
struct Slopes {
  float m, c, k0, k1, one;
};

// g and h: the derivatives of the result by the row's log-probability and its entropy.
template <bool ENTROPY>
__device__ __forceinline__ Slopes slopes_of(float m, float s, float mean_x, float temperature, float c, float g, float h) {
  const float per_T = 1.f / temperature;
  Slopes y{reference(m), c, 0.f, 0.f, g * per_T};
  if (s == 0.f) {  // nothing to put on any token
    y.one = 0.f;
    return y;
  }
  const float scale = per_T / s;
  y.k0 = -(ENTROPY ? g - h * LN2 * mean_x : g) * scale;
  if (ENTROPY) y.k1 = -h * LN2 * scale;
  return y;
}

template <bool ENTROPY>
__device__ __forceinline__ float slope_at(const Slopes& k, float l) {
  const float x = (l - k.m) * k.c, e = lm_exp2(x);
  return e * (ENTROPY ? fmaf(k.k1, fmaxf(x, NO_MASS), k.k0) : k.k0);
}

// The gradient of vectors [begin, end) and of this thread's single element, by STEP threads.
// `same`: logits and gradient stand alike to the 16-byte boundaries.
template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ void write_gradient(const T* p, T* out, const Layout<T>& at, int begin, int end, int thread,
                                               int single, int token, const Slopes& k, bool same) {
  if (single >= 0) out[single] = lm_cast<T>(slope_at<ENTROPY>(k, lm_float(p[single])) + (single == token ? k.one : 0.f));
  constexpr int N = PER_VECTOR<T>;
  const uint4* body = reinterpret_cast<const uint4*>(p + at.head);
  T* to = out + at.head;
  const Pair minus = pair(-k.m, -k.m), cc = pair(k.c, k.c), k0 = pair(k.k0, k.k0), k1 = pair(k.k1, k.k1);
  const int token_vector = token >= at.head ? (token - at.head) / N : -1;
  for (int i = begin; i < end; i += LOADS * STEP) {
    uint4 v[LOADS];
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + u * STEP + thread;
      if (j < end) v[u] = body[j];
    }
#pragma unroll
    for (int u = 0; u < LOADS; ++u) {
      const int j = i + u * STEP + thread;
      if (j >= end) break;
      alignas(16) T y[N];
#pragma unroll
      for (int q = 0; q < N / 2; ++q) {
        float x0, x1, y0, y1;
        split(mul2(add2(element_pair<T>(v[u], q), minus), cc), x0, x1);
        const Pair e = pair(lm_exp2(x0), lm_exp2(x1));
        split(mul2(e, ENTROPY ? fma2(k1, pair(fmaxf(x0, NO_MASS), fmaxf(x1, NO_MASS)), k0) : k0), y0, y1);
        if (j == token_vector) {
          const int q_token = token - at.head - j * N - 2 * q;
          if (q_token == 0) y0 += k.one;
          if (q_token == 1) y1 += k.one;
        }
        put_pair(y + 2 * q, y0, y1);
      }
      if (same) {
        reinterpret_cast<uint4*>(to)[j] = *reinterpret_cast<const uint4*>(y);
      } else {
#pragma unroll
        for (int q = 0; q < N; ++q) to[j * N + q] = y[q];
      }
    }
  }
}

template <typename T, int STEP>
__device__ __forceinline__ void write_zeros(T* out, const Layout<T>& at, int begin, int end, int thread, int single) {
  if (single >= 0) out[single] = lm_cast<T>(0.f);
  uint4* to = reinterpret_cast<uint4*>(out + at.head);
  for (int j = begin + thread; j < end; j += STEP) to[j] = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// A row's inputs besides its logits, and its outputs besides its gradient.

template <bool GRADIENT>
struct Row {
  int64_t token;
  float temperature, c, logit;
  float old_lp, advantage, ref_lp, weight;  // GRADIENT: of the policy loss
  bool live;
};

template <typename T, bool GRADIENT>
__device__ __forceinline__ Row<GRADIENT> load_row(const LogprobArgs& a, const PolicyHow& how, int64_t row) {
  Row<GRADIENT> r;
  r.token = a.tokens[row];
  r.temperature = a.temperature ? a.temperature[row] : a.all_temperature;
  r.c = inverse_temperature(r.temperature);
  r.live = r.token >= 0;
  if (a.weights && a.weights[row] == 0.f) r.live = false;
  if (a.offsets && (row < a.offsets[0] || row >= a.offsets[a.sequences])) r.live = false;
  // A token that the vocabulary has not is no number.
  r.logit = NAN;
  if (r.live && r.token < a.n) r.logit = lm_float(static_cast<const T*>(a.logits)[row * a.ld + r.token]);
  if (GRADIENT) {
    r.old_lp = how.old_logprobs[row];
    r.advantage = how.advantages[row];
    r.ref_lp = how.ref_logprobs ? how.ref_logprobs[row] : 0.f;
    r.weight = how.weights ? how.weights[row] : how.all_weight;
  }
  return r;
}

__device__ __forceinline__ void store_left_out(const LogprobArgs& a, int64_t row) {
  a.logprobs[row] = 0.f;
  if (a.entropies) a.entropies[row] = 0.f;
  if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
  if (a.zeros) a.zeros[row] = 0.f;
}

__device__ __forceinline__ float store_row(const LogprobArgs& a, int64_t row, const RowSum& y, float logit, float temperature, bool write) {
  const float lp = row_logprob(y, logit, temperature);
  if (write) {
    a.logprobs[row] = lp;
    if (a.entropies) a.entropies[row] = row_entropy(y);
    if (a.stats) a.stats[row] = make_float2(y.m, y.s);
    if (a.zeros) a.zeros[row] = 0.f;
  }
  return lp;
}

template <bool ENTROPY, bool GRADIENT>
__device__ __forceinline__ Slopes policy_slopes(const Row<GRADIENT>& r, const RowSum& y, float lp, const PolicyHow& how) {
  const PolicyTerm term = policy_term(lp, r.old_lp, r.advantage, how.ref_logprobs != nullptr, r.ref_lp, how);
  return slopes_of<ENTROPY>(y.m, y.s, y.t / y.s, r.temperature, r.c, r.weight * term.slope, -how.entropy * r.weight);
}

// ---------------------------------------------------------------------------
// A row by a cluster of CTAs.
template <typename T, bool ENTROPY, bool GRADIENT>
__global__ void __launch_bounds__(THREADS, 2) k_logprobs(LogprobArgs a, PolicyHow how) {
  pdl_trigger();
  pdl_wait();
  __shared__ RowSum sums[MAX_CLUSTER * WARPS];
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / parts;
  const int thread = threadIdx.x, lane = thread & 31, warp = thread >> 5, n = static_cast<int>(a.n);
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  const Row<GRADIENT> r = load_row<T, GRADIENT>(a, how, row);
  if (!r.live) {  // the same for the whole cluster: none of it waits
    if (rank == 0 && thread == 0) store_left_out(a, row);
    if (GRADIENT) {
      const Layout<T> to(out, n);
      write_zeros<T, THREADS>(out, to, part_begin(to.vectors, rank, parts), part_begin(to.vectors, rank + 1, parts), thread,
                              to.single(thread, rank == 0, rank == parts - 1));
    }
    return;
  }
  if (parts > 1) cluster.barrier_arrive();  // (a CTA's shared memory is written once it runs)
  const Layout<T> at(p, n);
  const int begin = part_begin(at.vectors, rank, parts), end = part_begin(at.vectors, rank + 1, parts);
  const int single = at.single(thread, rank == 0, rank == parts - 1);
  RowSum y = warp_join<ENTROPY>(total(pass<T, ENTROPY, THREADS>(p, at, begin, end, thread, single, r.c)), r.c);
  if (parts > 1) {
    cluster.barrier_wait();
    if (lane < parts) cluster.map_shared_rank(sums, lane)[rank * WARPS + warp] = y;
    cluster.sync();
  } else {
    if (lane == 0) sums[warp] = y;
    __syncthreads();
  }
  // Every warp joins all parts, in the same order.
  y = {-INFINITY, 0.f, 0.f};
  for (int i = lane; i < parts * WARPS; i += 32) y = joined(y, sums[i], r.c);
  y = warp_join<ENTROPY>(y, r.c);
  if (!(r.c > 0.f)) y.s = NAN;
  const float lp = store_row(a, row, y, r.logit, r.temperature, rank == 0 && thread == 0);
  if (GRADIENT) {
    const Slopes k = policy_slopes<ENTROPY>(r, y, lp, how);
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    write_gradient<T, ENTROPY, THREADS>(p, out, at, begin, end, thread, single,
                                        static_cast<int>(r.token < a.n ? r.token : -1), k, same);
  }
}

// A row by a warp.
template <typename T, bool ENTROPY, bool GRADIENT>
__global__ void __launch_bounds__(SHORT_THREADS) k_logprobs_short(LogprobArgs a, PolicyHow how) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, n = static_cast<int>(a.n);
  const int64_t row = int64_t(blockIdx.x) * (SHORT_THREADS / 32) + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  const Row<GRADIENT> r = load_row<T, GRADIENT>(a, how, row);
  if (!r.live) {
    if (lane == 0) store_left_out(a, row);
    if (GRADIENT) {
      const Layout<T> to(out, n);
      write_zeros<T, 32>(out, to, 0, to.vectors, lane, to.single(lane, true, true));
    }
    return;
  }
  const Layout<T> at(p, n);
  const int single = at.single(lane, true, true);
  RowSum y = warp_join<ENTROPY>(total(pass<T, ENTROPY, 32>(p, at, 0, at.vectors, lane, single, r.c)), r.c);
  if (!(r.c > 0.f)) y.s = NAN;
  const float lp = store_row(a, row, y, r.logit, r.temperature, lane == 0);
  if (GRADIENT) {
    const Slopes k = policy_slopes<ENTROPY>(r, y, lp, how);
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    write_gradient<T, ENTROPY, 32>(p, out, at, 0, at.vectors, lane, single, static_cast<int>(r.token < a.n ? r.token : -1), k, same);
  }
}

// ---------------------------------------------------------------------------
// The gradient from a forward pass's row sums: `parts` CTAs a row, or a warp a row.
template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ void backward_row(const LogprobBackwardArgs& a, int64_t row, int rank, int parts, int thread) {
  const int n = static_cast<int>(a.n);
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  const int64_t token = a.tokens[row];
  float g = a.grad_logprobs ? a.grad_logprobs[row] : 0.f;
  float h = ENTROPY ? a.grad_entropies[row] : 0.f;
  if (token < 0 || (g == 0.f && h == 0.f)) {  // left out, whatever the logits hold
    const Layout<T> to(out, n);
    write_zeros<T, STEP>(out, to, part_begin(to.vectors, rank, parts), part_begin(to.vectors, rank + 1, parts), thread,
                         to.single(thread, rank == 0, rank == parts - 1));
    return;
  }
  if (a.scale) {
    g *= *a.scale;
    h *= *a.scale;
  }
  if (token >= n) g = NAN;
  const Layout<T> at(p, n);
  const float temperature = a.temperature ? a.temperature[row] : a.all_temperature, c = inverse_temperature(temperature);
  const float2 stats = a.stats[row];
  const float mean_x = ENTROPY ? (logf(stats.y) - a.entropies[row]) * LOG2E : 0.f;
  const Slopes k = slopes_of<ENTROPY>(stats.x, stats.y, mean_x, temperature, c, g, h);
  const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  write_gradient<T, ENTROPY, STEP>(p, out, at, part_begin(at.vectors, rank, parts), part_begin(at.vectors, rank + 1, parts), thread,
                                   at.single(thread, rank == 0, rank == parts - 1), static_cast<int>(token < n ? token : -1), k, same);
}

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(THREADS, 2) k_logprobs_backward(LogprobBackwardArgs a, int parts) {
  pdl_trigger();
  pdl_wait();
  backward_row<T, ENTROPY, THREADS>(a, blockIdx.x / parts, static_cast<int>(blockIdx.x % parts), parts, threadIdx.x);
}

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(SHORT_THREADS) k_logprobs_backward_short(LogprobBackwardArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t row = int64_t(blockIdx.x) * (SHORT_THREADS / 32) + (threadIdx.x >> 5);
  if (row < a.rows) backward_row<T, ENTROPY, 32>(a, row, 0, 1, threadIdx.x & 31);
}

// ---------------------------------------------------------------------------
// The sums over rows.  Doubles, in a fixed order: the same call gives the same bits.

constexpr int JOIN_THREADS = 512;
constexpr int JOIN_CLUSTER = 8;

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

// Sums over the cluster of COUNT values a thread, to thread 0 of CTA 0.  All threads call it.
template <int COUNT>
__device__ __forceinline__ void cluster_sum(double (&v)[COUNT]) {
  __shared__ double part[COUNT][JOIN_CLUSTER * (JOIN_THREADS / 32)];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), parts = static_cast<int>(cluster.num_blocks());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster.sync();  // (a CTA's shared memory is written once it runs)
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    v[i] = warp_sum(v[i]);
    if (lane == 0) cluster.map_shared_rank(&part[i][0], 0)[rank * (JOIN_THREADS / 32) + warp] = v[i];
  }
  cluster.sync();
  if (rank == 0 && warp < COUNT) {
    double s = 0.;
    for (int i = lane; i < parts * (JOIN_THREADS / 32); i += 32) s += part[warp][i];
    s = warp_sum(s);
    __syncwarp();
    if (lane == 0) part[warp][0] = s;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = part[i][0];
}

__global__ void __launch_bounds__(JOIN_THREADS) k_policy_join(LogprobArgs a, PolicyHow how, PolicyOut out) {
  pdl_trigger();
  pdl_wait();
  double v[4] = {0., 0., 0., 0.};
  const int64_t step = int64_t(gridDim.x) * JOIN_THREADS;
  for (int64_t row = int64_t(blockIdx.x) * JOIN_THREADS + threadIdx.x; row < a.rows; row += step) {
    const float w = how.weights ? how.weights[row] : how.all_weight;
    const bool live = a.tokens[row] >= 0 && w != 0.f;
    float slope = 0.f, h = 0.f;
    if (live) {
      const PolicyTerm term = policy_term(a.logprobs[row], how.old_logprobs[row], how.advantages[row],
                                          how.ref_logprobs != nullptr, how.ref_logprobs ? how.ref_logprobs[row] : 0.f, how);
      const float H = a.entropies ? a.entropies[row] : 0.f;
      v[0] += double(w) * (double(term.loss) - (how.entropy != 0.f ? double(how.entropy) * H : 0.));
      v[1] += double(w) * term.kl;
      v[2] += term.clipped ? double(w) : 0.;
      v[3] += double(w) * H;
      slope = w * term.slope;
      h = -how.entropy * w;
    }
    out.slopes[row] = slope;
    if (out.entropy_slopes) out.entropy_slopes[row] = h;
  }
  cluster_sum(v);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *out.loss = static_cast<float>(v[0]);
#pragma unroll
    for (int i = 0; i < 3; ++i) out.sums[i] = static_cast<float>(v[i + 1]);
  }
}

// log(1 + exp v)
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// A pair by a team of `team` threads (a warp, or the CTA): its margin, its term of the loss
// and its rows' slopes.
__global__ void __launch_bounds__(JOIN_THREADS) k_preference_join(LogprobArgs a, PreferenceHow how, PreferenceOut out, int team) {
  pdl_trigger();
  pdl_wait();
  __shared__ double across[2][2][JOIN_THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, thread = threadIdx.x % team;
  const int64_t pairs = a.sequences / 2, teams = int64_t(gridDim.x) * (JOIN_THREADS / team);
  double loss[1] = {0.};
  // (A team of the whole CTA goes round together: the bound is the same for all of it.)
  for (int64_t pair = int64_t(blockIdx.x) * (JOIN_THREADS / team) + threadIdx.x / team; pair < pairs; pair += teams) {
    double sum[2], count[2];
    int64_t begin[2], end[2];
    bool good = true;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      begin[side] = a.offsets[2 * pair + side];
      end[side] = a.offsets[2 * pair + side + 1];
      // Offsets that fall or leave the rows: nothing of the sequence is looked at.
      if (begin[side] < 0 || end[side] < begin[side] || end[side] > a.rows) {
        good = false;
        begin[side] = end[side] = 0;
      }
      double s = 0.;
      int live = 0;
      for (int64_t row = begin[side] + thread; row < end[side]; row += team)
        if (a.tokens[row] >= 0) {
          s += double(a.logprobs[row]) - (how.ref_logprobs ? double(how.ref_logprobs[row]) : 0.);
          ++live;
        }
      sum[side] = warp_sum(s);
      count[side] = __reduce_add_sync(FULL_MASK, live);
    }
    if (team > 32) {
      __syncthreads();  // (of the pair before, all is read)
      if (lane == 0)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          across[side][0][warp] = sum[side];
          across[side][1][warp] = count[side];
        }
      __syncthreads();
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        sum[side] = warp_sum(lane < JOIN_THREADS / 32 ? across[side][0][lane] : 0.);
        count[side] = warp_sum(lane < JOIN_THREADS / 32 ? across[side][1][lane] : 0.);
      }
    }
    double share[2] = {1., 1.};
    if (how.average)
#pragma unroll
      for (int side = 0; side < 2; ++side) share[side] = 1. / fmax(count[side], 1.);
    float margin = static_cast<float>(how.beta * (sum[0] * share[0] - sum[1] * share[1]) - how.margin);
    if (!good) margin = NAN;
    const float eps = how.smoothing, rest = 1.f - eps;
    // (A side without weight is left out: it may be infinite.)
    float term = 0.f, slope = 0.f;
    if (rest != 0.f) {
      term += rest * softplus(-margin);
      slope -= rest / (1.f + expf(margin));
    }
    if (eps != 0.f) {
      term += eps * softplus(margin);
      slope += eps / (1.f + expf(-margin));
    }
    if (thread == 0) {
      loss[0] += term;
      out.margins[pair] = margin;
    }
    const double each = double(slope) * how.beta / double(pairs);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const float y = static_cast<float>((side ? -each : each) * share[side]);
      for (int64_t row = begin[side] + thread; row < end[side]; row += team)
        if (a.tokens[row] >= 0) out.slopes[row] = y;
    }
  }
  cluster_sum(loss);
  if (blockIdx.x == 0 && threadIdx.x == 0) *out.loss = pairs ? static_cast<float>(loss[0] / double(pairs)) : 0.f;
}

// ---------------------------------------------------------------------------
// Launches.

template <typename F>
cudaError_t by_type(int type, F&& f) {
  if (type == PROFK_F32) return f(float{});
  if (type == PROFK_BF16) return f(__nv_bfloat16{});
  return f(__half{});
}

template <typename F>
cudaError_t by_flag(bool flag, F&& f) {
  return flag ? f(std::true_type{}) : f(std::false_type{});
}

int64_t row_bytes(int64_t n, int type) { return n * (type == PROFK_F32 ? 4 : 2); }

bool is_short(int64_t n, int type) { return row_bytes(n, type) <= 8192; }

// CTAs a row: as many as fit the SMs at once, of 8 KB or more each.
int cluster_for(int64_t rows, int64_t n, int type) {
  int parts = 1;
  while (parts < MAX_CLUSTER && rows * parts * 2 <= 2 * sms() && row_bytes(n, type) / (parts * 2) >= 8192) parts *= 2;
  return parts;
}

cudaError_t launch_rows(const LogprobArgs& a, const PolicyHow& how, cudaStream_t stream) {
  return by_type(a.type, [&](auto type) {
    return by_flag(a.entropies != nullptr, [&](auto entropy) {
      return by_flag(a.grad_logits != nullptr, [&](auto gradient) {
        using T = decltype(type);
        constexpr bool E = decltype(entropy)::value, G = decltype(gradient)::value;
        if (is_short(a.n, a.type)) {
          const int64_t grid = (a.rows + SHORT_THREADS / 32 - 1) / (SHORT_THREADS / 32);
          return launch_kernel(k_logprobs_short<T, E, G>, dim3(static_cast<unsigned>(grid)), dim3(SHORT_THREADS), 0, stream, a, how);
        }
        const int parts = cluster_for(a.rows, a.n, a.type);
        return launch_clusters(k_logprobs<T, E, G>, a.rows * parts, THREADS, parts, 0, stream, a, how);
      });
    });
  });
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t stream) { return launch_rows(a, PolicyHow{}, stream); }

cudaError_t launch_token_logprobs_backward(const LogprobBackwardArgs& a, cudaStream_t stream) {
  return by_type(a.type, [&](auto type) {
    return by_flag(a.grad_entropies != nullptr, [&](auto entropy) {
      using T = decltype(type);
      constexpr bool E = decltype(entropy)::value;
      if (is_short(a.n, a.type)) {
        const int64_t grid = (a.rows + SHORT_THREADS / 32 - 1) / (SHORT_THREADS / 32);
        return launch_kernel(k_logprobs_backward_short<T, E>, dim3(static_cast<unsigned>(grid)), dim3(SHORT_THREADS), 0, stream, a);
      }
      int64_t parts = 1;
      while (parts < 64 && a.rows * parts < 8 * sms() && row_bytes(a.n, a.type) / (parts * 2) >= 16384) parts *= 2;
      return launch_kernel(k_logprobs_backward<T, E>, dim3(static_cast<unsigned>(a.rows * parts)), dim3(THREADS), 0, stream, a,
                           static_cast<int>(parts));
    });
  });
}

cudaError_t launch_policy_loss(const LogprobArgs& a, const PolicyHow& how, const PolicyOut& out, cudaStream_t stream) {
  cudaError_t err = a.rows > 0 ? launch_rows(a, how, stream) : cudaSuccess;
  if (err != cudaSuccess) return err;
  const int cluster = a.rows > JOIN_THREADS ? JOIN_CLUSTER : 1;
  return launch_clusters(k_policy_join, cluster, JOIN_THREADS, cluster, 0, stream, a, how, out);
}

cudaError_t launch_preference_loss(const LogprobArgs& a, const PreferenceHow& how, const PreferenceOut& out, cudaStream_t stream) {
  cudaError_t err = a.rows > 0 ? launch_rows(a, PolicyHow{}, stream) : cudaSuccess;
  if (err != cudaSuccess) return err;
  const int64_t pairs = a.sequences / 2;
  const int team = pairs >= 4 * JOIN_CLUSTER ? 32 : JOIN_THREADS;
  const int cluster = pairs * team > JOIN_THREADS ? JOIN_CLUSTER : 1;
  return launch_clusters(k_preference_join, cluster, JOIN_THREADS, cluster, 0, stream, a, how, out, team);
}

}  // namespace profk
