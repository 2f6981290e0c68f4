// Log-probabilities of given tokens from logits, the gradient, and the losses on them:
// the clipped policy loss (perhaps with its gradient in the same launch) and the
// preference loss of pairs.
//
// With c = log2(e) / T, m the row's largest logit, x_i = (l_i - m) c, s = sum 2^x_i and
// t = sum x_i 2^x_i:
//   logprob = ln 2 x_token - ln s,   H = ln s - ln 2 t / s,
//   d(g logprob + h H) / d l_i = [g 1(i = token) - p_i (g + h ln 2 (x_i - t / s))] / T,  p_i = 2^x_i / s.
//
// A row is taken by a CTA or a cluster of them (k_logprobs) or, where it is short, by a warp
// (k_logprobs_short): one pass with a running maximum and sums, one exchange.  A policy
// loss with its gradient keeps the row in shared memory between its sums and its gradient
// (k_policy_keep); only rows beyond 8 x 112 KB are read twice.  The sums over rows are a small
// kernel of their own, and the gradient of the rest is one (k_logprobs_backward): from
// saved maxima and sums, a row read and written once.
//
// What bounds it (device times by captured calls, inputs beyond L2; MB are what has to move):
//   many rows: memory.  4096 x 131072 bfloat16 forward 163 us (1074 MB, 6.6 TB/s), with policy loss
//     and gradient 335 (2148 MB, 6.4 TB/s), and 478 when the row was read a second time: L2 kept nothing
//     of what 608 CTAs had in work.  Forward and backward of 1500 x 128003 float32 347 (2304 MB, 6.6 TB/s).
//   entropies of 16-bit logits, more so into a gradient that stands otherwise to the 16-byte boundaries:
//     instructions.  600 x 100001 float16 issues 2.9 of 4 a cycle at 45 % of the memory's rate;
//     1001 of them 81 us (370 MB, 4.6 TB/s), 264 with single stores.
//   rows of 10 to 60 KB: a CTA's beginning and end, 4 to 5 us of which eight on an SM hide most.
//     1000 x 16384 bfloat16 forward 9.4 us (33 MB), 12.5 by CTAs of 256 threads.
//   few rows: latency.  1 x 32768 2.9 us, of which the launch is 2.5; 16 of them with policy loss and gradient 6.6.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cooperative_groups.h>

#include "../../include/profk.h"
#include "lm.h"
#include "logprobs.cuh"
#include "tcgen05.cuh"

namespace cg = cooperative_groups;

namespace profk {
namespace {

constexpr int THREADS = 128;    // of a CTA that takes a row or a part of one
constexpr int WARPS = THREADS / 32;
constexpr int SHORT_THREADS = 256;  // of a CTA whose warps take a row each
constexpr int SHORT_PER_SM = 4;     // such CTAs on an SM
constexpr int LOADS = 4;        // 16-byte loads of a thread before it looks at what came
constexpr int KEEP_LOADS = 4;   // the same from shared memory
constexpr int MAX_CLUSTER = 8;

// ---------------------------------------------------------------------------
// 16 bytes of a row.

template <typename T>
constexpr int PER_VECTOR = 16 / int(sizeof(T));

// Pair i of the elements in v.  BOUNDED: with -inf, and what is below LOWEST, as LOWEST (by one instruction
// for two elements of 16 bits).
template <typename T>
constexpr float LOWEST = -INFINITY;
template <>
constexpr float LOWEST<__nv_bfloat16> = -0x1p40f;
template <>
constexpr float LOWEST<__half> = -65504.f;

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
template <typename T, bool BOUNDED>
__device__ __forceinline__ Pair element_pair(const uint4& v, int i) {
  if constexpr (sizeof(T) == 4) {
    return i == 0 ? pair(__uint_as_float(v.x), __uint_as_float(v.y)) : pair(__uint_as_float(v.z), __uint_as_float(v.w));
  } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    uint32_t w = word(v, i);
    if (BOUNDED) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(w), "r"(0xd380d380u));
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    uint32_t w = word(v, i);
    if (BOUNDED) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(w) : "r"(w), "r"(0xfbfffbffu));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pair(f.x, f.y);
  }
}

// Whether LOWEST may stand for -inf: it has no mass by this centre, and a finite exponent.
template <typename T>
__device__ __forceinline__ bool lowest_will_do(const Centre& at) {
  return sizeof(T) == 2 && at.fused && (at.m - LOWEST<T>) * at.c > 200.f && at.c < 0x1p27f;
}

// The largest of all elements (NaN is passed over).
template <int COUNT>
__device__ __forceinline__ float largest(const uint4 (&v)[COUNT], float) {
  float m = -INFINITY;
#pragma unroll
  for (int u = 0; u < COUNT; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, __uint_as_float(word(v[u], i)));
  return m;
}
template <typename H2, int COUNT>
__device__ __forceinline__ float largest_half(const uint4 (&v)[COUNT]) {
  H2 m;
#pragma unroll
  for (int u = 0; u < COUNT; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = word(v[u], i);
      const H2 h = *reinterpret_cast<const H2*>(&w);
      m = u + i == 0 ? h : __hmax2(m, h);
    }
  return fmaxf(lm_float(m.x), lm_float(m.y));
}
template <int COUNT>
__device__ __forceinline__ float largest(const uint4 (&v)[COUNT], __nv_bfloat16) {
  return largest_half<__nv_bfloat162>(v);
}
template <int COUNT>
__device__ __forceinline__ float largest(const uint4 (&v)[COUNT], __half) {
  return largest_half<__half2>(v);
}

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

// One chunk of elements joins what has been seen.  LONG: what additions lose is kept.
template <typename T, bool ENTROPY, bool LONG, int COUNT>
__device__ __forceinline__ void take(Running& r, const uint4 (&v)[COUNT], float c) {
  const float m = fmaxf(r.m, largest(v, T{}));
  const float d = shrink(r.m, m, c), f = lm_exp2(d);
  if (ENTROPY) {
    r.t = f * (r.t + d * r.s);
    if (LONG) r.t_lost = f * (r.t_lost + d * r.s_lost);
  }
  r.s *= f;
  if (LONG) r.s_lost *= f;
  r.m = m;
  const Centre at(m, c);
  Pair s[2] = {0, 0}, t[2] = {0, 0};
  // Of a -inf, x 2^x is to be 0, not inf * 0: x is bounded, or the logit has been.
  const auto add = [&](Pair x, int i, auto bounded) {
    float x0, x1;
    split(x, x0, x1);
    const Pair e = pair(lm_exp2(x0), lm_exp2(x1));
    s[i & 1] = add2(s[i & 1], e);
    if (ENTROPY) t[i & 1] = fma2(decltype(bounded)::value ? x : pair(fmaxf(x0, NO_MASS), fmaxf(x1, NO_MASS)), e, t[i & 1]);
  };
  const Pair by = pair(at.by, at.by), cc = pair(c, c);
  if (ENTROPY && lowest_will_do<T>(at)) {
#pragma unroll
    for (int u = 0; u < COUNT; ++u)
#pragma unroll
      for (int i = 0; i < PER_VECTOR<T> / 2; ++i) add(fma2(element_pair<T, true>(v[u], i), cc, by), i, std::true_type{});
  } else if (at.fused) {
#pragma unroll
    for (int u = 0; u < COUNT; ++u)
#pragma unroll
      for (int i = 0; i < PER_VECTOR<T> / 2; ++i) add(fma2(element_pair<T, false>(v[u], i), cc, by), i, std::false_type{});
  } else {
#pragma unroll
    for (int u = 0; u < COUNT; ++u)
#pragma unroll
      for (int i = 0; i < PER_VECTOR<T> / 2; ++i) add(mul2(add2(element_pair<T, false>(v[u], i), by), cc), i, std::false_type{});
  }
  float a, b;
  if (ENTROPY) {
    split(add2(t[0], t[1]), a, b);
    if (LONG)
      add_exact(r.t, r.t_lost, a + b);
    else
      r.t += a + b;
  }
  split(add2(s[0], s[1]), a, b);
  if (LONG)
    add_exact(r.s, r.s_lost, a + b);
  else
    r.s += a + b;
}

// A single element (-inf: none).
__device__ __forceinline__ Running seen(float l, float c) {
  if (l == -INFINITY) return {-INFINITY, 0.f, 0.f, 0.f, 0.f};
  const float x = Centre(l, c).off(), e = lm_exp2(x) + (l - l);  // (NaN of NaN and +inf)
  return {fmaxf(l, -INFINITY), e, x * e, 0.f, 0.f};
}

// The pass over vectors [begin, end) of `body` by STEP threads, and this thread's single element
// (-inf: it has none).
template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ Running pass(const uint4* body, int begin, int end, int thread, float single, float c) {
  Running r = seen(single, c);
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
    take<T, ENTROPY, true>(r, v, c);
  }
  return r;
}

// The same over all of `count` vectors in shared memory, whose loads need no prefetch and which
// are few enough for sums in one float: KEEP_SHARED bytes are 7 additions a thread of four vectors' sums.
template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ Running pass_shared(const uint4* body, int count, int thread, float single, float c) {
  Running r = seen(single, c);
  for (int i = thread; i < count; i += KEEP_LOADS * STEP) {
    uint4 v[KEEP_LOADS];
#pragma unroll
    for (int u = 0; u < KEEP_LOADS; ++u) v[u] = i + u * STEP < count ? body[i + u * STEP] : nothing<T>();
    take<T, ENTROPY, false>(r, v, c);
  }
  return r;
}

// What a row's gradient is made of: element i gets e (k0 + k1 x) with x by the row's centre and
// e = 2^x, and the token's element `one` besides.
struct Slopes {
  Centre at;
  float k0, k1, one;
};

// g and h: the derivatives of the result by the row's log-probability and its entropy; mean_x =
// t / s.
template <bool ENTROPY>
__device__ __forceinline__ Slopes slopes_of(float m, float s, float mean_x, float temperature, float c, float g, float h) {
  const float per_T = 1.f / temperature;
  Slopes y{Centre(m, c), 0.f, 0.f, g * per_T};
  if (s == 0.f) {  // nothing to put on any token
    y.one = 0.f;
    return y;
  }
  const float r = y.at.off(), scale = per_T / (s * lm_exp2(r));
  y.k0 = -(ENTROPY ? g - h * LN2 * (mean_x + r) : g) * scale;
  if (ENTROPY) y.k1 = -h * LN2 * scale;
  return y;
}

template <bool ENTROPY>
__device__ __forceinline__ float slope_at(const Slopes& k, float l) {
  const float x = k.at(l), e = lm_exp2(x);
  return e * (ENTROPY ? fmaf(k.k1, fmaxf(x, NO_MASS), k.k0) : k.k0);
}

// 16 bytes from anywhere: words, of which half-words are put together where `odd` says that p does
// not stand on one (then from the word before p to the one behind).
__device__ __forceinline__ uint4 load_words(const char* p, bool odd) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p - (odd ? 2 : 0));
  uint4 v = make_uint4(w[0], w[1], w[2], w[3]);
  if (odd) {
    v.x = __funnelshift_r(v.x, v.y, 16);
    v.y = __funnelshift_r(v.y, v.z, 16);
    v.z = __funnelshift_r(v.z, v.w, 16);
    v.w = __funnelshift_r(v.w, w[4], 16);
  }
  return v;
}

// The gradient of `count` elements from `p` (in global or in shared memory) to `out`, by STEP
// threads; `token` is the token's place among them, out of range where it is none.  Where p and
// out stand differently to the 16-byte boundaries, 16 bytes of the gradient come from p's words.
// (p may be out: an element is read by the thread that writes it.)
template <typename T, bool ENTROPY, int STEP, int COUNT = LOADS>
__device__ __forceinline__ void write_gradient(const T* p, T* out, int count, int thread, int token, const Slopes& k) {
  constexpr int N = PER_VECTOR<T>, SIZE = sizeof(T);
  int head = min(static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out) & 15)) & 15) / SIZE, count);
  int vectors = (count - head) / N;
  const bool same = (reinterpret_cast<uintptr_t>(p + head) & 15) == 0, odd = (reinterpret_cast<uintptr_t>(p + head) & 3) != 0;
  if (odd) {  // (nothing outside the elements is read: the first or last vector may be left to single threads)
    if (vectors > 0 && head == 0) {
      head = N;
      --vectors;
    }
    if (vectors > 0 && head + vectors * N == count) --vectors;
  }
  const int tail = count - head - vectors * N;
  const int single = thread < head ? thread : thread >= 16 && thread < 16 + tail ? head + vectors * N + thread - 16 : -1;
  if (single >= 0) out[single] = lm_cast<T>(slope_at<ENTROPY>(k, lm_float(p[single])) + (single == token ? k.one : 0.f));
  const char* from = reinterpret_cast<const char*>(p + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  // The token's element is written once more by the thread that has its vector.
  const int place = token - head;
  const bool has_token = place >= 0 && place < vectors * N && (place / N) % STEP == thread;
  const float token_slope = has_token ? slope_at<ENTROPY>(k, lm_float(p[token])) + k.one : 0.f;
  const Pair by = pair(k.at.by, k.at.by), cc = pair(k.at.c, k.at.c), k0 = pair(k.k0, k.k0), k1 = pair(k.k1, k.k1);
  const bool bounded = ENTROPY && lowest_will_do<T>(k.at) && fabsf(k.k1 * fmaf(LOWEST<T>, k.at.c, k.at.by)) < INFINITY;
  for (int i = thread; i < vectors; i += COUNT * STEP) {
    uint4 v[COUNT];
    if (same) {
#pragma unroll
      for (int u = 0; u < COUNT; ++u)
        if (i + u * STEP < vectors) v[u] = reinterpret_cast<const uint4*>(from)[i + u * STEP];
    } else {
#pragma unroll
      for (int u = 0; u < COUNT; ++u)
        if (i + u * STEP < vectors) v[u] = load_words(from + int64_t(i + u * STEP) * 16, odd);
    }
#pragma unroll
    for (int u = 0; u < COUNT; ++u) {
      const int j = i + u * STEP;
      if (j >= vectors) break;
      alignas(16) T y[N];
      const auto put = [&](Pair x, int q, auto bounded) {
        float x0, x1, y0, y1;
        split(x, x0, x1);
        const Pair e = pair(lm_exp2(x0), lm_exp2(x1));
        const Pair kept = decltype(bounded)::value ? x : pair(fmaxf(x0, NO_MASS), fmaxf(x1, NO_MASS));
        split(mul2(e, ENTROPY ? fma2(k1, kept, k0) : k0), y0, y1);
        put_pair(y + 2 * q, y0, y1);
      };
      if (bounded) {
#pragma unroll
        for (int q = 0; q < N / 2; ++q) put(fma2(element_pair<T, true>(v[u], q), cc, by), q, std::true_type{});
      } else if (k.at.fused) {
#pragma unroll
        for (int q = 0; q < N / 2; ++q) put(fma2(element_pair<T, false>(v[u], q), cc, by), q, std::false_type{});
      } else {
#pragma unroll
        for (int q = 0; q < N / 2; ++q) put(mul2(add2(element_pair<T, false>(v[u], q), by), cc), q, std::false_type{});
      }
      to[j] = *reinterpret_cast<const uint4*>(y);
    }
  }
  if (has_token) out[token] = lm_cast<T>(token_slope);
}

// A part's elements: its vectors, and the row's first and last ones where it is the first or last part.
template <typename T>
struct Span {
  int first, count;
  __device__ __forceinline__ Span(const Layout<T>& at, int begin, int end, bool is_first, bool is_last) {
    first = is_first ? 0 : at.head + begin * PER_VECTOR<T>;
    count = at.head + end * PER_VECTOR<T> + (is_last ? at.tail : 0) - first;
  }
};

// The place of a row's token in a span, -1 where the row has none.
__device__ __forceinline__ int place_in(int64_t token, int64_t n, int first) {
  return token < n ? static_cast<int>(token) - first : -1;
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

__device__ __forceinline__ bool row_live(const LogprobArgs& a, int64_t row) {
  bool live = a.tokens[row] >= 0;
  if (a.weights && a.weights[row] == 0.f) live = false;
  if (a.offsets && (row < a.offsets[0] || row >= a.offsets[a.sequences])) live = false;
  return live;
}

// All but the token's logit.
template <bool GRADIENT>
__device__ __forceinline__ Row<GRADIENT> load_inputs(const LogprobArgs& a, const PolicyHow& how, int64_t row) {
  Row<GRADIENT> r;
  r.logit = 0.f;
  r.token = a.tokens[row];
  r.temperature = a.temperature ? a.temperature[row] : a.all_temperature;
  r.c = inverse_temperature(r.temperature);
  r.live = row_live(a, row);
  if (GRADIENT) {
    r.old_lp = how.old_logprobs[row];
    r.advantage = how.advantages[row];
    r.ref_lp = how.ref_logprobs ? how.ref_logprobs[row] : 0.f;
    r.weight = how.weights ? how.weights[row] : how.all_weight;
  }
  return r;
}

template <typename T, bool GRADIENT>
__device__ __forceinline__ void load_logit(Row<GRADIENT>& r, const T* p, int n) {
  r.logit = r.live && r.token < n ? lm_float(p[r.token]) : NAN;  // (a token that the vocabulary has not is no number)
}

__device__ __forceinline__ void store_left_out(const LogprobArgs& a, int64_t row) {
  a.logprobs[row] = 0.f;
  if (a.entropies) a.entropies[row] = 0.f;
  if (a.stats) a.stats[row] = make_float2(0.f, 0.f);
  if (a.lacks) a.lacks[row] = 0.f;
}

__device__ __forceinline__ float store_row(const LogprobArgs& a, int64_t row, const RowSum& y, float logit, float temperature, bool write) {
  float lacks;
  const float lp = row_logprob(y, logit, temperature, lacks);
  if (write) {
    a.logprobs[row] = lp;
    if (a.entropies) a.entropies[row] = row_entropy(y);
    if (a.stats) a.stats[row] = make_float2(y.m, y.s);
    if (a.lacks) a.lacks[row] = lacks;
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

// The exchange of the warps' sums within a cluster: each CTA has room for those of all, written
// there by stores that count on its barrier.  (No fence over what threads have written
// before, as a barrier of the cluster would be.)  A CTA leaves when all stores to it have come; one whose wait
// ran out could be gone when they do.  The longest part, 512 MB, takes 0.1 s where all SMs read at once, and a wait
// WAIT_POLLS polls of 3.8 us: 16 s.
template <int COUNT>  // warps of a CTA
struct Exchange {
  RowSum sums[MAX_CLUSTER * COUNT];
  uint64_t all;
  int given_up;

  // By one thread, before the cluster's first barrier.
  __device__ __forceinline__ void begin(int parts) {
    barrier_init(&all, 1);
    given_up = 0;
    barrier_init_done();
    barrier_arrive_expect(&all, parts * COUNT * sizeof(RowSum));
  }
  // By all threads, once every CTA of the cluster has begun: the row's sums, the same in
  // every warp; by m itself.  The logit of the row's token comes from the first warp of all: whoever
  // writes a gradient over the logits does so after it has been read.
  template <bool ENTROPY>
  __device__ __forceinline__ RowSum join(RowSum y, float& logit, float c, int parts, int rank) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < parts) store_remote(&sums[rank * COUNT + warp], make_float4(y.m, y.s, y.t, logit), &all, lane);
    if (!__all_sync(FULL_MASK, barrier_wait<true>(&all, 0, &given_up, WAIT_POLLS))) return {0.f, NAN, NAN, NAN};
    logit = sums[0].logit;
    y = {-INFINITY, 0.f, 0.f, 0.f};
    for (int i = lane; i < parts * COUNT; i += 32) y = joined(y, sums[i], c);
    y = centred(warp_join<ENTROPY>(y, c), c);
    if (!(c > 0.f)) y.s = NAN;
    return y;
  }
};

template <typename T, bool ENTROPY, bool GRADIENT>
__global__ void __launch_bounds__(THREADS, 8) k_logprobs(LogprobArgs a, PolicyHow how) {
  pdl_wait();
  pdl_trigger();  // (behind it: what follows may read what this reads)
  __shared__ Exchange<WARPS> exchange;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / parts;
  const int thread = threadIdx.x, n = static_cast<int>(a.n);
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  Row<GRADIENT> r = load_inputs<GRADIENT>(a, how, row);
  if (rank == 0 && thread < 32) load_logit(r, p, n);
  if (!r.live) {  // the same for the whole cluster: none of it waits
    if (rank == 0 && thread == 0) store_left_out(a, row);
    if (GRADIENT) {
      const Layout<T> to(out, n);
      write_zeros<T, THREADS>(out, to, part_begin(to.vectors, rank, parts), part_begin(to.vectors, rank + 1, parts), thread,
                              to.single(thread, rank == 0, rank == parts - 1));
    }
    return;
  }
  if (thread == 0) exchange.begin(parts);
  __syncthreads();
  cluster_begin();
  const Layout<T> at(p, n);
  const int begin = part_begin(at.vectors, rank, parts), end = part_begin(at.vectors, rank + 1, parts);
  const int single = at.single(thread, rank == 0, rank == parts - 1);
  const float alone = single >= 0 ? lm_float(p[single]) : -INFINITY;
  RowSum y = warp_join<ENTROPY>(total(pass<T, ENTROPY, THREADS>(reinterpret_cast<const uint4*>(p + at.head), begin, end, thread, alone, r.c)), r.c);
  cluster_begun();
  y = exchange.template join<ENTROPY>(y, r.logit, r.c, parts, rank);
  const float lp = store_row(a, row, y, r.logit, r.temperature, rank == 0 && thread == 0);
  if (GRADIENT) {
    const Slopes k = policy_slopes<ENTROPY>(r, y, lp, how);
    const Span<T> mine(at, begin, end, rank == 0, rank == parts - 1);
    write_gradient<T, ENTROPY, THREADS>(p + mine.first, out + mine.first, mine.count, thread, place_in(r.token, a.n, mine.first), k);
  }
}

// A row by a warp, which (without the gradient, where it goes on to another) has the next row's inputs on their way meanwhile.
template <typename T, bool ENTROPY, bool GRADIENT>
__global__ void __launch_bounds__(SHORT_THREADS, GRADIENT ? 3 : SHORT_PER_SM) k_logprobs_short(LogprobArgs a, PolicyHow how) {
  pdl_wait();
  pdl_trigger();  // (behind it: what follows may read what this reads)
  const int lane = threadIdx.x & 31, n = static_cast<int>(a.n);
  const int64_t step = int64_t(gridDim.x) * (SHORT_THREADS / 32);
  int64_t row = int64_t(blockIdx.x) * (SHORT_THREADS / 32) + (threadIdx.x >> 5);
  Row<false> next{};
  if (!GRADIENT && row < a.rows) next = load_inputs<false>(a, how, row);
  for (; row < a.rows; row += step) {
    Row<GRADIENT> r;
    if constexpr (GRADIENT)
      r = load_inputs<true>(a, how, row);
    else
      r = next;
    const T* p = static_cast<const T*>(a.logits) + row * a.ld;
    T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
    load_logit(r, p, n);
    if (!GRADIENT && row + step < a.rows) next = load_inputs<false>(a, how, row + step);
    if (!r.live) {
      if (lane == 0) store_left_out(a, row);
      if (GRADIENT) {
        const Layout<T> to(out, n);
        write_zeros<T, 32>(out, to, 0, to.vectors, lane, to.single(lane, true, true));
      }
      continue;
    }
    const Layout<T> at(p, n);
    const int single = at.single(lane, true, true);
    const float alone = single >= 0 ? lm_float(p[single]) : -INFINITY;
    RowSum y = warp_join<ENTROPY>(total(pass<T, ENTROPY, 32>(reinterpret_cast<const uint4*>(p + at.head), 0, at.vectors, lane, alone, r.c)), r.c);
    y = centred(y, r.c);
    if (!(r.c > 0.f)) y.s = NAN;
    const float lp = store_row(a, row, y, r.logit, r.temperature, lane == 0);
    if (GRADIENT) {
      const Slopes k = policy_slopes<ENTROPY>(r, y, lp, how);
      write_gradient<T, ENTROPY, 32>(p, out, n, lane, place_in(r.token, a.n, 0), k);
    }
  }
}

// ---------------------------------------------------------------------------
// The policy loss with its gradient, a row by a cluster whose CTAs keep their parts of it in
// shared memory: the row is read from memory once, and its sums and its gradient are both
// made from the copy.  Many such CTAs share an SM, so that some copy while others work.
constexpr int KEEP_SHARED = 112 * 1024;  // dynamic shared memory at most
static_assert(sizeof(Exchange<8>) + sizeof(uint64_t) <= STATIC_ROOM, "static shared memory of k_policy_keep");

template <typename T, bool ENTROPY, int KEEP_THREADS>
__global__ void __launch_bounds__(KEEP_THREADS, 1024 / KEEP_THREADS) k_policy_keep(LogprobArgs a, PolicyHow how) {
  extern __shared__ __align__(128) uint8_t room[];
  __shared__ Exchange<KEEP_THREADS / 32> exchange;
  __shared__ uint64_t full;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int thread = threadIdx.x, n = static_cast<int>(a.n);
  const int64_t row = blockIdx.x / parts;
  pdl_wait();
  pdl_trigger();  // (behind it: what follows may read what this reads)
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  if (!row_live(a, row)) {  // the same for the whole cluster: none of it waits
    if (rank == 0 && thread == 0) store_left_out(a, row);
    const Layout<T> to(out, n);
    write_zeros<T, KEEP_THREADS>(out, to, part_begin(to.vectors, rank, parts), part_begin(to.vectors, rank + 1, parts), thread,
                                 to.single(thread, rank == 0, rank == parts - 1));
    return;
  }
  const Layout<T> at(p, n);
  const int begin = part_begin(at.vectors, rank, parts), end = part_begin(at.vectors, rank + 1, parts);
  if (thread == 0) {
    barrier_init(&full, 1);
    exchange.begin(parts);
    if (end > begin) {
      barrier_arrive_expect(&full, unsigned(end - begin) * 16);
      copy_bytes(room + 16, p + at.head + begin * PER_VECTOR<T>, unsigned(end - begin) * 16, &full);
    } else {
      barrier_arrive(&full);
    }
  }
  __syncthreads();
  cluster_begin();
  Row<true> r = load_inputs<true>(a, how, row);
  if (rank == 0 && thread < 32) load_logit(r, p, n);
  const Span<T> mine(at, begin, end, rank == 0, rank == parts - 1);
  T* copy = reinterpret_cast<T*>(room + 16) - (rank == 0 ? at.head : 0);  // the span's first element
  const int single = at.single(thread, rank == 0, rank == parts - 1);
  const float alone = single >= 0 ? lm_float(p[single]) : -INFINITY;
  if (single >= 0) copy[single - mine.first] = p[single];
  cluster_begun();  // (the barriers are there, in all CTAs)
  __syncthreads();  // (and so are the single elements)
  const bool there = barrier_wait(&full, 0, &exchange.given_up, WAIT_POLLS);
  RowSum y = warp_join<ENTROPY>(
      total(pass_shared<T, ENTROPY, KEEP_THREADS>(reinterpret_cast<const uint4*>(room + 16), end - begin, thread, alone, r.c)), r.c);
  if (!__all_sync(FULL_MASK, there)) y.s = NAN;
  y = exchange.template join<ENTROPY>(y, r.logit, r.c, parts, rank);
  const float lp = store_row(a, row, y, r.logit, r.temperature, rank == 0 && thread == 0);
  const Slopes k = policy_slopes<ENTROPY>(r, y, lp, how);
  write_gradient<T, ENTROPY, KEEP_THREADS, KEEP_LOADS>(copy, out + mine.first, mine.count, thread, place_in(r.token, a.n, mine.first), k);
  if (thread == 0 && exchange.given_up) {  // a copy that was not waited for must not outlive the CTA
    int nobody = 0;
    barrier_wait(&full, 0, &nobody, WAIT_POLLS);
  }
}

// ---------------------------------------------------------------------------
// The gradient from a forward pass's row sums: `parts` CTAs a row, or a warp a row.
struct BackwardRow {
  int64_t token;
  float g, h, temperature, entropy;
  float2 stats;
};

template <bool ENTROPY>
__device__ __forceinline__ BackwardRow backward_inputs(const LogprobBackwardArgs& a, int64_t row) {
  BackwardRow r;
  r.token = a.tokens[row];
  r.g = a.grad_logprobs ? a.grad_logprobs[row] : 0.f;
  r.h = ENTROPY ? a.grad_entropies[row] : 0.f;
  r.temperature = a.temperature ? a.temperature[row] : a.all_temperature;
  r.stats = a.stats[row];
  r.entropy = ENTROPY ? a.entropies[row] : 0.f;
  return r;
}

template <typename T, bool ENTROPY, int STEP>
__device__ __forceinline__ void backward_row(const LogprobBackwardArgs& a, int64_t row, const BackwardRow& r, int rank, int parts, int thread) {
  const int n = static_cast<int>(a.n);
  const T* p = static_cast<const T*>(a.logits) + row * a.ld;
  T* out = static_cast<T*>(a.grad_logits) + row * a.grad_ld;
  if (r.token < 0 || (r.g == 0.f && r.h == 0.f)) {  // left out, whatever the logits hold
    const Layout<T> to(out, n);
    write_zeros<T, STEP>(out, to, part_begin(to.vectors, rank, parts), part_begin(to.vectors, rank + 1, parts), thread,
                         to.single(thread, rank == 0, rank == parts - 1));
    return;
  }
  const float scale = a.scale ? *a.scale : 1.f;
  const float g = r.token < n ? r.g * scale : NAN, h = r.h * scale;
  const Layout<T> at(p, n);
  const float mean_x = ENTROPY ? (logf(r.stats.y) - r.entropy) * LOG2E : 0.f;
  const Slopes k = slopes_of<ENTROPY>(r.stats.x, r.stats.y, mean_x, r.temperature, inverse_temperature(r.temperature), g, h);
  const Span<T> mine(at, part_begin(at.vectors, rank, parts), part_begin(at.vectors, rank + 1, parts), rank == 0, rank == parts - 1);
  write_gradient<T, ENTROPY, STEP>(p + mine.first, out + mine.first, mine.count, thread, place_in(r.token, n, mine.first), k);
}

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(THREADS, 8) k_logprobs_backward(LogprobBackwardArgs a, int parts) {
  pdl_trigger();
  pdl_wait();
  // From the last row on: of what the forward pass has read, that is what L2 still holds.
  const int64_t row = a.rows - 1 - blockIdx.x / parts;
  backward_row<T, ENTROPY, THREADS>(a, row, backward_inputs<ENTROPY>(a, row), static_cast<int>(blockIdx.x % parts), parts, threadIdx.x);
}

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(SHORT_THREADS, SHORT_PER_SM) k_logprobs_backward_short(LogprobBackwardArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t step = int64_t(gridDim.x) * (SHORT_THREADS / 32);
  int64_t back = int64_t(blockIdx.x) * (SHORT_THREADS / 32) + (threadIdx.x >> 5);  // rows from the last on
  BackwardRow next{};
  if (back < a.rows) next = backward_inputs<ENTROPY>(a, a.rows - 1 - back);
  for (; back < a.rows; back += step) {
    const BackwardRow r = next;
    if (back + step < a.rows) next = backward_inputs<ENTROPY>(a, a.rows - 1 - back - step);
    backward_row<T, ENTROPY, 32>(a, a.rows - 1 - back, r, 0, 1, threadIdx.x & 31);
  }
}

// ---------------------------------------------------------------------------
// The sums over rows: floats with their losses carried along (double precision takes
// several times as long here), in a fixed order: the same call gives the same bits.  One cluster has them all, which
// shows where rows are many and short: of 2^20 rows of 64 a policy loss takes 863 us, 222 of them the join.
//
// These kernels follow the one that writes the log-probabilities, which lets them start
// once it has begun itself, that is once all before it is done: what the user gave can be read
// before pdl_wait, only what that kernel writes comes after it.

constexpr int JOIN_THREADS = 512;
constexpr int JOIN_WARPS = JOIN_THREADS / 32;
constexpr int JOIN_CLUSTER = 8;

struct Sum {
  float v = 0.f, lost = 0.f;
  __device__ __forceinline__ void add(float x) { add_exact(v, lost, x); }
  __device__ __forceinline__ void add(const Sum& x) {
    add_exact(v, lost, x.v);
    lost += x.lost;
  }
  // Of an infinite or NaN sum the losses are NaN, and do not count.
  __device__ __forceinline__ float value() const { return fabsf(v) < INFINITY ? v + lost : v; }
};

__device__ __forceinline__ Sum warp_sum(Sum x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Sum y;
    y.v = __shfl_xor_sync(FULL_MASK, x.v, d);
    y.lost = __shfl_xor_sync(FULL_MASK, x.lost, d);
    x.add(y);
  }
  return x;
}

// Sums over the cluster of COUNT values a thread, to thread 0 of CTA 0.  All threads call it.
template <int COUNT>
__device__ __forceinline__ void cluster_sum(Sum (&x)[COUNT]) {
  __shared__ Sum part[COUNT][JOIN_CLUSTER * JOIN_WARPS];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), parts = static_cast<int>(cluster.num_blocks());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (parts > 1) cluster.sync();  // (a CTA's shared memory is written once it runs)
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    x[i] = warp_sum(x[i]);
    if (lane == 0) cluster.map_shared_rank(&part[i][0], 0)[rank * JOIN_WARPS + warp] = x[i];
  }
  if (parts > 1)
    cluster.sync();
  else
    __syncthreads();
  if (rank != 0 || warp != 0) return;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    x[i] = Sum{};
    for (int k = lane; k < parts * JOIN_WARPS; k += 32) x[i].add(part[i][k]);
    x[i] = warp_sum(x[i]);
  }
}

// What the user gave for a token.
struct TokenInputs {
  float weight, old_lp, advantage, ref_lp;
  bool live;
};

__device__ __forceinline__ TokenInputs token_inputs(const LogprobArgs& a, const PolicyHow& how, int64_t row) {
  TokenInputs y;
  y.weight = how.weights ? how.weights[row] : how.all_weight;
  y.old_lp = how.old_logprobs[row];
  y.advantage = how.advantages[row];
  y.ref_lp = how.ref_logprobs ? how.ref_logprobs[row] : 0.f;
  y.live = a.tokens[row] >= 0 && y.weight != 0.f;
  return y;
}

__global__ void __launch_bounds__(JOIN_THREADS) k_policy_join(LogprobArgs a, PolicyHow how, PolicyOut out) {
  constexpr int AHEAD = 4;  // rows whose inputs are on their way at once
  const int64_t step = int64_t(gridDim.x) * JOIN_THREADS;
  int64_t row = int64_t(blockIdx.x) * JOIN_THREADS + threadIdx.x;
  TokenInputs in[AHEAD];
  const auto load = [&] {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (row + i * step < a.rows) in[i] = token_inputs(a, how, row + i * step);
  };
  load();
  pdl_wait();
  pdl_trigger();
  Sum sums[4];  // loss, KL terms, clipped weights, entropies
  while (row < a.rows) {
    float lp[AHEAD], H[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const bool there = row + i * step < a.rows;
      lp[i] = there ? a.logprobs[row + i * step] : 0.f;
      H[i] = there && a.entropies ? a.entropies[row + i * step] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (row + i * step >= a.rows) break;
      float slope = 0.f, h = 0.f;
      if (in[i].live) {
        const PolicyTerm term = policy_term(lp[i], in[i].old_lp, in[i].advantage, how.ref_logprobs != nullptr, in[i].ref_lp, how);
        sums[0].add(in[i].weight * (how.entropy != 0.f ? fmaf(-how.entropy, H[i], term.loss) : term.loss));
        sums[1].add(in[i].weight * term.kl);
        sums[2].add(term.clipped ? in[i].weight : 0.f);
        sums[3].add(in[i].weight * H[i]);
        slope = in[i].weight * term.slope;
        h = -how.entropy * in[i].weight;
      }
      out.slopes[row + i * step] = slope;
      if (out.entropy_slopes) out.entropy_slopes[row + i * step] = h;
    }
    row += AHEAD * step;
    load();
  }
  cluster_sum(sums);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *out.loss = sums[0].value();
#pragma unroll
    for (int i = 0; i < 3; ++i) out.sums[i] = sums[i + 1].value();
  }
}

// log(1 + exp v)
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// Whether no offset falls or leaves the rows, for all threads of the CTA.  (Of offsets that fall, two sequences that are in
// order by themselves may share rows, and two teams their slopes: every CTA looks at all of them before any row.)
__device__ __forceinline__ bool offsets_sound(const LogprobArgs& a) {
  bool sound = a.offsets[0] >= 0 && a.offsets[a.sequences] <= a.rows;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < a.sequences; i += JOIN_THREADS) sound &= a.offsets[i] <= a.offsets[i + 1];
  return __syncthreads_and(sound);
}

// A pair by a team of TEAM threads (a warp, or the CTA): its margin, its term of the loss
// and its rows' slopes.
template <int TEAM>
__global__ void __launch_bounds__(JOIN_THREADS) k_preference_join(LogprobArgs a, PreferenceHow how, PreferenceOut out) {
  __shared__ Sum across[2][JOIN_WARPS];
  __shared__ int across_live[2][JOIN_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, thread = threadIdx.x % TEAM;
  const int64_t pairs = a.sequences / 2, teams = int64_t(gridDim.x) * (JOIN_THREADS / TEAM);
  const int64_t first = int64_t(blockIdx.x) * (JOIN_THREADS / TEAM) + threadIdx.x / TEAM;
  bool waited = a.rows == 0;  // (no kernel went before that let this one start)
  if (waited) pdl_wait();
  Sum loss[1];
  if (pairs > 0 && !offsets_sound(a)) {  // nothing is known of any sequence (and all CTAs leave)
    if (!waited) pdl_wait();
    pdl_trigger();
    const int64_t step = int64_t(gridDim.x) * JOIN_THREADS, index = int64_t(blockIdx.x) * JOIN_THREADS + threadIdx.x;
    for (int64_t pair = index; pair < pairs; pair += step) out.margins[pair] = NAN;
    for (int64_t row = index; row < a.rows; row += step)
      if (row_live(a, row)) out.slopes[row] = NAN;
    if (index == 0) *out.loss = NAN;
    return;
  }
  // (A team of the whole CTA goes round together: the bound is the same for all of it.)
  for (int64_t pair = first; pair < pairs; pair += teams) {
    Sum sum[2];
    int live[2];
    int64_t edge[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) edge[i] = a.offsets[2 * pair + i];
    live[0] = live[1] = 0;
    if (!waited) {  // what is about to be read, on its way while the log-probabilities are not there yet
#pragma unroll
      for (int side = 0; side < 2; ++side)
        for (int64_t row = edge[side] + thread * 4; row < edge[side + 1]; row += TEAM * 4) {
          prefetch(a.tokens + row);
          if (how.ref_logprobs) prefetch(how.ref_logprobs + row);
        }
      pdl_wait();
      waited = true;
    }
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll 4
      for (int64_t row = edge[side] + thread; row < edge[side + 1]; row += TEAM) {
        const float lp = a.logprobs[row], ref = how.ref_logprobs ? how.ref_logprobs[row] : 0.f;
        if (a.tokens[row] >= 0) {
          sum[side].add(lp);
          sum[side].add(-ref);
          sum[side].lost += out.slopes[row];  // (what lp lacks: the slopes come in its place)
          ++live[side];
        }
      }
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      sum[side] = warp_sum(sum[side]);
      live[side] = __reduce_add_sync(FULL_MASK, live[side]);
    }
    if (TEAM > 32) {
      __syncthreads();  // (of the pair before, all is read)
      if (lane == 0)
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          across[side][warp] = sum[side];
          across_live[side][warp] = live[side];
        }
      __syncthreads();
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        sum[side] = warp_sum(lane < JOIN_WARPS ? across[side][lane] : Sum{});
        live[side] = __reduce_add_sync(FULL_MASK, lane < JOIN_WARPS ? across_live[side][lane] : 0);
      }
    }
    // The difference before anything is rounded to one float.
    float share[2] = {1.f, 1.f}, apart;
    if (how.average) {
#pragma unroll
      for (int side = 0; side < 2; ++side) share[side] = 1.f / static_cast<float>(max(live[side], 1));
      apart = sum[0].value() * share[0] - sum[1].value() * share[1];
    } else {
      Sum d = sum[0];
      d.add(Sum{-sum[1].v, -sum[1].lost});
      apart = d.value();
    }
    const float margin = fmaf(how.beta, apart, -how.margin);
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
      loss[0].add(term);
      out.margins[pair] = margin;
    }
    const float each = slope * (how.beta / static_cast<float>(pairs));
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll 4
      for (int64_t row = edge[side] + thread; row < edge[side + 1]; row += TEAM)
        if (a.tokens[row] >= 0) out.slopes[row] = (side ? -each : each) * share[side];
  }
  if (!waited) pdl_wait();
  pdl_trigger();
  cluster_sum(loss);
  if (blockIdx.x == 0 && threadIdx.x == 0) *out.loss = pairs ? loss[0].value() / static_cast<float>(pairs) : 0.f;
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

// Shared memory of a CTA that keeps a part of a row: its vectors, and room for single elements before and behind.
int64_t keep_bytes(int64_t n, int type, int parts) { return (row_bytes(n, type) / parts + 16 + 2 * 16 + 127) / 128 * 128; }

// Whether a warp takes a row, and not CTAs: rows up to so many bytes, more where there are rows for all warps of the
// SMs.  Microseconds by warps and by CTAs, bfloat16:
//   forward   300 x 2000 2.8, 3.3; 400 x 5001 4.1, 3.9; 2000 x 5001 7.4, 11.8; 1000 x 16384 12.8, 9.5;
//             4000 x 32768 44.9, 48.4; 2000 x 65536 50.7, 45.1
//   with the policy's gradient  300 x 2000 7.6, 7.0; 3000 x 2000 10.2, 17.9; 400 x 5001 9.3, 8.4;
//             2000 x 5001 15.0, 18.0; 1000 x 16384 25.0, 18.5
//   backward  3000 x 2000 5.3, 7.1; 400 x 5001 4.6, 3.0; 2000 x 5001 10.0, 6.9; 20000 x 5001 62, 63
int64_t short_bytes(int64_t rows, bool gradient) {
  if (gradient) return rows >= 4 * sms() ? 16384 : 2048;
  return rows >= 24 * sms() ? 65536 : rows >= 4 * sms() ? 16384 : 8192;
}
constexpr int64_t SHORT_BACKWARD = 8192;

// CTAs of warps that take rows: those that fit the SMs, or (once) one for every 8 rows.
unsigned short_grid(int64_t rows, bool once) {
  const int64_t all = (rows + SHORT_THREADS / 32 - 1) / (SHORT_THREADS / 32);
  return static_cast<unsigned>(once ? all : std::min<int64_t>(all, SHORT_PER_SM * sms()));
}

// CTAs a row, of 8 KB or more each: the number that is quickest by what a CTA was measured to take, 0.35 us of its
// SM's time for its beginning and end, and its part of the row at the memory's rate, shared with the others that run
// at once, or (fewer of them) at the 11 KB a microsecond that its own loads in flight allow.  (300 x 128000 bfloat16
// 17.4 us by two CTAs a row, 25.7 by one and 21.2 by four; 300 x 128003 float32 30.7, 47.5, 36.8;
// 1500 of them 120, 133, 129; 700 x 50001 27.7 by one, 31.4 by two; 200 x 16384 bfloat16 3.8 by two, 4.2 by one.)
int cluster_for(int64_t rows, int64_t n, int type) {
  constexpr double EACH = 0.35, RATE = 6700., OWN = 11.;  // microseconds, KB a microsecond
  const double kb = double(row_bytes(n, type)) / 1024., sm = sms(), slots = 8 * sm;
  const auto round = [&](double ctas, double part) { return ctas > 0 ? std::max(ctas * part / RATE, part / OWN) : 0.; };
  int best = 1;
  double least = INFINITY;
  for (int parts = 1; parts <= MAX_CLUSTER && (parts == 1 || kb / parts >= 8.); parts *= 2) {
    const double ctas = double(rows) * parts, full = std::floor(ctas / slots), part = kb / parts;
    const double cost = EACH * ctas / sm + full * round(slots, part) + round(ctas - full * slots, part);
    if (cost < least) {
      least = cost;
      best = parts;
    }
  }
  return best;
}

// CTAs a row of the kernel that keeps it; 0 where it does not fit.  Parts of 32 KB or less where 8 parts allow
// it (4096 x 131072 bfloat16: 332 us; of 64 KB 340), and where rows are few as many as fit the SMs.
int keep_parts(int64_t rows, int64_t n, int type) {
  const int64_t bytes = row_bytes(n, type);
  int parts = 1;
  while (parts < MAX_CLUSTER &&
         (bytes / parts > 32768 || (rows * parts * 2 <= 4 * sms() && bytes / (parts * 2) >= 8192)))
    parts *= 2;
  return keep_bytes(n, type, parts) <= KEEP_SHARED ? parts : 0;
}

cudaError_t launch_rows(const LogprobArgs& a, const PolicyHow& how, cudaStream_t stream) {
  return by_type(a.type, [&](auto type) {
    return by_flag(a.entropies != nullptr, [&](auto entropy) {
      return by_flag(a.grad_logits != nullptr, [&](auto gradient) {
        using T = decltype(type);
        constexpr bool E = decltype(entropy)::value, G = decltype(gradient)::value;
        // (With the gradient a warp that went on to another row would hold its registers' worth of others
        // back: 20000 x 2000 54 us, and 44 with a warp for every row; without it 19.8 and 21.6.)
        if (row_bytes(a.n, a.type) <= short_bytes(a.rows, G))
          return launch_kernel(k_logprobs_short<T, E, G>, dim3(short_grid(a.rows, G)), dim3(SHORT_THREADS), 0, stream, a, how);
        if constexpr (G) {
          const int keep = keep_parts(a.rows, a.n, a.type);
          if (keep)
            // (4 warps for 32 KB, 8 for more: 1000 x 16384 bfloat16 18.5 us, 19.2 by 8; 2000 x 65536 in one part 90, 98 by 4.)
            return by_flag(row_bytes(a.n, a.type) / keep <= 32768, [&](auto few) {
              constexpr int N = decltype(few)::value ? 128 : 256;
              return launch_clusters_most(k_policy_keep<T, E, N>, a.rows * keep, N, keep, keep_bytes(a.n, a.type, keep), KEEP_SHARED, stream, a, how);
            });
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
      if (row_bytes(a.n, a.type) <= SHORT_BACKWARD)
        return launch_kernel(k_logprobs_backward_short<T, E>, dim3(short_grid(a.rows, false)), dim3(SHORT_THREADS), 0, stream, a);
      // Parts of 32 KB: the last CTAs are not long alone.  (1500 x 128003 float32, forward and backward: 354 us, with parts of
      // 16 KB 383, of 128 KB 360, a row a CTA 378; 8192 x 131072 bfloat16, a third of it left out: 752, 822, 762, 770.)
      const int64_t parts = std::min(std::max<int64_t>(row_bytes(a.n, a.type) / 32768, 1), (int64_t(1) << 30) / a.rows);
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
  // A warp a pair where pairs are many or short.  (Captured alone: 8 pairs of 2 x 64 rows 6.4 us by warps; 5 of
  // 2 x 150 11.4 by warps, 8 of 2 x 512 7.5 by CTAs.)
  const int64_t pairs = a.sequences / 2;
  const bool warps = pairs >= 4 * JOIN_CLUSTER || a.rows <= 192 * pairs;
  const int cluster = pairs > (warps ? JOIN_WARPS : 1) ? JOIN_CLUSTER : 1;
  return warps ? launch_clusters(k_preference_join<32>, cluster, JOIN_THREADS, cluster, 0, stream, a, how, out)
               : launch_clusters(k_preference_join<JOIN_THREADS>, cluster, JOIN_THREADS, cluster, 0, stream, a, how, out);
}

}  // namespace profk
