// Choice of one token per row of logits.
//
// With m the largest allowed logit, x_i = (l_i - m) / T and w_i = exp(x_i),
// the kept tokens are a prefix of the library order (logits descending, ties
// by lower index): its first k, cut where the mass before a token reaches p of
// theirs, cut where w_i < min_p.  The token is argmax over the kept of
// x_i - log q_i for the given Exp(1) numbers q_i, which picks i with
// probability w_i / sum kept w (the least of independent exponential times of
// rates w_i); its log-probability is x_i - log sum kept w.
//
// Masses are summed as 64-bit integers (w scaled by a power of two up to
// 2^44, the largest that n of them cannot overflow), so that every sum is
// the same whatever order the atomics take.
#include "lm.cuh"
#include "lm.h"
#include "../../include/profk.h"

namespace profk {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BINS = 2048;
constexpr int PER = BINS / THREADS;
using u64 = unsigned long long;

struct Smem {
  unsigned count[BINS];
  unsigned lo[BINS], hi[BINS];  // 64-bit masses in two words
  u64 wc[WARPS], wm[WARPS];
  u64 red[WARPS];
  float score[WARPS];
  unsigned index[WARPS];
  int flag;
  // The crossing found by a pass.
  unsigned bin;
  u64 above_c, above_m, in_c, in_m;
};

__device__ __forceinline__ u64 warp_max64(u64 v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const u64 o = __shfl_xor_sync(FULL_MASK, v, d);
    v = o > v ? o : v;
  }
  return v;
}

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

template <bool MAX>
__device__ __forceinline__ u64 block_reduce64(u64 v, Smem& s) {
  v = MAX ? warp_max64(v) : warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 r = s.red[0];
  for (int w = 1; w < WARPS; ++w) r = MAX ? (s.red[w] > r ? s.red[w] : r) : r + s.red[w];
  return r;
}

// One row as its CTA sees it.
template <typename T>
struct Row {
  const T* logits;
  const uint32_t* mask;
  int64_t n;
  float m, inv, scale;

  __device__ __forceinline__ bool allowed(int64_t i) const { return !mask || (mask[i >> 5] >> (i & 31) & 1u); }
  __device__ __forceinline__ float logit(int64_t i) const { return lm_float(logits[i]); }
  __device__ __forceinline__ uint32_t key(int64_t i) const { return allowed(i) ? choice_key(logit(i)) : 0u; }
  __device__ __forceinline__ float x(float l) const {
    const float d = l - m;
    return l == m ? 0.f : d == -INFINITY ? -INFINITY : d * inv;
  }
  __device__ __forceinline__ u64 mass(float l) const { return __float2ull_rn(expf(x(l)) * scale); }
};

// What a selection returns: the value (or index) key where the running
// quantity reaches the target, and the sums above it and of its copies.
struct Cross {
  uint32_t key;
  u64 above_c, above_m, in_c, in_m;
};

// Radix selection over the row's items in descending key order: the key at
// which the running count (by_mass false) or mass first reaches `target`
// (1 <= target <= the total).  item(i, key, mass) says whether i takes part.
template <typename F>
__device__ Cross radix_cross(int64_t n, bool by_mass, u64 target, Smem& s, F&& item) {
  Cross c{0u, 0, 0, 0, 0};
  int shift = 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const uint32_t high = c.key;  // the resolved digits
    const int resolved = shift;
    shift -= bits;
    __syncthreads();
    for (int b = threadIdx.x; b < BINS; b += THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0u;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += THREADS) {
      uint32_t key;
      u64 mass;
      if (!item(i, key, mass)) continue;
      if (resolved < 32 && (key >> resolved) != (high >> resolved)) continue;
      const unsigned b = (key >> shift) & ((1u << bits) - 1u);
      atomicAdd(&s.count[b], 1u);
      const unsigned lo = static_cast<unsigned>(mass), old = atomicAdd(&s.lo[b], lo);
      const unsigned hi = static_cast<unsigned>(mass >> 32) + (old + lo < old ? 1u : 0u);
      if (hi) atomicAdd(&s.hi[b], hi);
    }
    __syncthreads();
    // Thread t takes bins BINS - 1 - PER t .. downwards.
    u64 tc = 0, tm = 0;
    const int top = BINS - 1 - PER * threadIdx.x;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      tc += s.count[top - j];
      tm += (u64(s.hi[top - j]) << 32) + s.lo[top - j];
    }
    u64 ic = tc, im = tm;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 oc = __shfl_up_sync(FULL_MASK, ic, d), om = __shfl_up_sync(FULL_MASK, im, d);
      if (lane >= d) {
        ic += oc;
        im += om;
      }
    }
    if (lane == 31) {
      s.wc[warp] = ic;
      s.wm[warp] = im;
    }
    __syncthreads();
    u64 bc = c.above_c + ic - tc, bm = c.above_m + im - tm;
    for (int w = 0; w < warp; ++w) {
      bc += s.wc[w];
      bm += s.wm[w];
    }
    for (int j = 0; j < PER; ++j) {
      const u64 nc = s.count[top - j], nm = (u64(s.hi[top - j]) << 32) + s.lo[top - j];
      const u64 before = by_mass ? bm : bc, with = before + (by_mass ? nm : nc);
      if (before < target && target <= with) {
        s.bin = static_cast<unsigned>(top - j);
        s.above_c = bc;
        s.above_m = bm;
        s.in_c = nc;
        s.in_m = nm;
      }
      bc += nc;
      bm += nm;
    }
    __syncthreads();
    c = Cross{high | (s.bin << shift), s.above_c, s.above_m, s.in_c, s.in_m};
  }
  return c;
}

// The candidate key down to which the first `r` copies of c.key are kept.
template <typename T>
__device__ u64 cut_key(const Row<T>& row, const Cross& c, u64 r, Smem& s) {
  const u64 base = u64(c.key) << 32;
  if (r >= c.in_c) return base;
  const Cross at = radix_cross(row.n, false, r, s, [&](int64_t i, uint32_t& key, u64& mass) {
    key = ~static_cast<uint32_t>(i);
    mass = 0;
    return row.key(i) == c.key;
  });
  return base | at.key;
}

template <typename T>
__global__ void __launch_bounds__(THREADS) k_sample_tokens(TokenArgs a) {
  __shared__ Smem s;
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const float T_ = a.temperature ? a.temperature[r] : a.all_temperature;
  const int32_t k = a.top_k ? a.top_k[r] : a.all_top_k;
  const float p = a.top_p ? a.top_p[r] : a.all_top_p;
  const float min_p = a.min_p ? a.min_p[r] : a.all_min_p;
  Row<T> row{static_cast<const T*>(a.logits) + r * a.ld, a.mask ? a.mask + r * a.mask_ld : nullptr, a.n, 0.f, 0.f, 0.f};
  // The largest key, the number of tokens that may be chosen, any NaN.
  if (threadIdx.x == 0) s.flag = 0;
  __syncthreads();
  u64 best = 0, live = 0;
  bool nan = false;
  for (int64_t i = threadIdx.x; i < a.n; i += THREADS) {
    if (!row.allowed(i)) continue;
    const float l = row.logit(i);
    nan |= isnan(l);
    const uint32_t key = choice_key(l);
    if (key == 0u) continue;
    ++live;
    const u64 c = (u64(key) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(i));
    best = c > best ? c : best;
  }
  if (nan) s.flag = 1;
  best = block_reduce64<true>(best, s);
  live = block_reduce64<false>(live, s);
  const bool bad = s.flag || !(T_ >= 0.f) || isnan(p) || isnan(min_p);
  if (bad || best == 0 || T_ == 0.f) {
    if (threadIdx.x == 0) {
      const bool none = bad || best == 0;
      a.out_tokens[r] = none ? -1 : static_cast<int64_t>(cand_index(best));
      a.out_logprobs[r] = bad ? __int_as_float(0x7fc00000) : best == 0 ? -INFINITY : 0.f;
    }
    return;
  }
  row.m = key_to_float(static_cast<uint32_t>(best >> 32));
  row.inv = 1.f / T_;
  int digits = 0;
  while ((int64_t(1) << digits) < a.n) ++digits;
  const int e = 62 - digits < 44 ? 62 - digits : 44;
  row.scale = __int_as_float((127 + e) << 23);
  auto item = [&](int64_t i, uint32_t& key, u64& mass) {
    key = row.key(i);
    if (key == 0u) return false;
    mass = row.mass(row.logit(i));
    return true;
  };
  u64 thr = 1, Z = 0;
  const bool by_k = k > 0 && static_cast<u64>(k) < live;
  if (by_k) {
    const Cross c = radix_cross(a.n, false, static_cast<u64>(k), s, item);
    const u64 copies = static_cast<u64>(k) - c.above_c;
    thr = cut_key(row, c, copies, s);
    Z = c.above_m + c.in_m / c.in_c * copies;  // copies of one value have one mass
  }
  if (p < 1.f) {
    if (!by_k) {
      for (int64_t i = threadIdx.x; i < a.n; i += THREADS) {
        uint32_t key;
        u64 mass;
        if (item(i, key, mass)) Z += mass;
      }
      Z = block_reduce64<false>(Z, s);
    }
    // Kept while the mass before is below p Z: an integer comparison.
    const double want = ceil(static_cast<double>(p) * static_cast<double>(Z));
    u64 target = want >= 1.0 ? static_cast<u64>(want) : 1ull;
    target = target < Z ? target : Z;
    const Cross c = radix_cross(a.n, true, target, s, item);
    const u64 each = c.in_m / c.in_c;
    const u64 cut = cut_key(row, c, (target - c.above_m + each - 1) / each, s);
    thr = cut > thr ? cut : thr;
  }
  // The race over the kept.
  const float floor_w = fminf(min_p, 1.f);
  float score = -INFINITY;
  unsigned index = 0xFFFFFFFFu;
  u64 kept = 0;
  for (int64_t i = threadIdx.x; i < a.n; i += THREADS) {
    const uint32_t key = row.key(i);
    if (key == 0u || ((u64(key) << 32) | static_cast<uint32_t>(~static_cast<uint32_t>(i))) < thr) continue;
    const float x = row.x(row.logit(i)), w = expf(x);
    if (w < floor_w || x == -INFINITY) continue;
    kept += __float2ull_rn(w * row.scale);
    const float v = fmaxf(x - logf(a.noise[r * a.noise_ld + i]), -INFINITY);  // NaN noise: never ahead
    if (index == 0xFFFFFFFFu || v > score) {
      score = v;
      index = static_cast<unsigned>(i);
    }
  }
  kept = block_reduce64<false>(kept, s);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float ov = __shfl_xor_sync(FULL_MASK, score, d);
    const unsigned oi = __shfl_xor_sync(FULL_MASK, index, d);
    if (oi != 0xFFFFFFFFu && (index == 0xFFFFFFFFu || ov > score || (ov == score && oi < index))) {
      score = ov;
      index = oi;
    }
  }
  if (lane == 0) {
    s.score[warp] = score;
    s.index[warp] = index;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < WARPS; ++w) {
      const unsigned oi = s.index[w];
      if (oi != 0xFFFFFFFFu && (index == 0xFFFFFFFFu || s.score[w] > score || (s.score[w] == score && oi < index))) {
        score = s.score[w];
        index = oi;
      }
    }
    // The largest logit is always kept, so an index has been found.
    a.out_tokens[r] = static_cast<int64_t>(index);
    a.out_logprobs[r] = row.x(row.logit(index)) - logf(static_cast<float>(kept) / row.scale);
  }
}

}  // namespace

cudaError_t launch_sample_tokens(const TokenArgs& a, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(a.rows)), block(THREADS);
  switch (a.type) {
    case PROFK_F32: return launch_kernel(k_sample_tokens<float>, grid, block, 0, stream, a);
    case PROFK_BF16: return launch_kernel(k_sample_tokens<__nv_bfloat16>, grid, block, 0, stream, a);
    default: return launch_kernel(k_sample_tokens<__half>, grid, block, 0, stream, a);
  }
}

}  // namespace profk
