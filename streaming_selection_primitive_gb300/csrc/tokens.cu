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
// A cluster of CTAs takes a row.  Each CTA reads its slice once, into shared
// memory where it fits, and makes its passes there:
//   1. the maximum (joined over the cluster through distributed shared memory);
//   2. for top-p the mass of the row, and for both cuts a histogram of one
//      element in 16, from which a value is taken that should lie just below
//      the last token to be kept: what follows touches only elements above it;
//   3. a histogram of counts and masses over 1024 equal ranges of keys between
//      that value and the maximum, repeated inside the range where the count or
//      the mass crosses its target until that holds at most LIST keys, which
//      every CTA ranks;
//   4. the race among the kept, the only pass that reads noise.
// Steps 2 and 3 are this library's method (sample, filter, check, refine): the
// check is the crossing itself, and where the value of step 2 turns out too
// high, step 3 runs over everything.
//
// Masses are summed as 64-bit integers (w scaled by a power of two up to
// 2^44, the largest that n of them cannot overflow), so that every sum is
// the same whatever order the atomics take.
#include <cooperative_groups.h>

#include "../../include/profk.h"
#include "lm.cuh"
#include "lm.h"

namespace cg = cooperative_groups;

namespace profk {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_CLUSTER = 8;
constexpr int BINS = 1024;     // of one histogram pass
constexpr int PER = BINS / THREADS;
constexpr int LIST = 256;      // keys that are ranked directly
constexpr int SAMPLE_BINS = 256;
constexpr float SAMPLE_SCALE = 8.f;  // bins per unit of x
constexpr int SAMPLE_EVERY = 16;
constexpr int SLICE_BYTES = 64 << 10;   // of a row in one CTA's shared memory, where the cluster is not at its largest
constexpr int SLICE_MOST = 190 << 10;   // and in any case; beyond it the passes read global memory
constexpr int SLICE_LEAST = 8 << 10;
using u64 = unsigned long long;

// The race's state: the best score, its logit and index (NONE: none yet).
struct Best {
  float score, logit;
  unsigned index;
};
constexpr unsigned NONE = 0xFFFFFFFFu;

__device__ __forceinline__ void better(Best& a, const Best& b) {
  if (b.index != NONE && (a.index == NONE || b.score > a.score || (b.score == a.score && b.index < a.index))) a = b;
}

struct Shared {
  // Written by other CTAs of the cluster.
  unsigned merged_c[BINS];
  u64 merged_m[BINS];
  u64 list[2][LIST];
  unsigned sample[SAMPLE_BINS];
  float ex_max[MAX_CLUSTER];
  u64 ex_z[MAX_CLUSTER];
  u64 ex_kept[MAX_CLUSTER];
  Best ex_best[MAX_CLUSTER];
  // This CTA's own.
  unsigned count[BINS];
  unsigned lo[BINS], hi[BINS];  // 64-bit masses in two words
  u64 sorted[LIST];
  u64 wc[WARPS], wm[WARPS], red[WARPS];
  float redf[WARPS];
  Best best[WARPS];
  unsigned slot;
  unsigned bin;  // the crossing found by a pass: BINS if there is none
  u64 above_c, above_m, in_c, total_m;
  u64 thr, z;
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max_of(const float* x, int n) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < n; ++j) top = fmaxf(top, x[j]);
  return top;
}

// log2 of a positive number by the hardware's approximation; zero gives -inf.
__device__ __forceinline__ float lm_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One row as a CTA of its cluster sees it.  Positions are counted from the
// 16-byte boundary at or before the row (`phase` elements before it); a
// vector is the VEC positions from a boundary.
template <typename T, bool RESIDENT>
struct Slice {
  static constexpr int VEC = 16 / int(sizeof(T));
  const T* row;
  const uint32_t* mask;
  uint4* store;  // the slice's vectors in shared memory (RESIDENT)
  int64_t n;     // of the row
  int64_t v0;    // first vector
  int nv;        // vectors
  int phase;
  float m, inv, inv2, scale;  // the maximum, 1 / T, log2(e) / T, the masses' unit
  int index_bits;

  // First element of a vector of the slice (may be outside the row).
  __device__ __forceinline__ int64_t element(int v) const { return (v0 + v) * VEC - phase; }

  // Bit j: element i + j of the row is allowed (VEC bits; i + VEC <= n).
  __device__ __forceinline__ unsigned allowed(int64_t i) const {
    const int at = static_cast<int>(i & 31);
    const uint32_t* w = mask + (i >> 5);
    const uint32_t hi = at + VEC > 32 ? w[1] : 0u;
    return __funnelshift_r(w[0], hi, at);
  }

  __device__ __forceinline__ bool inside(int v) const {
    const int64_t i = element(v);
    return i >= 0 && i + VEC <= n;
  }

  __device__ __forceinline__ uint4 raw(int v) const { return __ldg(reinterpret_cast<const uint4*>(row + element(v))); }

  __device__ __forceinline__ void unpack(uint4 bits, float (&x)[VEC]) const {
    union {
      uint4 bits;
      T t[VEC];
    } u;
    u.bits = bits;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = lm_float(u.t[j]);
  }

  __device__ __forceinline__ void hide(int64_t i, float (&x)[VEC]) const {
    const unsigned ok = allowed(i);
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = ok >> j & 1u ? x[j] : -INFINITY;
  }

  // A vector from global memory; elements outside the row or not allowed are -inf.
  __device__ __forceinline__ void fetch(int v, float (&x)[VEC]) const {
    const int64_t i = element(v);
    if (inside(v)) {
      unpack(raw(v), x);
      if (mask) hide(i, x);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int64_t e = i + j;
        x[j] = e >= 0 && e < n && (!mask || (mask[e >> 5] >> (e & 31) & 1u)) ? lm_float(row[e]) : -INFINITY;
      }
    }
  }

  __device__ __forceinline__ void load(int v, float (&x)[VEC]) const {
    if constexpr (RESIDENT)
      unpack(store[v], x);
    else
      fetch(v, x);
  }

  __device__ __forceinline__ void keep(int v, const float (&x)[VEC]) const {
    union {
      uint4 bits;
      T t[VEC];
    } u;
#pragma unroll
    for (int j = 0; j < VEC; ++j) u.t[j] = lm_cast<T>(x[j]);  // exact: they came from T
    store[v] = u.bits;
  }

  // (l - m) / T: a NaN (an infinite maximum less itself, 0 times an infinite
  // 1 / T) is the maximum's own, 0.
  __device__ __forceinline__ float x(float l) const { return fminf((l - m) * inv, 0.f); }
  __device__ __forceinline__ float weight(float l) const { return lm_exp2(fminf((l - m) * inv2, 0.f)); }
  __device__ __forceinline__ u64 fixed(float w) const { return __float2ull_rn(w * scale); }

  // Keys: the order key of the logit (16-bit types: its upper half) above the
  // inverted index in index_bits bits.
  static constexpr int DROP = sizeof(T) == 2 ? 13 : 0;
  __device__ __forceinline__ u64 value_key(float l) const { return u64(ord_key(l) >> DROP) << index_bits; }
  __device__ __forceinline__ u64 key(float l, int64_t i) const {
    return value_key(l) | ((u64(1) << index_bits) - 1 - static_cast<u64>(i));
  }
  __device__ __forceinline__ float logit_of(u64 key) const {
    const uint32_t ord = static_cast<uint32_t>(key >> index_bits) << DROP;
    // The dropped bits of a negative value's order key are ones.
    return key_to_float(ord & 0x80000000u ? ord : ord | ((1u << DROP) - 1u));
  }
};

__device__ __forceinline__ u64 block_sum64(u64 v, Shared& s) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 r = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) r += s.red[w];
  __syncthreads();
  return r;
}

// Histogram of the slice's keys in [lo, hi], joined over the cluster, and the
// bin where the running count (or mass) from the top first reaches `target`:
// s.bin, s.above_*, s.in_c; s.bin = BINS where it does not.  fresh: the joined
// histogram of the same range is still in place.
template <typename S>
__device__ void cross(const S& sl, Shared& s, cg::cluster_group& cluster, u64 lo, u64 hi, int shift, bool by_mass,
                      u64 target, bool fresh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!fresh) {
    for (int b = threadIdx.x; b < BINS; b += THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0u;
    __syncthreads();
    const float floor_l = sl.logit_of(lo);
    for (int v = threadIdx.x; v < sl.nv; v += THREADS) {
      float x[S::VEC];
      sl.load(v, x);
      const float top = max_of(x, S::VEC);
      if (top == -INFINITY || top < floor_l) continue;
#pragma unroll
      for (int j = 0; j < S::VEC; ++j) {
        if (x[j] == -INFINITY) continue;
        const u64 key = sl.key(x[j], sl.element(v) + j);
        if (key < lo || key > hi) continue;
        const unsigned b = static_cast<unsigned>((key - lo) >> shift);
        const u64 mass = sl.fixed(sl.weight(x[j]));
        atomicAdd(&s.count[b], 1u);
        const unsigned ml = static_cast<unsigned>(mass), old = atomicAdd(&s.lo[b], ml);
        const unsigned mh = static_cast<unsigned>(mass >> 32) + (old + ml < old ? 1u : 0u);
        if (mh) atomicAdd(&s.hi[b], mh);
      }
    }
    cluster.sync();
    // This CTA joins every C-th bin and tells everybody.
    const int C = cluster.num_blocks();
    for (int b = threadIdx.x * C + cluster.block_rank(); b < BINS; b += THREADS * C) {
      unsigned c = 0;
      u64 m = 0;
      for (int i = 0; i < C; ++i) {
        const Shared* o = cluster.map_shared_rank(&s, i);
        c += o->count[b];
        m += (u64(o->hi[b]) << 32) + o->lo[b];
      }
      for (int i = 0; i < C; ++i) {
        Shared* o = cluster.map_shared_rank(&s, i);
        o->merged_c[b] = c;
        o->merged_m[b] = m;
      }
    }
    cluster.sync();
  }
  // Thread t takes bins BINS - 1 - PER t .. downwards.
  const int top = BINS - 1 - PER * threadIdx.x;
  u64 tc = 0, tm = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    tc += s.merged_c[top - j];
    tm += s.merged_m[top - j];
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
  if (threadIdx.x == 0) s.bin = BINS;
  __syncthreads();
  u64 bc = ic - tc, bm = im - tm;
  for (int w = 0; w < warp; ++w) {
    bc += s.wc[w];
    bm += s.wm[w];
  }
  if (threadIdx.x == THREADS - 1) s.total_m = bm + tm;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const u64 nc = s.merged_c[top - j], nm = s.merged_m[top - j];
    const u64 before = by_mass ? bm : bc, with = before + (by_mass ? nm : nc);
    if (before < target && target <= with) {
      s.bin = static_cast<unsigned>(top - j);
      s.above_c = bc;
      s.above_m = bm;
      s.in_c = nc;
    }
    bc += nc;
    bm += nm;
  }
  __syncthreads();
}

__device__ __forceinline__ int shift_for(u64 lo, u64 hi) {
  int shift = 0;
  while (((hi - lo) >> shift) >= BINS) ++shift;
  return shift;
}

// The key down to which tokens are kept, s.thr (every kept key >= it), and the
// mass of those, s.z: the first `target` keys of [lo, hi] from the top, or as
// many as it takes for their mass to reach it.  False: all of [lo, hi] does
// not reach it (then s.total_m is its mass).
template <typename S>
__device__ bool select(const S& sl, Shared& s, cg::cluster_group& cluster, u64 lo, u64 hi, bool by_mass, u64 target,
                       int which, bool& fresh) {
  const int lane = threadIdx.x & 31;
  u64 above_c = 0, above_m = 0;
  for (int level = 0;; ++level) {
    const int shift = shift_for(lo, hi);
    cross(sl, s, cluster, lo, hi, shift, by_mass, target - (by_mass ? above_m : above_c), fresh && level == 0);
    if (s.bin == BINS) {
      fresh = level == 0;
      return false;
    }
    above_c += s.above_c;
    above_m += s.above_m;
    const u64 in_c = s.in_c;
    const unsigned bin = s.bin;
    lo += u64(bin) << shift;
    const u64 last = lo + ((u64(1) << shift) - 1);
    hi = last < hi ? last : hi;
    fresh = level == 0;
    if (in_c > LIST) {
      __syncthreads();  // s.bin and the rest have been read
      continue;
    }
    // Few enough: every CTA sends the keys that it has to all, after those
    // of the CTAs before it.
    const int C = cluster.num_blocks(), rank = cluster.block_rank();
    unsigned base = 0;
    for (int i = 0; i < rank; ++i) base += cluster.map_shared_rank(&s, i)->count[bin];
    if (threadIdx.x == 0) s.slot = base;
    __syncthreads();
    if (s.count[bin] != 0u) {
      const float floor_l = sl.logit_of(lo);
      for (int v = threadIdx.x; v < sl.nv; v += THREADS) {
        float x[S::VEC];
        sl.load(v, x);
        const float top = max_of(x, S::VEC);
        if (top == -INFINITY || top < floor_l) continue;
#pragma unroll
        for (int j = 0; j < S::VEC; ++j) {
          if (x[j] == -INFINITY) continue;
          const u64 key = sl.key(x[j], sl.element(v) + j);
          if (key < lo || key > hi) continue;
          const unsigned at = atomicAdd(&s.slot, 1u);
          if (at < LIST)
            for (int i = 0; i < C; ++i) cluster.map_shared_rank(&s, i)->list[which][at] = key;
        }
      }
    }
    cluster.sync();
    // Rank of each key: two threads count the larger ones of half the list each.
    const int m = static_cast<int>(in_c), item = threadIdx.x >> 1;
    const u64* list = s.list[which];
    const u64 mine = item < m ? list[item] : 0;
    int above = 0;
    for (int i = threadIdx.x & 1; i < m; i += 2) above += list[i] > mine;
    above += __shfl_xor_sync(FULL_MASK, above, 1);
    if (item < m && !(threadIdx.x & 1)) s.sorted[above] = mine;
    __syncthreads();
    if (threadIdx.x < 32) {  // one warp adds the masses up in that order
      constexpr int EACH = LIST / 32;
      u64 mass[EACH], sum = 0;
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int at = lane * EACH + j;
        mass[j] = at < m ? sl.fixed(sl.weight(sl.logit_of(s.sorted[at]))) : 0;
        sum += mass[j];
      }
      u64 before = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(FULL_MASK, before, d);
        if (lane >= d) before += o;
      }
      before = above_m + before - sum;
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int at = lane * EACH + j;
        const u64 b = by_mass ? before : above_c + at, w = b + (by_mass ? mass[j] : 1);
        if (at < m && b < target && target <= w) {
          s.thr = s.sorted[at];
          s.z = before + mass[j];
        }
        before += mass[j];
      }
    }
    __syncthreads();
    return true;
  }
}

// Where x should be cut (in bins of the sample's histogram) so that the tokens
// above hold the first k of the row, or all but a share of the mass: whole
// warp, every lane gets the answer.  SAMPLE_BINS: nowhere.
__device__ __forceinline__ int sample_cut(const unsigned* hist, bool by_k, float k, float spare) {
  constexpr int EACH = SAMPLE_BINS / 32;
  const int lane = threadIdx.x & 31;
  float v[EACH], sum = 0.f;
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int b = lane * EACH + j;
    v[j] = static_cast<float>(hist[b]);
    if (!by_k) v[j] *= SAMPLE_EVERY * __expf(-static_cast<float>(b) / SAMPLE_SCALE);
    sum += v[j];
  }
  float before = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float o = __shfl_up_sync(FULL_MASK, before, d);
    if (lane >= d) before += o;
  }
  const float total = __shfl_sync(FULL_MASK, before, 31);
  before -= sum;
  // k: four standard deviations of the sample's count above its mean, and a few.
  const float expect = k / SAMPLE_EVERY, want = expect + 4.f * sqrtf(expect) + 8.f;
  int cut = SAMPLE_BINS;
#pragma unroll
  for (int j = EACH - 1; j >= 0; --j) {
    float above = before;  // with bins up to this one
#pragma unroll
    for (int i = 0; i <= j; ++i) above += v[i];
    const int b = lane * EACH + j;
    // Mass: what the bins below hold by the sample, two more of its elements
    // at the edge, and a fifth of room.
    const float tail = total - above + 2.f * SAMPLE_EVERY * __expf(-static_cast<float>(b + 1) / SAMPLE_SCALE);
    if (by_k ? above >= want : tail <= 0.8f * spare) cut = b + 1;
  }
  return static_cast<int>(__reduce_min_sync(FULL_MASK, static_cast<unsigned>(cut)));
}

template <typename T, bool RESIDENT>
__global__ void __launch_bounds__(THREADS, 2) k_sample_tokens(TokenArgs a, int per_cta) {
  extern __shared__ __align__(16) unsigned char smem[];
  using S = Slice<T, RESIDENT>;
  constexpr int VEC = S::VEC;
  Shared& s = *reinterpret_cast<Shared*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = blockIdx.x / C;
  for (int b = threadIdx.x; b < SAMPLE_BINS; b += THREADS) s.sample[b] = s.count[b] = 0u;
  pdl_wait();
  pdl_trigger();
  const float temperature = a.temperature ? a.temperature[r] : a.all_temperature;
  const int32_t k = a.top_k ? a.top_k[r] : a.all_top_k;
  const float p = a.top_p ? a.top_p[r] : a.all_top_p;
  const float min_p = a.min_p ? a.min_p[r] : a.all_min_p;
  S sl;
  sl.row = static_cast<const T*>(a.logits) + r * a.ld;
  sl.mask = a.mask ? a.mask + r * a.mask_ld : nullptr;
  sl.store = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  sl.n = a.n;
  sl.phase = static_cast<int>(reinterpret_cast<uintptr_t>(sl.row) % 16 / sizeof(T));
  const int64_t all = (a.n + sl.phase + VEC - 1) / VEC;
  sl.v0 = static_cast<int64_t>(rank) * per_cta;
  sl.nv = static_cast<int>(all <= sl.v0 ? 0 : all - sl.v0 < per_cta ? all - sl.v0 : per_cta);

  // 1. The slice, and the largest logit (NaN if there is one).
  float top = -INFINITY;
  {
    constexpr int AHEAD = 4;  // loads under way a thread
    for (int v = threadIdx.x; v < sl.nv; v += AHEAD * THREADS) {
      uint4 bits[AHEAD];
      bool in[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int u = v + i * THREADS;
        in[i] = u < sl.nv && sl.inside(u);
        if (in[i]) bits[i] = sl.raw(u);
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int u = v + i * THREADS;
        if (u >= sl.nv) break;
        float x[VEC];
        if (in[i]) {
          sl.unpack(bits[i], x);
          if (sl.mask) sl.hide(sl.element(u), x);
        } else {
          sl.fetch(u, x);
        }
        if constexpr (RESIDENT) {
          if (in[i] && !sl.mask)
            sl.store[u] = bits[i];
          else
            sl.keep(u, x);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) top = max_nan(top, x[j]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) top = max_nan(top, __shfl_xor_sync(FULL_MASK, top, d));
  if (lane == 0) s.redf[warp] = top;
  cluster.sync();  // every CTA runs, and has cleared what others add to
  if (threadIdx.x < C) {
    top = s.redf[0];
    for (int w = 1; w < WARPS; ++w) top = max_nan(top, s.redf[w]);
    cluster.map_shared_rank(&s, threadIdx.x)->ex_max[rank] = top;
  }
  cluster.sync();
  top = s.ex_max[0];
  for (int i = 1; i < C; ++i) top = max_nan(top, s.ex_max[i]);
  const bool bad = isnan(top) || !(temperature >= 0.f) || isnan(p) || isnan(min_p);
  if (bad || top == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      a.out_tokens[r] = -1;
      a.out_logprobs[r] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
    }
    return;
  }
  sl.m = top;
  // An infinite T: the smallest number, so that -inf stays -inf.
  sl.inv = fmaxf(1.f / temperature, __int_as_float(1));
  sl.inv2 = sl.inv * LOG2E;
  int digits = 0;
  while ((int64_t(1) << digits) < a.n) ++digits;
  sl.index_bits = digits;
  const int e = 62 - digits < 44 ? 62 - digits : 44;
  sl.scale = __int_as_float((127 + e) << 23);

  const bool greedy = temperature == 0.f;
  const bool by_k = !greedy && k > 0 && k < a.n, by_p = !greedy && p < 1.f;
  u64 thr = greedy ? sl.value_key(top) : 0;  // copies of the maximum; the lowest index wins the race
  if (by_k || by_p) {
    // 2. The row's mass, and the value below which nothing should be kept.
    u64 Z = 0;
    if (!by_k) {
      for (int v = threadIdx.x; v < sl.nv;) {
        float sum = 0.f;
        for (int i = 0; i < 16 && v < sl.nv; ++i, v += THREADS) {
          float x[VEC];
          sl.load(v, x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[j] = sl.weight(x[j]);
#pragma unroll
          for (int d = VEC / 2; d; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) x[j] += x[j + d];
          sum += x[0];
        }
        Z += sl.fixed(sum);
      }
      Z = block_sum64(Z, s);
      if (threadIdx.x < C) cluster.map_shared_rank(&s, threadIdx.x)->ex_z[rank] = Z;
    }
    const bool sampled = a.n > 4096;
    if (sampled) {
      // One vector in SAMPLE_EVERY, at a place that moves along (and so spreads over the banks).
      for (int q = threadIdx.x; q * SAMPLE_EVERY < sl.nv; q += THREADS) {
        const int v = q * SAMPLE_EVERY + (q & (SAMPLE_EVERY - 1));
        if (v >= sl.nv) continue;
        float x[VEC];
        sl.load(v, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (x[j] != -INFINITY) {
            const float at = fminf(-sl.x(x[j]) * SAMPLE_SCALE, SAMPLE_BINS - 1.f);
            atomicAdd(&s.count[static_cast<int>(at)], 1u);
          }
      }
      __syncthreads();
      for (int b = threadIdx.x; b < SAMPLE_BINS * C; b += THREADS) {
        const unsigned c = s.count[b % SAMPLE_BINS];
        if (c) atomicAdd(&cluster.map_shared_rank(&s, b / SAMPLE_BINS)->sample[b % SAMPLE_BINS], c);
      }
    }
    if (sampled || !by_k) cluster.sync();
    if (!by_k) {
      Z = 0;
      for (int i = 0; i < C; ++i) Z += s.ex_z[i];
    }
    // Without a sample, or without an answer: weights below the last bin's are
    // nothing beside the maximum's.
    const int cut = sampled ? sample_cut(s.sample, by_k, static_cast<float>(k),
                                         (1.f - p) * (static_cast<float>(Z) / sl.scale))
                            : SAMPLE_BINS;
    const float at = top - temperature * (static_cast<float>(cut) / SAMPLE_SCALE);
    const u64 hi = sl.value_key(top) | ((u64(1) << sl.index_bits) - 1);
    // (A maximum of +inf, or a cut that is no number: from the bottom.)
    u64 lo = at < top && at > -INFINITY ? sl.value_key(at) : 0;

    // 3. The cuts.
    bool fresh = false, cut_k = by_k;
    if (by_k) {
      bool found = select(sl, s, cluster, lo, hi, false, static_cast<u64>(k), 0, fresh);
      if (!found && lo) {
        lo = 0;
        fresh = false;
        found = select(sl, s, cluster, lo, hi, false, static_cast<u64>(k), 0, fresh);
      }
      cut_k = found;
      Z = found ? s.z : s.total_m;  // not found: there are no more than k
      if (found) thr = s.thr;
    }
    if (by_p) {
      // Kept while the mass before is below p Z: an integer comparison.
      const double want = ceil(static_cast<double>(p) * static_cast<double>(Z));
      u64 target = want >= 1.0 ? static_cast<u64>(want) : 1ull;
      target = target < Z ? target : Z;
      __syncthreads();  // s.z, s.thr and s.total_m have been read
      bool found = select(sl, s, cluster, lo, hi, true, target, 1, fresh);
      if (!found && lo) {
        fresh = false;
        found = select(sl, s, cluster, 0, hi, true, target, 1, fresh);
      }
      // Not found: Z's rounding asks for more than there is, so everything stays.
      if (found && (!cut_k || s.thr > thr)) thr = s.thr;
    }
  }

  // 4. The race over the kept.
  const float floor_w = fminf(min_p, 1.f);
  const float* noise = a.noise + r * a.noise_ld;
  Best best{-INFINITY, 0.f, NONE};
  u64 kept = 0;
  const float floor_l = sl.logit_of(thr);
  for (int v = threadIdx.x; v < sl.nv;) {
    float sum = 0.f;
    for (int i = 0; i < 16 && v < sl.nv; ++i, v += THREADS) {
      float x[VEC];
      sl.load(v, x);
      const float most = max_of(x, VEC);
      if (most == -INFINITY || most < floor_l) continue;
      const int64_t first = sl.element(v);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (x[j] == -INFINITY || (thr && sl.key(x[j], first + j) < thr)) continue;
        const float w = sl.weight(x[j]), xt = sl.x(x[j]);
        if (w < floor_w || xt == -INFINITY) continue;
        if (thr)
          kept += sl.fixed(w);
        else
          sum += w;
        // NaN noise is never ahead.
        const float score = greedy ? 0.f : fmaxf(fmaf(lm_log2(noise[first + j]), -LN2, xt), -INFINITY);
        if (best.index == NONE || score > best.score) best = Best{score, x[j], static_cast<unsigned>(first + j)};
      }
    }
    kept += sl.fixed(sum);
  }
  kept = block_sum64(kept, s);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Best o;
    o.score = __shfl_xor_sync(FULL_MASK, best.score, d);
    o.logit = __shfl_xor_sync(FULL_MASK, best.logit, d);
    o.index = __shfl_xor_sync(FULL_MASK, best.index, d);
    better(best, o);
  }
  if (lane == 0) s.best[warp] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < WARPS; ++w) better(best, s.best[w]);
    Shared* leader = cluster.map_shared_rank(&s, 0);
    leader->ex_best[rank] = best;
    leader->ex_kept[rank] = kept;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    for (int i = 1; i < C; ++i) {
      better(best, s.ex_best[i]);
      kept += s.ex_kept[i];
    }
    // The largest logit is always kept, so an index has been found.
    a.out_tokens[r] = static_cast<int64_t>(best.index);
    a.out_logprobs[r] = greedy ? 0.f : sl.x(best.logit) - logf(static_cast<float>(kept) / sl.scale);
  }
}

// CTAs of a row's cluster.  As few as hold its slices in shared memory at two
// CTAs an SM, and more while the rows leave SMs idle.
int cluster_of(int64_t rows, int64_t bytes) {
  int c = 1;
  while (c < MAX_CLUSTER && bytes > c * SLICE_BYTES) c *= 2;
  while (c < MAX_CLUSTER && rows * c * 2 <= sms() && bytes / (2 * c) >= SLICE_LEAST) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_typed(const TokenArgs& a, cudaStream_t stream) {
  constexpr int VEC = 16 / int(sizeof(T));
  const int64_t vectors = (a.n + 2 * VEC - 2) / VEC;  // at any alignment of the row
  int c = cluster_of(a.rows, vectors * 16);
  if (a.rows * c >= (int64_t(1) << 31)) c = 1;
  const int64_t per_cta = (vectors + c - 1) / c;
  const size_t base = (sizeof(Shared) + 15) / 16 * 16;
  if (per_cta * 16 <= SLICE_MOST)
    return launch_clusters(k_sample_tokens<T, true>, a.rows * c, THREADS, c, base + size_t(per_cta) * 16, stream, a,
                           static_cast<int>(per_cta));
  return launch_clusters(k_sample_tokens<T, false>, a.rows * c, THREADS, c, base, stream, a, static_cast<int>(per_cta));
}

}  // namespace

cudaError_t launch_sample_tokens(const TokenArgs& a, cudaStream_t stream) {
  switch (a.type) {
    case PROFK_F32: return launch_typed<float>(a, stream);
    case PROFK_BF16: return launch_typed<__nv_bfloat16>(a, stream);
    default: return launch_typed<__half>(a, stream);
  }
}

}  // namespace profk
