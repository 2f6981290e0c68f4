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
// memory where it fits, and works there:
//   1. its maximum, and for top-p its mass, both relative to its own maximum;
//   2. the first keys of its slice, sorted: of the threads' maxima a value is
//      taken that at least that many of them reach, and only what lies at or
//      above it is ranked;
//   3. the CTAs exchange these (one cluster barrier), and the row's first keys
//      are known.  For top-k up to TOP, and for most rows under top-p and
//      min-p, they are all that can be kept: one warp cuts them and runs the
//      race, which reads the noise of the kept tokens only;
//   4. otherwise the cuts are found by histograms of counts and masses over
//      equal ranges of keys, repeated inside the range where the count or the
//      mass crosses its target until that holds at most LIST keys; then every
//      CTA races over its kept tokens.
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
constexpr int TOP = 128;        // keys of a slice that step 2 can sort
constexpr int TOP_P = 64;       // and those it sorts for top-p and min-p
constexpr int CANDIDATES = 1024;
constexpr int BINS = 1024;      // of one histogram pass
constexpr int PER = BINS / THREADS;
constexpr int LIST = 256;       // keys of a bin that are ranked directly
constexpr int SLICE_BYTES = 64 << 10;  // of a row in one CTA's shared memory, where the cluster is not at its largest
constexpr int SLICE_MOST = 180 << 10;  // and in any case; beyond it the passes read global memory
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

// What a CTA tells the others after step 2.
struct Part {
  float top;     // the slice's maximum (NaN if it holds one)
  float tau;     // as many of its keys as were asked for reach this value
  float mass;    // sum of exp((l - top) / T), for top-p
  int keys;      // sorted keys sent; -1: too many candidates to rank
};

struct Shared {
  // Written by other CTAs of the cluster.
  alignas(16) unsigned merged_c[BINS];
  alignas(16) u64 merged_m[BINS];
  union {
    u64 tops[MAX_CLUSTER][TOP];  // step 3
    u64 list[2][LIST];           // step 4
  };
  Part part[MAX_CLUSTER];
  Best ex_best[MAX_CLUSTER];
  u64 ex_kept[MAX_CLUSTER];
  // This CTA's own.
  union {
    struct {
      alignas(16) unsigned count[BINS];
      alignas(16) unsigned lo[BINS];  // 64-bit masses in two words
      alignas(16) unsigned hi[BINS];
    };
    alignas(16) u64 candidates[CANDIDATES + 2];
  };
  u64 sorted[LIST];
  u64 wc[WARPS], wm[WARPS], red[WARPS];
  float redf[WARPS], redt[WARPS];
  Best best[WARPS];
  unsigned slot;
  int enough;
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
    // This CTA joins its share of the bins, four a thread, and tells everybody.
    const int C = cluster.num_blocks(), share = BINS / C;
    for (int b = cluster.block_rank() * share + 4 * threadIdx.x; b < (static_cast<int>(cluster.block_rank()) + 1) * share;
         b += 4 * THREADS) {
      uint4 c = make_uint4(0, 0, 0, 0);
      u64 m[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int i = 0; i < C; ++i) {
        const Shared* o = cluster.map_shared_rank(&s, i);
        const uint4 oc = *reinterpret_cast<const uint4*>(o->count + b), ol = *reinterpret_cast<const uint4*>(o->lo + b),
                    oh = *reinterpret_cast<const uint4*>(o->hi + b);
        c.x += oc.x;
        c.y += oc.y;
        c.z += oc.z;
        c.w += oc.w;
        m[0] += (u64(oh.x) << 32) + ol.x;
        m[1] += (u64(oh.y) << 32) + ol.y;
        m[2] += (u64(oh.z) << 32) + ol.z;
        m[3] += (u64(oh.w) << 32) + ol.w;
      }
      for (int i = 0; i < C; ++i) {
        Shared* o = cluster.map_shared_rank(&s, i);
        *reinterpret_cast<uint4*>(o->merged_c + b) = c;
        *reinterpret_cast<ulonglong2*>(o->merged_m + b) = make_ulonglong2(m[0], m[1]);
        *reinterpret_cast<ulonglong2*>(o->merged_m + b + 2) = make_ulonglong2(m[2], m[3]);
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

// ceil(p Z) in integers, at least 1 and at most Z: a token is kept while the
// mass before it is below this.
__device__ __forceinline__ u64 mass_target(float p, u64 Z) {
  if (!(p > 0.f)) return 1;
  const unsigned bits = __float_as_uint(p), ex = bits >> 23;  // p < 1
  const u64 man = (bits & 0x7fffffu) | (ex ? 0x800000u : 0u);
  const int e = ex ? 150 - static_cast<int>(ex) : 149;  // p = man 2^-e, e >= 24
  const u64 hi = __umul64hi(Z, man), lo = Z * man;
  u64 q = 0;
  bool rest;
  if (e >= 128) {
    rest = (hi | lo) != 0;
  } else if (e >= 64) {
    q = hi >> (e - 64);
    rest = lo != 0 || (e > 64 && (hi << (128 - e)) != 0);
  } else {
    q = (hi << (64 - e)) | (lo >> e);
    rest = (lo << (64 - e)) != 0;
  }
  q += rest ? 1 : 0;
  return q < 1 ? 1 : q > Z ? Z : q;
}

// The want-th largest of the block's thread maxima, or less: of each warp the
// ceil(want / WARPS)-th largest, of those the least.  At least `want` threads
// reach it.  Called with the warp's own maxima; the block's value is in redt
// after a barrier.
__device__ __forceinline__ float warp_tau(float top, int want) {
  uint32_t key = choice_key(top);
  uint32_t got = 0u;
  const int lane = threadIdx.x & 31;
  for (int j = 0; j < want; j += WARPS) {
    got = __reduce_max_sync(FULL_MASK, key);
    if (lane == __ffs(__ballot_sync(FULL_MASK, key == got)) - 1) key = 0u;
  }
  return got ? key_to_float(got) : -INFINITY;
}

// Candidates larger than a key: its rank, as keys are distinct.  (An odd number
// of them is followed by a 0.)
__device__ __forceinline__ int larger_keys(const Shared& s, int keys, u64 key) {
  int above = 0;
#pragma unroll 4
  for (int j = 0; j < keys; j += 2) {
    const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s.candidates + j);
    above += (o.x > key) + (o.y > key);
  }
  return above;
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
  auto started = cluster.barrier_arrive();  // waited for before the first write to another CTA
  if (threadIdx.x == 0) s.slot = 0;
  pdl_wait();
  pdl_trigger();
  const float temperature = a.temperature ? a.temperature[r] : a.all_temperature;
  const int32_t k = a.top_k ? a.top_k[r] : a.all_top_k;
  const float p = a.top_p ? a.top_p[r] : a.all_top_p;
  const float min_p = a.min_p ? a.min_p[r] : a.all_min_p;
  const bool greedy = temperature == 0.f;
  const bool by_k = !greedy && k > 0 && k < a.n, by_p = !greedy && p < 1.f;
  // Keys that step 2 sorts (0: it would not help).
  const int want = greedy ? 1 : by_k ? (k <= TOP ? k : 0) : by_p || min_p > 0.f ? TOP_P : 0;
  // Keys for which a value is looked for that as many reach.
  const int reach = want ? want : by_k && k <= THREADS ? k : 0;
  S sl;
  sl.row = static_cast<const T*>(a.logits) + r * a.ld;
  sl.mask = a.mask ? a.mask + r * a.mask_ld : nullptr;
  sl.store = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  sl.n = a.n;
  sl.phase = static_cast<int>(reinterpret_cast<uintptr_t>(sl.row) % 16 / sizeof(T));
  const int64_t all = (a.n + sl.phase + VEC - 1) / VEC;
  sl.v0 = static_cast<int64_t>(rank) * per_cta;
  sl.nv = static_cast<int>(all <= sl.v0 ? 0 : all - sl.v0 < per_cta ? all - sl.v0 : per_cta);
  // An infinite T: the smallest number, so that -inf stays -inf.
  sl.inv = fmaxf(1.f / temperature, __int_as_float(1));
  sl.inv2 = sl.inv * LOG2E;
  sl.index_bits = 32 - __clz(static_cast<int>(a.n - 1));
  const int e = min(62 - sl.index_bits, 44);
  sl.scale = __int_as_float((127 + e) << 23);

  // 1. The slice, and its largest logit (NaN if there is one).
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
  float widest = top;
#pragma unroll
  for (int d = 16; d; d >>= 1) widest = max_nan(widest, __shfl_xor_sync(FULL_MASK, widest, d));
  if (lane == 0) s.redf[warp] = widest;
  if (reach) {
    if (RESIDENT && sl.nv < THREADS) {
      // Fewer vectors than threads: the threads' maxima of single elements instead.
      __syncthreads();
      const T* flat = reinterpret_cast<const T*>(sl.store);
      top = -INFINITY;
      for (int i = threadIdx.x; i < sl.nv * VEC; i += THREADS) top = fmaxf(top, lm_float(flat[i]));
    }
    const float least = warp_tau(top, reach);
    if (lane == 0) s.redt[warp] = least;
  }
  __syncthreads();
  widest = s.redf[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) widest = max_nan(widest, s.redf[w]);
  float tau = -INFINITY;
  if (reach) {
    tau = s.redt[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) tau = fminf(tau, s.redt[w]);
  }
  sl.m = widest;

  // 2. The slice's mass, and its first keys.
  float mass = 0.f;
  const bool need_mass = by_p && !by_k;
  int keys = 0;
  if (want || need_mass) {
    for (int turn = 0;; ++turn) {
      for (int v = threadIdx.x; v < sl.nv; v += THREADS) {
        float x[VEC];
        sl.load(v, x);
        const float most = max_of(x, VEC);
        if (want && most >= tau && most > -INFINITY) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (x[j] >= tau && x[j] > -INFINITY) {
              const unsigned at = atomicAdd(&s.slot, 1u);
              if (at < CANDIDATES) s.candidates[at] = sl.key(x[j], sl.element(v) + j);
            }
        }
        if (need_mass && turn == 0) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[j] = sl.weight(x[j]);
#pragma unroll
          for (int d = VEC / 2; d; d >>= 1)
#pragma unroll
            for (int j = 0; j < d; ++j) x[j] += x[j + d];
          mass += x[0];
        }
      }
      __syncthreads();  // the candidates are complete; redf has been read
      keys = static_cast<int>(s.slot);
      if (keys <= CANDIDATES || turn == 2) break;
      // Too many (neighbours are alike, so that some warps' maxima are low):
      // again from the want-th largest of those that were stored.
      for (int i = threadIdx.x; i < CANDIDATES; i += THREADS)
        if (larger_keys(s, CANDIDATES, s.candidates[i]) == want - 1) s.thr = s.candidates[i];
      __syncthreads();
      tau = sl.logit_of(s.thr);
      if (threadIdx.x == 0) s.slot = 0;
      __syncthreads();
    }
    mass = warp_sum(mass);
    if (lane == 0) s.redf[warp] = mass;
  }
  cluster.barrier_wait(std::move(started));
  if (keys > CANDIDATES) {  // copies of one value
    keys = -1;
  } else if (want) {
    // The first `want` go to every CTA that looks at them.
    const int readers = by_k || greedy ? 1 : C;
    if (threadIdx.x == 0) s.candidates[keys] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < keys; i += THREADS) {
      const u64 mine = s.candidates[i];
      const int above = larger_keys(s, keys, mine);
      if (above < want)
        for (int c = 0; c < readers; ++c) cluster.map_shared_rank(&s, c)->tops[rank][above] = mine;
    }
    keys = keys < want ? keys : want;
  }
  __syncthreads();
  if (threadIdx.x < C) {
    mass = 0.f;
    if (need_mass)
      for (int w = 0; w < WARPS; ++w) mass += s.redf[w];
    cluster.map_shared_rank(&s, threadIdx.x)->part[rank] = Part{widest, tau, mass, keys};
  }
  cluster.sync();

  // 3. The row's maximum, mass and first keys.
  top = s.part[0].top;
  tau = s.part[0].tau;
  int found = 0;  // keys of all CTAs, or -1
  for (int i = 0; i < C; ++i) {
    top = max_nan(top, s.part[i].top);
    tau = fmaxf(tau, s.part[i].tau);
    found = found < 0 || s.part[i].keys < 0 ? -1 : found + s.part[i].keys;
  }
  const bool bad = isnan(top) || !(temperature >= 0.f) || isnan(p) || isnan(min_p);
  if (bad || top == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      a.out_tokens[r] = -1;
      a.out_logprobs[r] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
    }
    return;
  }
  sl.m = top;
  u64 Z = 0;
  if (need_mass)
    for (int i = 0; i < C; ++i) Z += sl.fixed(s.part[i].mass * sl.weight(s.part[i].top));
  const float floor_w = fminf(min_p, 1.f);
  const float* noise = a.noise + r * a.noise_ld;
  if (want && found >= 0) {
    const bool decide = !by_k && !greedy;  // whether these keys are enough is not known beforehand
    if (rank != 0 && !decide) return;
    // Merge: a key's place is the number of larger ones in each of the sorted lists.
    const int got = found < want ? found : want;
    for (int i = threadIdx.x; i < C * want; i += THREADS) {
      const int c = i / want, j = i - c * want;
      if (j >= s.part[c].keys) continue;
      const u64 mine = s.tops[c][j];
      int place = j;
      for (int o = 0; o < C && place < want; ++o) {
        if (o == c) continue;
        int lo = 0, hi = s.part[o].keys;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (s.tops[o][mid] > mine)
            lo = mid + 1;
          else
            hi = mid;
        }
        place += lo;
      }
      if (place < want) s.sorted[place] = mine;
    }
    __syncthreads();
    if (warp == 0) {
      constexpr int EACH = TOP / 32;
      float l[EACH], w[EACH];
      u64 part[EACH], sum = 0;
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int at = lane * EACH + j;
        l[j] = at < got ? sl.logit_of(s.sorted[at]) : -INFINITY;
        w[j] = at < got ? sl.weight(l[j]) : 0.f;
        part[j] = sl.fixed(w[j]);
        sum += part[j];
      }
      u64 before = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(FULL_MASK, before, d);
        if (lane >= d) before += o;
      }
      const u64 total = __shfl_sync(FULL_MASK, before, 31);
      before -= sum;
      if (by_k) Z = total;
      const u64 target = by_p ? mass_target(p, Z) : ~u64(0);
      // Enough: the list holds everything, or reaches the mass, or falls below min-p.
      const float last = got ? sl.weight(sl.logit_of(s.sorted[got - 1])) : 0.f;
      const bool enough = !decide || found < want || (by_p && total >= target) || last < floor_w;
      if (lane == 0) s.enough = enough;
      if (enough && rank == 0) {
        u64 kept = 0;
        Best best{-INFINITY, 0.f, NONE};
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const int at = lane * EACH + j;
          if (at < got && (before < target || at == 0) && w[j] >= floor_w && sl.x(l[j]) > -INFINITY) {
            const unsigned i =
                static_cast<unsigned>(((u64(1) << sl.index_bits) - 1) - (s.sorted[at] & ((u64(1) << sl.index_bits) - 1)));
            const float score = greedy ? 0.f : fmaxf(fmaf(lm_log2(noise[i]), -LN2, sl.x(l[j])), -INFINITY);
            kept += part[j];
            better(best, Best{score, l[j], i});
          }
          before += part[j];
        }
        kept = warp_sum64(kept);
#pragma unroll
        for (int d = 16; d; d >>= 1) {
          Best o;
          o.score = __shfl_xor_sync(FULL_MASK, best.score, d);
          o.logit = __shfl_xor_sync(FULL_MASK, best.logit, d);
          o.index = __shfl_xor_sync(FULL_MASK, best.index, d);
          better(best, o);
        }
        if (lane == 0) {  // the largest logit is always kept, so there is one
          a.out_tokens[r] = static_cast<int64_t>(best.index);
          a.out_logprobs[r] = greedy ? 0.f : sl.x(best.logit) - logf(static_cast<float>(kept) / sl.scale);
        }
      }
    }
    __syncthreads();
    if (s.enough) return;
  }

  // 4. The cuts, over everything above a value that surely is not kept: for
  // top-k a value that k keys of one slice reach; for top-p the value at which
  // n tokens together weigh less than what may be left out.
  u64 thr = greedy ? sl.value_key(top) : 0;  // copies of the maximum; the lowest index wins the race
  if (by_k || by_p) {
    float at = -INFINITY;
    if (by_k)
      at = tau;
    else
      at = top - temperature * __logf(static_cast<float>(a.n) / (0.99f * (1.f - fmaxf(p, 0.f)) * (static_cast<float>(Z) / sl.scale)));
    const u64 hi = sl.value_key(top) | ((u64(1) << sl.index_bits) - 1);
    const u64 lo = at <= top && at > -INFINITY ? sl.value_key(at) : 0;
    bool fresh = false, cut_k = false;
    cluster.sync();  // the keys of step 3 have been read: list takes their place
    if (by_k) {
      cut_k = select(sl, s, cluster, lo, hi, false, static_cast<u64>(k), 0, fresh);
      Z = cut_k ? s.z : s.total_m;  // not found: there are no more than k
      if (cut_k) thr = s.thr;
    }
    if (by_p) {
      __syncthreads();  // s.z, s.thr and s.total_m have been read
      const u64 target = mass_target(p, Z);
      bool cut_p = select(sl, s, cluster, lo, hi, true, target, 1, fresh);
      if (!cut_p && lo) {  // the masses' roundings used up what `lo` leaves out
        fresh = false;
        cut_p = select(sl, s, cluster, 0, hi, true, target, 1, fresh);
      }
      // Still not: Z's rounding asks for more than there is, so everything stays.
      if (cut_p && s.thr > thr) thr = s.thr;
    }
  }

  // The race over the kept.
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
