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
//      equal ranges of x, then of keys, repeated inside the range where the
//      count or the mass crosses its target until that holds at most LIST
//      keys; then every CTA races over its kept tokens.  For top-p a sample of
//      the row tells above which value the crossing should lie, so that the
//      histogram touches little else; where it does not, it is made again from
//      a value that surely is below.
//
// Masses are summed as 64-bit integers (w scaled by a power of two up to
// 2^44, the largest that n of them cannot overflow), so that every sum is
// the same whatever order the atomics take.
#include <cfloat>

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
constexpr int TOP = 128;        // keys of a slice that step 2 can sort (the merge searches lists of up to 2^8 - 1)
constexpr int TOP_P = 128;      // and those it sorts for top-p and min-p
constexpr int CANDIDATES = 1024;
constexpr int BINS = 256;       // of one histogram pass (the joining of 1024 took 6 us in a cluster of 8)
constexpr int SAMPLE_BINS = 128;       // of the sample of a slice,
constexpr float SAMPLE_SCALE = 8.f;    // so many a unit of x
constexpr int SAMPLE_EVERY = 16;
constexpr int LIST = 256;       // keys of a bin that are ranked directly
constexpr int SLICE_BYTES = 66 << 10;  // of a row in one CTA's shared memory, where the cluster is not at its largest
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

// What late_row gets.
struct Late {
  const float* noise;
  int64_t* token;
  float* logprob;
  u64 Z;
  int32_t k;
  float p, temperature, floor_w, tau;
  bool by_k, by_p;
};

struct Shared {
  // Written by other CTAs of the cluster.
  alignas(16) unsigned merged_c[BINS];
  alignas(16) u64 merged_m[BINS];
  u64 tops[MAX_CLUSTER][TOP];     // step 3: first keys, and their noise
  float tops_q[MAX_CLUSTER][TOP];
  u64 list[2][LIST];              // step 4
  unsigned sample[MAX_CLUSTER][SAMPLE_BINS];
  Part part[MAX_CLUSTER];
  int enough;
  Best ex_best[MAX_CLUSTER];
  u64 ex_kept[MAX_CLUSTER];
  u64 beyond[MAX_CLUSTER];
  // This CTA's own.
  union {
    struct {
      alignas(16) unsigned count[BINS];
      alignas(16) unsigned lo[BINS];  // 64-bit masses in two words
      alignas(16) unsigned hi[BINS];
    };
    struct {
      alignas(16) u64 candidates[CANDIDATES + 2];
      float candidates_q[CANDIDATES];
    };
  };
  unsigned own_sample[SAMPLE_BINS];
  u64 sorted[LIST];
  float sorted_q[TOP];
  u64 wc[WARPS], wm[WARPS], red[WARPS];
  float redf[WARPS], mass[WARPS];
  uint32_t redk[WARPS];
  Best best[WARPS];
  unsigned slot, merged;
  unsigned bin;  // the crossing found by a pass: BINS if there is none
  u64 above_c, above_m, in_c, total_m;
  u64 thr, z;
  float likely[2];
  Late late;
  alignas(8) unsigned char slice[96];  // the row's Slice
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

// log2 of a positive number by the hardware's approximation; zero gives -inf.
__device__ __forceinline__ float lm_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max_of(const float* x, int n) {
  float top = x[0];
#pragma unroll
  for (int j = 1; j < n; ++j) top = fmaxf(top, x[j]);
  return top;
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

  // Element j of a vector (inside the row, allowed).
  __device__ __forceinline__ float one(int v, int j) const {
    if constexpr (RESIDENT)
      return lm_float(reinterpret_cast<const T*>(store + v)[j]);
    else
      return lm_float(row[element(v) + j]);
  }

  // body(l, i, given(i)) for every element of the slice in [floor, ceil] (floor
  // finite or +inf).  A thread first marks those of several vectors and then
  // takes them four by four, so that the lanes' hits meet in the same turns and
  // what `given` reads for them is under way together.  each(x) sees every
  // vector that is looked at.
  template <typename E, typename G, typename F>
  __device__ __forceinline__ void among(float floor, float ceil, E&& each, G&& given, F&& body) const {
    constexpr int GROUP = 32 / VEC, BATCH = 4;
    for (int v = threadIdx.x; v < nv; v += GROUP * THREADS) {
      unsigned hits = 0;
#pragma unroll
      for (int g = 0; g < GROUP; ++g) {
        const int u = v + g * THREADS;
        if (u >= nv) break;
        float x[VEC];
        load(u, x);
        each(x);
        if (max_of(x, VEC) < floor) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) hits |= x[j] >= floor && x[j] <= ceil ? 1u << (g * VEC + j) : 0u;
      }
      while (hits) {
        float l[BATCH];
        int64_t at[BATCH];
        decltype(given(int64_t(0))) what[BATCH];
        int some = 0;
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (hits) {
            const int b = __ffs(hits) - 1, u = v + b / VEC * THREADS;
            hits &= hits - 1;
            at[i] = element(u) + b % VEC;
            l[i] = one(u, b % VEC);
            what[i] = given(at[i]);
            some = i + 1;
          }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (i < some) body(l[i], at[i], what[i]);
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void among(float floor, float ceil, F&& body) const {
    among(floor, ceil, [](const float (&)[VEC]) {}, [](int64_t) { return 0; },
          [&](float l, int64_t i, int) { body(l, i); });
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
  __device__ __forceinline__ int64_t index_of(u64 key) const {
    const u64 ones = (u64(1) << index_bits) - 1;
    return static_cast<int64_t>(ones - (key & ones));
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

// What a histogram is made of: first, the elements with logits in [floor,
// ceil], in equal ranges of x from ceil down (the last takes what is beyond);
// then those of the first one's bin `bin0` with keys in [lo, hi], in equal
// ranges of keys from hi down.
struct Level {
  float floor, ceil;
  float x0, per_x;  // -x of ceil; bins per unit of x of the first
  int bin0;         // -1: the first
  u64 lo, hi;
  int shift;

  template <typename S>
  __device__ __forceinline__ int bin_of(const S& sl, float l, int64_t i) const {
    const int b = static_cast<int>(fmaxf(fminf((-sl.x(l) - x0) * per_x, BINS - 1.f), 0.f));
    if (bin0 < 0) return b;
    const u64 key = sl.key(l, i);
    return b != bin0 || key < lo || key > hi ? -1 : static_cast<int>((hi - key) >> shift);
  }
  // A value at or above all of a bin of the first, and one at or below (x's
  // roundings blur its edges by far less than half a bin).
  template <typename S>
  __device__ __forceinline__ float high(const S& sl, int bin) const {
    const float v = sl.m - (x0 + (bin - 0.5f) / per_x) / sl.inv;
    return bin > 0 && v <= ceil ? v : ceil;
  }
  template <typename S>
  __device__ __forceinline__ float low(const S& sl, int bin) const {
    const float v = sl.m - (x0 + (bin + 1.5f) / per_x) / sl.inv;
    return bin + 1 < BINS && v >= floor ? v : floor;
  }
  __device__ __forceinline__ void fit() {
    shift = 0;
    while (((hi - lo) >> shift) >= BINS) ++shift;
  }
};

// The histogram, joined over the cluster, and the bin where the running count
// (or mass) from the top first reaches `target`: s.bin, s.above_*, s.in_c;
// s.bin = BINS where it does not.  What lies above the first level's ceil
// counts as above (its mass only).  fresh: the joined histogram is in place.
template <typename S>
__device__ __forceinline__ void cross(const S& sl, Shared& s, cg::cluster_group& cluster, const Level& lv, bool by_mass,
                                      u64 target, bool fresh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool over = lv.bin0 < 0 && lv.ceil < sl.m;
  if (!fresh) {
    for (int b = threadIdx.x; b < BINS; b += THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0u;
    __syncthreads();
    u64 beyond = 0;
    float partial = 0.f;
    int vectors = 0;
    sl.among(
        lv.floor, lv.ceil,
        [&](const float (&x)[S::VEC]) {
          if (!over) return;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < S::VEC; ++j) sum += x[j] > lv.ceil ? sl.weight(x[j]) : 0.f;
          partial += sum;
          if (++vectors % 16 == 0) {
            beyond += sl.fixed(partial);
            partial = 0.f;
          }
        },
        [](int64_t) { return 0; },
        [&](float l, int64_t i, int) {
          const int b = lv.bin_of(sl, l, i);
          if (b < 0) return;
          const u64 mass = sl.fixed(sl.weight(l));
          atomicAdd(&s.count[b], 1u);
          const unsigned ml = static_cast<unsigned>(mass), old = atomicAdd(&s.lo[b], ml);
          const unsigned mh = static_cast<unsigned>(mass >> 32) + (old + ml < old ? 1u : 0u);
          if (mh) atomicAdd(&s.hi[b], mh);
        });
    if (over) {
      beyond = block_sum64(beyond + sl.fixed(partial), s);
      if (threadIdx.x < cluster.num_blocks()) cluster.map_shared_rank(&s, threadIdx.x)->beyond[cluster.block_rank()] = beyond;
    }
    cluster.sync();
    // This CTA joins its share of the bins: of C neighbouring threads each reads
    // four bins of one CTA, and, when they have added them up, tells one.
    const int C = cluster.num_blocks(), share = BINS / C, with = threadIdx.x % C;
    const Shared* from = cluster.map_shared_rank(&s, with);
    Shared* to = cluster.map_shared_rank(&s, with);
    for (int base = 0; base < share * C / 4; base += THREADS) {
      const int b = cluster.block_rank() * share + (base + static_cast<int>(threadIdx.x)) / C * 4;
      const bool some = base + static_cast<int>(threadIdx.x) < share * C / 4;
      uint4 c = make_uint4(0, 0, 0, 0), ml = c, mh = c;
      if (some) {
        c = *reinterpret_cast<const uint4*>(from->count + b);
        ml = *reinterpret_cast<const uint4*>(from->lo + b);
        mh = *reinterpret_cast<const uint4*>(from->hi + b);
      }
      u64 m[4] = {(u64(mh.x) << 32) + ml.x, (u64(mh.y) << 32) + ml.y, (u64(mh.z) << 32) + ml.z, (u64(mh.w) << 32) + ml.w};
      for (int d = C >> 1; d; d >>= 1) {
        c.x += __shfl_xor_sync(FULL_MASK, c.x, d);
        c.y += __shfl_xor_sync(FULL_MASK, c.y, d);
        c.z += __shfl_xor_sync(FULL_MASK, c.z, d);
        c.w += __shfl_xor_sync(FULL_MASK, c.w, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] += __shfl_xor_sync(FULL_MASK, m[j], d);
      }
      if (some) {
        *reinterpret_cast<uint4*>(to->merged_c + b) = c;
        *reinterpret_cast<ulonglong2*>(to->merged_m + b) = make_ulonglong2(m[0], m[1]);
        *reinterpret_cast<ulonglong2*>(to->merged_m + b + 2) = make_ulonglong2(m[2], m[3]);
      }
    }
    cluster.sync();
  }
  u64 base = 0;
  if (over)
    for (int i = 0; i < static_cast<int>(cluster.num_blocks()); ++i) base += s.beyond[i];
  // Thread t takes bin t.
  const bool mine = threadIdx.x < BINS;
  const u64 nc = mine ? s.merged_c[threadIdx.x] : 0, nm = mine ? s.merged_m[threadIdx.x] : 0;
  u64 ic = nc, im = nm;
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
  u64 bc = ic - nc, bm = base + im - nm;
  for (int w = 0; w < warp; ++w) {
    bc += s.wc[w];
    bm += s.wm[w];
  }
  if (threadIdx.x == BINS - 1) s.total_m = bm + nm;
  const u64 before = by_mass ? bm : bc, with = before + (by_mass ? nm : nc);
  if (before < target && target <= with) {
    s.bin = threadIdx.x;
    s.above_c = bc;
    s.above_m = bm;
    s.in_c = nc;
  }
  __syncthreads();
}

// The key down to which tokens are kept, s.thr (every kept key >= it), and the
// mass of those, s.z: the first `target` keys from the top, or as many as it
// takes for their mass to reach it.  False: all that `lv` counts does not reach
// it (then s.total_m is its mass).
template <typename S>
__device__ bool select(const S& sl, Shared& s, cg::cluster_group& cluster, Level lv, bool by_mass, u64 target, int which,
                       bool& fresh) {
  const int lane = threadIdx.x & 31;
  u64 above_c = 0, above_m = 0;
  for (int level = 0;; ++level) {
    cross(sl, s, cluster, lv, by_mass, target - (by_mass ? above_m : above_c), fresh && level == 0);
    fresh = level == 0;
    if (s.bin == BINS) return false;
    above_c += s.above_c;
    above_m += s.above_m;
    const u64 in_c = s.in_c;
    const int bin = static_cast<int>(s.bin);
    if (in_c > LIST) {
      if (lv.bin0 < 0) {
        const float high = lv.high(sl, bin), low = lv.low(sl, bin);
        lv.bin0 = bin;
        lv.hi = sl.value_key(high) | ((u64(1) << sl.index_bits) - 1);
        lv.lo = sl.value_key(low);
        lv.floor = low;
        lv.ceil = high;
      } else {
        lv.hi -= u64(bin) << lv.shift;
        const u64 width = (u64(1) << lv.shift) - 1;
        if (lv.hi - lv.lo > width) lv.lo = lv.hi - width;
      }
      lv.fit();
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
    const float floor = lv.bin0 < 0 ? lv.low(sl, bin) : lv.floor, ceil = lv.bin0 < 0 ? lv.high(sl, bin) : lv.ceil;
    if (s.count[bin] != 0u)
      sl.among(floor, ceil, [&](float l, int64_t i) {
        if (lv.bin_of(sl, l, i) != bin) return;
        const unsigned at = atomicAdd(&s.slot, 1u);
        if (at < LIST)
          for (int c = 0; c < C; ++c) cluster.map_shared_rank(&s, c)->list[which][at] = sl.key(l, i);
      });
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

// A value that at least `want` of the block's thread maxima reach, and not many
// more: bisection over the keys between the least maximum and the largest
// (each under a count over the block).  -inf if there are no more than `want`.
__device__ __forceinline__ float block_tau(float top, float widest, int want, Shared& s) {
  const uint32_t key = choice_key(top);
  const uint32_t least = __reduce_min_sync(FULL_MASK, key ? key : ~0u);
  if ((threadIdx.x & 31) == 0) s.redk[threadIdx.x >> 5] = least;
  int count = __syncthreads_count(key != 0u);
  if (count <= want) return -INFINITY;
  uint32_t lo = s.redk[0], hi = choice_key(widest) + 1u;
#pragma unroll
  for (int w = 1; w < WARPS; ++w) lo = min(lo, s.redk[w]);
  while (hi - lo > 1u && count > want + want / 8 + 4) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int c = __syncthreads_count(key >= mid);
    if (c >= want) {
      lo = mid;
      count = c;
    } else {
      hi = mid;
    }
  }
  return key_to_float(lo);
}

// body(i, rank) for every candidate, rank being the number of larger ones (they
// are distinct); each is ranked by as many neighbouring threads as there are
// to spare, up to 8, and the first of them calls body.  begin(i) runs before
// the ranking (with whether there is an i) and returns what body gets as well.  Called by the whole block;
// an odd number of candidates is followed by a 0.
template <typename B, typename F>
__device__ __forceinline__ void rank_candidates(const Shared& s, int keys, B&& begin, F&& body) {
  int split = 1;
  while (split < 8 && keys * split * 2 <= THREADS) split *= 2;
  const int sub = threadIdx.x & (split - 1);
  for (int base = 0; base < keys; base += THREADS / split) {
    const int i = base + threadIdx.x / split;
    const u64 mine = i < keys ? s.candidates[i] : ~u64(0);
    const auto what = begin(i < keys && sub == 0, i, mine);
    int above = 0;
#pragma unroll 4
    for (int j = 2 * sub; j < keys; j += 2 * split) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s.candidates + j);
      above += (o.x > mine) + (o.y > mine);
    }
    for (int d = split >> 1; d; d >>= 1) above += __shfl_xor_sync(FULL_MASK, above, d);
    if (i < keys && sub == 0) body(mine, above, what);
  }
}

// x - log q; NaN noise is never ahead.
__device__ __forceinline__ float race(float x, float q) { return fmaxf(fmaf(lm_log2(q), -LN2, x), -INFINITY); }

// The best of the lanes' bests, in every lane.
__device__ __forceinline__ void warp_best(Best& best) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    Best o;
    o.score = __shfl_xor_sync(FULL_MASK, best.score, d);
    o.logit = __shfl_xor_sync(FULL_MASK, best.logit, d);
    o.index = __shfl_xor_sync(FULL_MASK, best.index, d);
    better(best, o);
  }
}

template <typename S>
__device__ __forceinline__ void write_row(const S& sl, const Best& best, u64 kept, bool greedy, int64_t* token,
                                          float* logprob) {
  // The largest logit is always kept, so an index has been found.
  *token = static_cast<int64_t>(best.index);
  *logprob = greedy ? 0.f : sl.x(best.logit) - logf(static_cast<float>(kept) / sl.scale);
}

// Joins the race over the threads and CTAs and writes the row's answer.
template <typename S>
__device__ __forceinline__ void finish(const S& sl, Shared& s, cg::cluster_group& cluster, Best best, u64 kept, bool greedy,
                                       int64_t* token, float* logprob) {
  const int rank = cluster.block_rank();
  kept = block_sum64(kept, s);
  warp_best(best);
  if ((threadIdx.x & 31) == 0) s.best[threadIdx.x >> 5] = best;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < WARPS; ++w) better(best, s.best[w]);
    Shared* leader = cluster.map_shared_rank(&s, 0);
    leader->ex_best[rank] = best;
    leader->ex_kept[rank] = kept;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    for (int i = 1; i < static_cast<int>(cluster.num_blocks()); ++i) {
      better(best, s.ex_best[i]);
      kept += s.ex_kept[i];
    }
    write_row(sl, best, kept, greedy, token, logprob);
  }
}

// The first level of a selection among the logits in [floor, ceil] (a floor
// that is no number of the row's: from the bottom).
template <typename S>
__device__ __forceinline__ Level level_between(const S& sl, float floor, float ceil) {
  const bool bounded = floor <= ceil && floor > -INFINITY;
  Level lv{};
  lv.bin0 = -1;
  lv.floor = bounded ? floor : -FLT_MAX;
  lv.ceil = ceil;
  lv.x0 = -sl.x(ceil);
  // The bins end at the floor, and where weights are nothing beside the maximum's.
  const float reach = bounded ? fminf(-sl.x(floor), 64.f) : 64.f;
  lv.per_x = BINS / fmaxf(reach - lv.x0, 1e-4f);
  return lv;
}

// Where (in x below the maximum) the slices' samples put the point under which
// `left` of mass lies: s.likely[0] surely further than that, and, where the
// tokens above are many, s.likely[1] surely nearer (else 0).  Surely: by four
// standard deviations of the sample's sum below the point.
template <typename S>
__device__ __forceinline__ void sample_point(const S& sl, Shared& s, float left) {
  constexpr int EACH = SAMPLE_BINS / 32;
  const int C = cg::this_cluster().num_blocks();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    float count[EACH] = {};
    for (int c = 0; c < C; ++c) {
      // Bins of a slice count from its own maximum.
      const int away = static_cast<int>(fminf(-SAMPLE_SCALE * sl.x(s.part[c].top), SAMPLE_BINS) + 0.5f);
#pragma unroll
      for (int j = 0; j < EACH; ++j) {
        const int b = EACH * lane + j - away;
        if (b >= 0) count[j] += static_cast<float>(s.sample[c][b]);
      }
    }
    // Mass and its variance, of a lane's bins and all below; tokens, of those above.
    float weight[EACH], mass[EACH], tail = 0.f, var = 0.f, tokens = 0.f;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      weight[j] = SAMPLE_EVERY * __expf(-(EACH * lane + j + 0.5f) / SAMPLE_SCALE);
      mass[j] = count[j] * weight[j];
      tail += mass[j];
      var += mass[j] * weight[j];
      tokens += count[j];
    }
    const float own_tail = tail, own_var = var, own_tokens = tokens;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const float ot = __shfl_down_sync(FULL_MASK, tail, d), ov = __shfl_down_sync(FULL_MASK, var, d),
                  on = __shfl_up_sync(FULL_MASK, tokens, d);
      if (lane + d < 32) {
        tail += ot;
        var += ov;
      }
      if (lane >= d) tokens += on;
    }
    tail -= own_tail;  // below the lane's bins
    var -= own_var;
    tokens -= own_tokens;
    // The bin inside which the tail reaches `left`: the lane's last first.
    float far = -1.f, near = 0.f;
#pragma unroll
    for (int j = EACH - 1; j >= 0; --j) {
      if (tail <= left && left < tail + mass[j]) {
        const float point = (EACH * lane + j + 1 - (left - tail) / mass[j]) / SAMPLE_SCALE;
        const float blur = 0.02f + 4.f * sqrtf(var + weight[j] * mass[j]) / (mass[j] * SAMPLE_SCALE);
        far = point + blur;
        float above = tokens;
#pragma unroll
        for (int i = 0; i < j; ++i) above += count[i];
        near = above * SAMPLE_EVERY > 4096.f ? fmaxf(point - blur, 0.f) : 0.f;
      }
      tail += mass[j];
      var += mass[j] * weight[j];
    }
    const unsigned which = __ballot_sync(FULL_MASK, far >= 0.f);
    if (which == 0u) far = INFINITY;  // the sample has no answer
    if (which == 0u ? lane == 0 : lane == __ffs(which) - 1) {
      s.likely[0] = far;
      s.likely[1] = near;
    }
  }
  __syncthreads();
}

// 4. The cuts, over everything above a value that is not kept: for top-k one
// that k keys of one slice reach; for top-p the sample's, or the one at which n
// tokens together weigh less than what may be left out.  Then the race.  (A
// function of its own: the registers that it needs would be spilled by rows
// that never come here, at a microsecond a row.)
template <typename S>
__device__ __noinline__ void late_row(Shared& s) {
  static_assert(sizeof(S) <= sizeof(s.slice), "room for the slice");
  const S sl = *reinterpret_cast<const S*>(s.slice);
  const Late& late = s.late;
  cg::cluster_group cluster = cg::this_cluster();
  const float temperature = late.temperature, top = sl.m;
  const bool greedy = temperature == 0.f;
  u64 Z = late.Z;
  u64 thr = greedy ? sl.value_key(top) : 0;  // copies of the maximum; the lowest index wins the race
  if (late.by_k || late.by_p) {
    const float left = (1.f - fmaxf(late.p, 0.f)) * (static_cast<float>(Z) / sl.scale);
    const float sure = late.by_k ? late.tau : top - temperature * __logf(static_cast<float>(sl.n) / (0.99f * left));
    if (!late.by_k) sample_point(sl, s, left);
    const float far = late.by_k ? sure : top - temperature * s.likely[0];
    const float ceil = late.by_k || s.likely[1] <= 0.f ? top : top - temperature * s.likely[1];
    // From the narrowest range to the widest, tried one after another.
    Level lv = far <= top && far > sure ? level_between(sl, far, ceil) : level_between(sl, sure, top);
    bool fresh = false;
    for (int turn = late.by_k ? 0 : 1; turn < (late.by_p ? 2 : 1); ++turn) {  // the first k, then their share p
      const u64 target = turn ? mass_target(late.p, Z) : static_cast<u64>(late.k);
      bool cut;
      for (;;) {
        __syncthreads();  // what the turn before left in s has been read
        cut = select(sl, s, cluster, lv, turn == 1, target, turn, fresh);
        if (cut || turn == 0 || lv.floor == -FLT_MAX) break;
        // The sample's answer was wrong, or roundings used up what the sure floor
        // leaves out.
        lv = level_between(sl, lv.floor > sure ? sure : -INFINITY, top);
        fresh = false;
      }
      // Without a cut: there are no more than k, or Z's rounding asks for more
      // mass than there is, so that everything stays.
      if (turn == 0) Z = cut ? s.z : s.total_m;
      if (cut && s.thr > thr) thr = s.thr;
    }
  }
  // (ln min_p: with room for its and the weights' roundings.)
  const float floor_w = late.floor_w;
  float floor = thr ? sl.logit_of(thr) : -FLT_MAX;
  if (floor_w > 0.f) floor = fmaxf(floor, fminf(top, top + temperature * (1.001f * __logf(floor_w) - 1e-3f)));
  Best best{-INFINITY, 0.f, NONE};
  u64 kept = 0;
  const float* noise = late.noise;
  sl.among(
      floor, INFINITY, [](const float (&)[S::VEC]) {}, [&](int64_t i) { return greedy ? 1.f : noise[i]; },
      [&](float l, int64_t i, float q) {
        const float w = sl.weight(l), x = sl.x(l);
        if (sl.key(l, i) < thr || w < floor_w || x == -INFINITY) return;
        kept += sl.fixed(w);
        better(best, Best{greedy ? 0.f : race(x, q), l, static_cast<unsigned>(i)});
      });
  finish(sl, s, cluster, best, kept, greedy, late.token, late.logprob);
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
  if (threadIdx.x == 0) s.slot = s.merged = 0;
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

  if (!want && !by_k && !by_p) {
    // Every token's noise will be read: L2 fetches it meanwhile.
    const int64_t first = max(sl.element(0), int64_t(0)), last = min(sl.element(sl.nv), a.n);
    const uintptr_t from = (reinterpret_cast<uintptr_t>(a.noise + r * a.noise_ld + first) + 15) & ~uintptr_t(15),
                    to = reinterpret_cast<uintptr_t>(a.noise + r * a.noise_ld + last) & ~uintptr_t(15);
    constexpr unsigned PIECE = 4096;
    for (uintptr_t at = from + threadIdx.x * PIECE; at < to; at += THREADS * PIECE)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at),
                   "r"(static_cast<unsigned>(to - at < PIECE ? to - at : PIECE)) : "memory");
  }

  // 1. The slice, its largest logit (NaN if there is one) and, for top-p, its
  // mass: a thread's sum of exp((l - ref) / T), ref being the largest of its
  // logits so far.
  const bool need_mass = by_p && !by_k;
  if (threadIdx.x < SAMPLE_BINS) s.own_sample[threadIdx.x] = 0u;
  float top = -INFINITY, mass = 0.f;
  auto take = [&](float (&x)[VEC]) {
    const float before = top;
#pragma unroll
    for (int j = 0; j < VEC; ++j) top = max_nan(top, x[j]);
    if (need_mass && top > -INFINITY) {
      sl.m = top;
      mass *= sl.weight(before);
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = sl.weight(x[j]);
#pragma unroll
      for (int d = VEC / 2; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < d; ++j) x[j] += x[j + d];
      mass += x[0];
    }
  };
  if constexpr (RESIDENT) {
    // The whole slice is on its way at once, in four groups of copies; a thread
    // reads what it copied itself.
    const int group = ((sl.nv + THREADS - 1) / THREADS + 3) / 4 * THREADS;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      for (int v = g * group + threadIdx.x; v < min((g + 1) * group, sl.nv); v += THREADS) {
        if (sl.inside(v)) {
          const unsigned to = static_cast<unsigned>(__cvta_generic_to_shared(sl.store + v));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(sl.row + sl.element(v)) : "memory");
        } else {
          float x[VEC];
          sl.fetch(v, x);
          sl.keep(v, x);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      if (g == 0) asm volatile("cp.async.wait_group 3;" ::: "memory");
      if (g == 1) asm volatile("cp.async.wait_group 2;" ::: "memory");
      if (g == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (g == 3) asm volatile("cp.async.wait_group 0;" ::: "memory");
      for (int v = g * group + threadIdx.x; v < min((g + 1) * group, sl.nv); v += THREADS) {
        float x[VEC];
        sl.load(v, x);
        if (sl.mask && sl.inside(v)) {
          sl.hide(sl.element(v), x);
          sl.keep(v, x);
        }
        take(x);
      }
    }
  } else {
#pragma unroll 4
    for (int v = threadIdx.x; v < sl.nv; v += THREADS) {
      float x[VEC];
      sl.fetch(v, x);
      take(x);
    }
  }
  const float ref = top;
  float widest = top;
#pragma unroll
  for (int d = 16; d; d >>= 1) widest = max_nan(widest, __shfl_xor_sync(FULL_MASK, widest, d));
  if (lane == 0) s.redf[warp] = widest;
  __syncthreads();
  widest = s.redf[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) widest = max_nan(widest, s.redf[w]);
  float tau = -INFINITY;
  if (reach > 1 && !isnan(widest)) {
    if (RESIDENT && sl.nv < THREADS) {
      // Fewer vectors than threads: the threads' maxima of single elements instead.
      const T* flat = reinterpret_cast<const T*>(sl.store);
      top = -INFINITY;
      for (int i = threadIdx.x; i < sl.nv * VEC; i += THREADS) top = fmaxf(top, lm_float(flat[i]));
    }
    tau = block_tau(top, widest, reach, s);
  }
  if (reach == 1) tau = widest;
  sl.m = widest;
  if (need_mass) {
    // (A thread without a logit has no mass; nor has a slice, and its maximum is -inf.)
    mass = warp_sum(mass > 0.f ? mass * sl.weight(ref) : 0.f);
    if (lane == 0) s.mass[warp] = mass;
    // One vector in SAMPLE_EVERY, at a place that moves along (and so spreads over the banks).
    for (int q = threadIdx.x; q < sl.nv / SAMPLE_EVERY; q += THREADS) {
      float x[VEC];
      sl.load(q * SAMPLE_EVERY + (q & (SAMPLE_EVERY - 1)), x);
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (x[j] > -INFINITY)
          atomicAdd(&s.own_sample[static_cast<int>(fminf(-SAMPLE_SCALE * sl.x(x[j]), SAMPLE_BINS - 1.f))], 1u);
    }
  }

  // 2. The slice's first keys.
  const float* noise = a.noise + r * a.noise_ld;
  int keys = 0;
  if (want && !isnan(widest)) {
    for (int turn = 0;; ++turn) {
      sl.among(fmaxf(tau, -FLT_MAX), INFINITY, [&](float l, int64_t i) {
        const unsigned at = atomicAdd(&s.slot, 1u);
        if (at < CANDIDATES) s.candidates[at] = sl.key(l, i);
      });
      __syncthreads();
      keys = static_cast<int>(s.slot);
      if (keys <= CANDIDATES || turn == 2) break;
      // Too many (neighbours are alike, so that a thread holds several):
      // again from the want-th largest of those that were stored.
      rank_candidates(
          s, CANDIDATES, [](bool, int, u64) { return 0; },
          [&](u64 key, int rank, int) {
            if (rank == want - 1) s.thr = key;
          });
      __syncthreads();
      tau = sl.logit_of(s.thr);
      if (threadIdx.x == 0) s.slot = 0;
      __syncthreads();
    }
    if (threadIdx.x == 0 && keys <= CANDIDATES) s.candidates[keys] = 0;
  }
  __syncthreads();
  cluster.barrier_wait(std::move(started));
  if (keys > CANDIDATES) {  // copies of one value
    keys = -1;
  } else if (keys > 0) {
    // The first `want`, with their noise, go to the cluster's first CTA.
    Shared* leader = cluster.map_shared_rank(&s, 0);
    rank_candidates(
        s, keys, [&](bool some, int, u64 key) { return some && !greedy ? noise[sl.index_of(key)] : 1.f; },
        [&](u64 key, int place, float q) {
          if (place < want) {
            leader->tops[rank][place] = key;
            leader->tops_q[rank][place] = q;
          }
        });
    keys = keys < want ? keys : want;
  }
  if (need_mass)
    for (int i = threadIdx.x; i < SAMPLE_BINS * C; i += THREADS)
      cluster.map_shared_rank(&s, i / SAMPLE_BINS)->sample[rank][i % SAMPLE_BINS] = s.own_sample[i % SAMPLE_BINS];
  if (threadIdx.x < C) {
    mass = 0.f;
    if (need_mass)
#pragma unroll
      for (int w = 0; w < WARPS; ++w) mass += s.mass[w];
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
  if (want && found >= 0) {
    const bool decide = !by_k && !greedy;  // whether these keys are enough is not known beforehand
    if (rank != 0) {
      if (!decide) return;
      cluster.sync();  // the first CTA has written `enough`
    } else {
    // Merge.  (The lists' shares of `want` reach the least of them, so no key
    // below it counts.)
    const int got = found < want ? found : want, each = (want + C - 1) / C;
    u64 least = ~u64(0);
    for (int c = 0; c < C; ++c) {
      const u64 key = s.part[c].keys >= each ? s.tops[c][each - 1] : 0;
      least = key < least ? key : least;
    }
    for (int i = threadIdx.x; i < C * TOP; i += THREADS) {
      const int c = i / TOP, j = i % TOP;
      if (j >= s.part[c].keys || s.tops[c][j] < least) continue;
      const unsigned at = atomicAdd(&s.merged, 1u);
      s.candidates[at] = s.tops[c][j];
      s.candidates_q[at] = s.tops_q[c][j];
    }
    __syncthreads();
    const int merged = static_cast<int>(s.merged);
    if (threadIdx.x == 0) s.candidates[merged] = 0;
    __syncthreads();
    rank_candidates(
        s, merged, [&](bool some, int i, u64) { return some ? s.candidates_q[i] : 1.f; },
        [&](u64 key, int place, float q) {
          if (place < want) {
            s.sorted[place] = key;
            s.sorted_q[place] = q;
          }
        });
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
      if (decide && lane < C) cluster.map_shared_rank(&s, lane)->enough = enough;
      if (enough) {
        u64 kept = 0;
        Best best{-INFINITY, 0.f, NONE};
#pragma unroll
        for (int j = 0; j < EACH; ++j) {
          const int at = lane * EACH + j;
          if (at < got && (before < target || at == 0) && w[j] >= floor_w && sl.x(l[j]) > -INFINITY) {
            kept += part[j];
            better(best, Best{greedy ? 0.f : race(sl.x(l[j]), s.sorted_q[at]), l[j],
                              static_cast<unsigned>(sl.index_of(s.sorted[at]))});
          }
          before += part[j];
        }
        kept = warp_sum64(kept);
        warp_best(best);
        if (lane == 0) write_row(sl, best, kept, greedy, a.out_tokens + r, a.out_logprobs + r);
      }
    }
    if (!decide) return;
    cluster.sync();
    }
    if (s.enough) return;
  }

  if (want || by_k || by_p) {
    if (threadIdx.x == 0) {
      *reinterpret_cast<S*>(s.slice) = sl;
      s.late = Late{noise, a.out_tokens + r, a.out_logprobs + r, Z, k, p, temperature, floor_w, tau, by_k, by_p};
    }
    __syncthreads();
    late_row<S>(s);
    return;
  }

  // No filter: a race among all.
  Best best{-INFINITY, 0.f, NONE};
  u64 kept = 0;
  constexpr int AHEAD = 16 / VEC;
  const bool vec = reinterpret_cast<uintptr_t>(noise + sl.element(0)) % 16 == 0;
  for (int v = threadIdx.x; v < sl.nv; v += AHEAD * THREADS) {
    float q[AHEAD][VEC];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int u = v + i * THREADS;
      if (u >= sl.nv) break;
      const int64_t first = sl.element(u);
      if (vec && sl.inside(u)) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const float4 f = __ldcs(reinterpret_cast<const float4*>(noise + first + j));
          q[i][j] = f.x;
          q[i][j + 1] = f.y;
          q[i][j + 2] = f.z;
          q[i][j + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[i][j] = first + j >= 0 && first + j < a.n ? noise[first + j] : 1.f;
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int u = v + i * THREADS;
      if (u >= sl.nv) break;
      float x[VEC];
      sl.load(u, x);
      const unsigned first = static_cast<unsigned>(sl.element(u));
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xt = sl.x(x[j]);
        sum += lm_exp2(xt * LOG2E);
        const float score = race(xt, q[i][j]);
        // (-inf: a token that cannot be kept, or one that noise of +inf puts last.)
        if (score > best.score || (best.index == NONE && xt > -INFINITY)) best = Best{score, x[j], first + j};
      }
    }
    kept += sl.fixed(sum);
  }
  finish(sl, s, cluster, best, kept, false, a.out_tokens + r, a.out_logprobs + r);
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
