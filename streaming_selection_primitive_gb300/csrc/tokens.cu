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
// One CTA takes a row, or a cluster of up to 8 where there are few rows (then
// each takes a slice):
//   1. one read of the slice gives its maximum and, for top-p, its mass.
//      What is needed of the slice again comes from the caches;
//   2. its first keys, sorted: of the threads' maxima a value is taken that at
//      least that many of them reach, and only what lies at or above it is
//      ranked.  For top-p a sample of the row tells how many should do;
//   3. a cluster's CTAs send theirs to the first, which merges them.  For top-k
//      up to TOP, and for most rows under top-p and min-p, they are all that can
//      be kept: one warp cuts them and runs the race, which reads the noise of
//      these tokens only;
//   4. otherwise the tokens among which the cut lies are listed (for top-p those
//      between two values that the sample gives; what is above them joins the
//      race in the same pass), and a histogram of the list's counts and masses
//      over equal ranges of x, then of keys, is repeated inside the range
//      where the count or the mass crosses its target until that holds at most
//      LIST keys.  Where the sample was wrong or the list is too long, the
//      same is done over the slice.
//
// A row without filters is one pass over its logits and noise together
// (free_row).
//
// What bounds it, with the times of a call on the device (bfloat16, several sets
// of inputs in turn, beyond L2 where they are that large; logits that fall by 1 to
// 2 per unit of the logarithm of their rank):
//   many rows without filters: loads and the instructions of a token's exponential
//     and logarithm, which take turns.  512 x 65536 float32: 268 MB in 51.6 us, 5.2
//     TB/s, 0.78 of a copy's rate; 64 x 131072: 50 MB in 15.6 us;
//   many rows under top-k or greedily: the read, and step 2.  256 x 131072, 67 MB:
//     16 us greedily, 22 us with k = 50;
//   top-p: the weights of the first pass, and then the slowest row of step 4,
//     some thirty steps between barriers beside the slices' scans.  64 x 131072,
//     p = 0.9: 47 us, and 27 us at T = 0.7, where fewer rows get there;
//   top-k above what step 2 sorts: step 4 for every row.  64 x 131072, k = 1000: 68 us;
//   one row: the same chain of steps, whatever its length.  1 x 32768: 5.8 us
//     without filters, 6.7 greedily, 8.7 with k = 50, 15 with p = 0.9.
//
// Masses are summed as 64-bit integers (w scaled by a power of two up to
// 2^44, the largest that n of them cannot overflow), so that every sum is
// the same whatever order the atomics take.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <type_traits>

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
// Keys that step 2 can sort in a CTA that has the row to itself (half its
// threads; 256 x 131072, p = 0.9, T = 0.7, 24 inputs: 61 us in the median and 82 at
// most, with 128 as much in the median and 145 at most), in a
// cluster's (its lists of 128 just fit the first CTA's), and those that min-p
// seldom leaves more of (64 x 131072, min-p = 0.01: 23.3 us, and 26.9 with 128;
// 0.05 in 256 rows: 35.4 us, and 29.9 with 128).
constexpr int TOP = 256;
constexpr int TOP_SHARED = 128;
constexpr int TOP_MIN_P = 64;
constexpr int CANDIDATES = 1024;
constexpr int LISTED = 4096;    // tokens of a slice among which step 4 finds the cut,
constexpr int LISTED_ALONE = 8192;  // and of a long row in one CTA, in dynamic shared memory (256 x 131072,
                                    // p = 0.9: 119 us, and 196 with 4096)
constexpr int BINS = 256;       // of one histogram pass (64 x 131072, k = 1000: 68 us, and 73 with 128)
constexpr int SAMPLE_BINS = 128;       // of the sample of a slice,
constexpr float SAMPLE_SCALE = 8.f;    // so many a unit of x
constexpr int LIST = 128;       // keys of a bin that are ranked directly
// Bytes of a row that are worth a CTA of a cluster.  (1 x 32768 bfloat16, k = 50 and
// p = 0.9: 8.7 and 15.0 us with these four CTAs, 8.0 and 19.3 with one, 8.8 and 16.5
// with two, 10.3 and 16.8 with eight; 1 x 4096, k = 50: 7.2 us with one, 8.9 with two.)
constexpr int SLICE_LEAST = 16 << 10;
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

// What a CTA tells the others after step 1 (for top-p),
struct Part {
  float top;   // the slice's maximum (NaN if it holds one)
  float mass;  // sum of exp((l - top) / T)
};
// and after step 2.
struct Sent {
  float top;
  float tau;  // as many of its keys as were asked for reach this value
  int keys;   // sorted keys sent; -1: too many candidates to rank
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

// What scan_row tells: the best of the tokens above the list, their mass, and that of those which min-p keeps.
struct Scan {
  Best best;
  u64 mass, kept;
};

struct Shared {
  // Written by other CTAs of the cluster.
  union {
    struct {  // step 3: first keys, and their noise
      u64 tops[MAX_CLUSTER][TOP_SHARED];
      float tops_q[MAX_CLUSTER][TOP_SHARED];
    };
    struct {  // step 4
      alignas(16) unsigned merged_c[BINS];
      alignas(16) u64 merged_m[BINS];
      alignas(16) u64 list[2][LIST + 2];
    };
  };
  unsigned sample[MAX_CLUSTER][SAMPLE_BINS];
  Part part[MAX_CLUSTER];
  Sent sent[MAX_CLUSTER];
  int enough;
  Best ex_best[MAX_CLUSTER];
  u64 ex_kept[MAX_CLUSTER];
  u64 beyond[MAX_CLUSTER];  // mass above the list
  unsigned lists[MAX_CLUSTER];
  // This CTA's own.
  alignas(16) unsigned count[BINS];
  alignas(16) unsigned lo[BINS];  // 64-bit masses in two words
  alignas(16) unsigned hi[BINS];
  union {
    struct {
      alignas(16) u64 candidates[CANDIDATES + 2];
      float candidates_q[CANDIDATES];
    };
    int list_at[LISTED];  // step 4: their indices (unless they are in dynamic shared memory)
  };
  unsigned own_sample[SAMPLE_BINS];
  alignas(16) float row_sample[SAMPLE_BINS];
  u64 sorted[TOP];  // of step 3's list, or step 4's
  float sorted_q[TOP];
  u64 wc[WARPS], wm[WARPS], red[WARPS];
  float redf[WARPS], mass[WARPS];
  uint32_t redk[WARPS];
  Best best[WARPS];
  unsigned slot, merged, hits;
  int* list_to;     // the list, and its length at most
  unsigned room;
  unsigned listed;  // tokens that scan_row found for the list (which holds them unless there are more than fit)
  unsigned short hit[THREADS];
  unsigned bin;  // the crossing found by a pass: BINS if there is none
  u64 above_c, above_m, in_c, total_m;
  u64 thr, z;
  float likely[3];
  uint4 edge[2];
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

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = max_nan(v, __shfl_xor_sync(FULL_MASK, v, d));
  return v;
}

// Room for n entries of each lane of a list with the given length, which it
// moves on: the lane's first place.  One atomic a warp (a thousand of them on
// one word take microseconds); the whole warp calls it.
__device__ __forceinline__ unsigned warp_reserve(unsigned* length, int n) {
  const int lane = threadIdx.x & 31;
  int with = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(FULL_MASK, with, d);
    if (lane >= d) with += o;
  }
  unsigned base = 0;
  if (lane == 31 && with) base = atomicAdd(length, static_cast<unsigned>(with));
  return __shfl_sync(FULL_MASK, base, 31) + with - n;
}

// log2 of a positive number by the hardware's approximation; zero gives -inf.
__device__ __forceinline__ float lm_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The same for numbers of the normal range (below it: -inf).
__device__ __forceinline__ float lm_log2_normal(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats at a time.
__device__ __forceinline__ u64 pair_of(float a, float b) {
  return u64(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float pair_low(u64 a) { return __uint_as_float(static_cast<unsigned>(a)); }
__device__ __forceinline__ float pair_high(u64 a) { return __uint_as_float(static_cast<unsigned>(a >> 32)); }
__device__ __forceinline__ u64 pair_add(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 pair_mul(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A thread's sum of many weights: `part`, to which they are added, is moved to
// `whole` every so many, and what the move rounds off stays in it.  (One float
// alone drifts: a row of 2^28 with equal weights, of which a thread adds up
// 65536, gave a log-probability that was off by up to 1.9e-4, and 1.4e-6 with this;
// 64 x 131072 bfloat16 without filters take 15.5 us, and 15.2 without it.)
struct LongSum {
  static constexpr int TURNS = 16;  // of a loop over vectors, between moves
  float part = 0.f, whole = 0.f;
  __device__ __forceinline__ void add(float w) { part += w; }
  __device__ __forceinline__ void scale(float by) {
    part *= by;
    whole *= by;
  }
  __device__ __forceinline__ void move() {
    const float next = whole + part;
    part -= next - whole;
    whole = next;
  }
  // After the vectors from v on, `step` (a power of two) being what v moves by.
  __device__ __forceinline__ void turn(int v, int step) {
    const int last = (TURNS - 1) * step;
    if ((v & last) == last) move();
  }
  __device__ __forceinline__ float get() const { return whole + part; }
};

// One row as a CTA of its cluster sees it.  Positions are counted from the
// 16-byte boundary at or before the row (`phase` elements before it); a
// vector is the VEC positions from a boundary.  (Everything that reads a vector
// goes through load, and what happens at a row's ends is kept out of it: these
// kernels run most of their code once, so that its length is time.)
template <typename T>
struct Slice {
  static constexpr int VEC = 16 / int(sizeof(T));
  const T* row;
  const uint32_t* mask;
  const uint4* edge;  // shared memory: the row's first and last vector where they are not whole
  const uint4* base;  // the slice's first vector
  int n;              // of the row (an index has 32 bits: n < 2^30)
  int first;          // element of the slice's first vector's first position (may be outside the row)
  int nv;             // vectors
  int in0, in1;       // those that lie inside the row
  float m, T_, inv, inv2;   // the maximum, T, 1 / T, log2(e) / T
  float scale, unit;        // the masses' scale, and its inverse
  int index_bits, sample_shift;  // one vector in 2^sample_shift is sampled

  // First element of a vector of the slice (may be outside the row).
  __device__ __forceinline__ int element(int v) const { return first + v * VEC; }

  __device__ __forceinline__ bool is_allowed(int i) const { return !mask || (mask[i >> 5] >> (i & 31) & 1u); }

  __device__ __forceinline__ bool inside(int v) const { return v >= in0 && v < in1; }

  // -inf, in each element of a packed word.
  static constexpr unsigned NOTHING = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;

  // Elements that are not allowed become -inf, in the packed vector.
  __device__ __forceinline__ uint4 hide(int i, uint4 bits) const {
    const int at = i & 31;
    const uint32_t* w = mask + (i >> 5);
    const uint32_t ok = __funnelshift_r(w[0], at + VEC > 32 ? w[1] : 0u, at);
    unsigned* b = &bits.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        b[j] = ok >> j & 1u ? b[j] : NOTHING;
      } else {
        const unsigned keep = (ok >> 2 * j & 1u) * 0xffffu | (ok >> (2 * j + 1) & 1u) * 0xffff0000u;
        b[j] = (b[j] & keep) | (NOTHING & ~keep);
      }
    }
    return bits;
  }

  // A vector that lies inside the row.
  __device__ __forceinline__ uint4 whole(int v) const {
    const uint4 bits = __ldg(base + v);
    return mask ? hide(element(v), bits) : bits;
  }

  __device__ __forceinline__ void unpack(uint4 bits, float (&x)[VEC]) const {
    union {
      uint4 bits;
      T t[VEC];
    } u;
    u.bits = bits;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = lm_float(u.t[j]);
  }

  // The first four elements of packed ones.
  __device__ __forceinline__ void unpack4(uint4 bits, float (&x)[4]) const {
    union {
      uint4 bits;
      T t[VEC];
    } u;
    u.bits = bits;
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = lm_float(u.t[j]);
  }

  // Any vector; elements outside the row or not allowed are -inf.
  __device__ __forceinline__ void load(int v, float (&x)[VEC]) const {
    unpack(inside(v) ? whole(v) : edge[v < in0 ? 0 : 1], x);
  }

  // Element j of a vector (inside the row, allowed).
  __device__ __forceinline__ float one(int v, int j) const { return lm_float(row[element(v) + j]); }

  // body(l, i) for every element of the slice in [floor, ceil] (floor finite or
  // +inf).  A lane first marks those of several vectors and then takes them one
  // by one, so that the lanes' hits meet in the same turns.
  template <typename F>
  __device__ __forceinline__ void among(float floor, float ceil, F&& body) const {
    constexpr int GROUP = 32 / VEC;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int base = threadIdx.x - lane; base < nv; base += GROUP * THREADS) {
      unsigned hits = 0;
#pragma unroll 2
      for (int g = 0; g < GROUP; ++g) {
        const int u = base + lane + g * THREADS;
        if (u < nv) {
          float x[VEC];
          load(u, x);
          unsigned some = 0;
#pragma unroll
          for (int j = 0; j < VEC; ++j) some |= x[j] >= floor && x[j] <= ceil ? 1u << j : 0u;
          hits |= some << (g * VEC);
        }
      }
#pragma unroll 1
      for (; hits; hits &= hits - 1) {
        const int b = __ffs(hits) - 1, u = base + lane + b / VEC * THREADS;
        body(one(u, b % VEC), element(u) + b % VEC);
      }
      __syncwarp();
    }
  }

  // (l - m) / T: a NaN (an infinite maximum less itself, 0 times an infinite
  // 1 / T) is the maximum's own, 0.
  __device__ __forceinline__ float x(float l) const { return fminf((l - m) * inv, 0.f); }
  __device__ __forceinline__ float weight(float l) const { return lm_exp2(fminf((l - m) * inv2, 0.f)); }
  // Sum of a vector's weights.
  __device__ __forceinline__ float weights(const float (&x)[VEC]) const {
    float w[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[j] = weight(x[j]);
#pragma unroll
    for (int d = VEC / 2; d; d >>= 1)
#pragma unroll
      for (int j = 0; j < d; ++j) w[j] += w[j + d];
    return w[0];
  }
  // The same where neither m nor 1 / T is infinite, two at a time.
  __device__ __forceinline__ float finite_weights(const float (&x)[VEC]) const {
    const u64 less = pair_of(-m, -m), by = pair_of(inv2, inv2);
    u64 w[VEC / 2];
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) {
      const u64 y = pair_mul(pair_add(pair_of(x[2 * j], x[2 * j + 1]), less), by);
      w[j] = pair_of(lm_exp2(pair_low(y)), lm_exp2(pair_high(y)));
    }
#pragma unroll
    for (int d = VEC / 4; d; d >>= 1)
#pragma unroll
      for (int j = 0; j < d; ++j) w[j] = pair_add(w[j], w[j + d]);
    return pair_low(w[0]) + pair_high(w[0]);
  }
  __device__ __forceinline__ u64 fixed(float w) const { return __float2ull_rn(w * scale); }

  // Keys: the order key of the logit (16-bit types: its upper half) above the
  // inverted index in index_bits bits.
  static constexpr int DROP = sizeof(T) == 2 ? 13 : 0;
  __device__ __forceinline__ u64 value_key(float l) const { return u64(ord_key(l) >> DROP) << index_bits; }
  __device__ __forceinline__ u64 key(float l, int i) const {
    return value_key(l) | (((1u << index_bits) - 1u) - static_cast<unsigned>(i));
  }
  __device__ __forceinline__ int index_of(u64 key) const {
    const unsigned ones = (1u << index_bits) - 1u;
    return static_cast<int>(ones - (static_cast<unsigned>(key) & ones));
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

// Sum of the values of the threads before this one.
__device__ __forceinline__ u64 block_before64(u64 v, u64 (&sums)[WARPS]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 with = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(FULL_MASK, with, d);
    if (lane >= d) with += o;
  }
  if (lane == 31) sums[warp] = with;
  __syncthreads();
  u64 before = with - v;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) before += sums[w];
  return before;
}

// What a histogram is made of: first, the elements with logits in [floor,
// ceil], in equal ranges of x from ceil down (the last takes what is beyond);
// then those of the first one's bin `bin0` with keys in [lo, hi], in equal
// ranges of keys from hi down.
struct Level {
  float floor, ceil;
  float x0, per_x, x_per;  // -x of ceil; bins of the first per unit of x, and the inverse
  int bin0;         // -1: the first
  u64 lo, hi;
  int shift;

  template <typename S>
  __device__ __forceinline__ int bin_of(const S& sl, float l, int i) const {
    const int b = static_cast<int>(fmaxf(fminf((-sl.x(l) - x0) * per_x, BINS - 1.f), 0.f));
    if (bin0 < 0) return b;
    const u64 key = sl.key(l, i);
    return b != bin0 || key < lo || key > hi ? -1 : static_cast<int>((hi - key) >> shift);
  }
  // A value at or above all of a bin of the first, and one at or below (x's
  // roundings blur its edges by far less than half a bin).
  template <typename S>
  __device__ __forceinline__ float high(const S& sl, int bin) const {
    const float v = sl.m - (x0 + (bin - 0.5f) * x_per) * sl.T_;
    return bin > 0 && v <= ceil ? v : ceil;
  }
  template <typename S>
  __device__ __forceinline__ float low(const S& sl, int bin) const {
    const float v = sl.m - (x0 + (bin + 1.5f) * x_per) * sl.T_;
    return bin + 1 < BINS && v >= floor ? v : floor;
  }
  __device__ __forceinline__ void fit() {
    shift = 0;
#pragma unroll 1
    while (((hi - lo) >> shift) >= BINS) ++shift;
  }
};

// The histogram, joined over the cluster, and the bin where the running count
// (or mass) from the top first reaches `target`: s.bin, s.above_*, s.in_c;
// s.bin = BINS where it does not.  What lies above the first level's ceil
// counts as above (its mass only, s.beyond).  fresh: the joined histogram is in
// place.  listed: the list holds all that the first level counts.
template <typename S>
__device__ __forceinline__ void cross(const S& sl, Shared& s, cg::cluster_group& cluster, const Level& lv, bool by_mass,
                                      u64 target, bool fresh, bool listed) {
  if (!fresh) {
#pragma unroll 1
    for (int b = threadIdx.x; b < BINS; b += THREADS) s.count[b] = s.lo[b] = s.hi[b] = 0u;
    __syncthreads();
    auto add = [&](float l, int i) {
      const int b = lv.bin_of(sl, l, i);
      if (b < 0) return;
      const u64 mass = sl.fixed(sl.weight(l));
      atomicAdd(&s.count[b], 1u);
      const unsigned ml = static_cast<unsigned>(mass), old = atomicAdd(&s.lo[b], ml);
      const unsigned mh = static_cast<unsigned>(mass >> 32) + (old + ml < old ? 1u : 0u);
      if (mh) atomicAdd(&s.hi[b], mh);
    };
    if (listed) {
#pragma unroll 1
      for (int i = threadIdx.x; i < static_cast<int>(s.listed); i += THREADS) {
        const int at = s.list_to[i];
        add(lm_float(sl.row[at]), at);
      }
    } else {
      sl.among(lv.floor, lv.ceil, add);
    }
    cluster.sync();
    // This CTA joins its share of the bins: of C neighbouring threads each reads
    // four bins of one CTA, and, when they have added them up, tells one.
    const int C = cluster.num_blocks(), log_c = __ffs(C) - 1, share = BINS >> log_c, with = threadIdx.x & (C - 1);
    const Shared* from = cluster.map_shared_rank(&s, with);
    Shared* to = cluster.map_shared_rank(&s, with);
#pragma unroll 1
    for (int base = 0; base < BINS / 4; base += THREADS) {
      const int b = cluster.block_rank() * share + ((base + static_cast<int>(threadIdx.x)) >> log_c) * 4;
      const bool some = base + static_cast<int>(threadIdx.x) < BINS / 4;
      uint4 c = make_uint4(0, 0, 0, 0), ml = c, mh = c;
      if (some) {
        c = *reinterpret_cast<const uint4*>(from->count + b);
        ml = *reinterpret_cast<const uint4*>(from->lo + b);
        mh = *reinterpret_cast<const uint4*>(from->hi + b);
      }
      u64 m[4] = {(u64(mh.x) << 32) + ml.x, (u64(mh.y) << 32) + ml.y, (u64(mh.z) << 32) + ml.z, (u64(mh.w) << 32) + ml.w};
#pragma unroll 1
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
  if (lv.bin0 < 0 && lv.ceil < sl.m)
#pragma unroll 1
    for (int i = 0; i < static_cast<int>(cluster.num_blocks()); ++i) base += s.beyond[i];
  // One warp, eight neighbouring bins a lane.
  if (threadIdx.x < 32) {
    constexpr int EACH = BINS / 32;
    static_assert(EACH == 8, "eight bins a lane");
    const int first = EACH * static_cast<int>(threadIdx.x);
    u64 nc = 0, nm = 0;
#pragma unroll 1
    for (int j = 0; j < EACH; ++j) {
      nc += s.merged_c[first + j];
      nm += s.merged_m[first + j];
    }
    u64 bc = nc, bm = nm;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const u64 oc = __shfl_up_sync(FULL_MASK, bc, d), om = __shfl_up_sync(FULL_MASK, bm, d);
      if (static_cast<int>(threadIdx.x) >= d) {
        bc += oc;
        bm += om;
      }
    }
    bm += base;
    if (threadIdx.x == 31) s.total_m = bm;
    const u64 with = by_mass ? bm : bc;
    bc -= nc;
    bm -= nm;
    const bool here = (by_mass ? bm : bc) < target && target <= with;
    if (here) {
      int j = 0;
#pragma unroll 1
      for (; j + 1 < EACH; ++j) {
        const u64 c = s.merged_c[first + j], m = s.merged_m[first + j];
        if ((by_mass ? bm + m : bc + c) >= target) break;
        bc += c;
        bm += m;
      }
      s.bin = first + j;
      s.above_c = bc;
      s.above_m = bm;
      s.in_c = s.merged_c[first + j];
    }
    if (!__any_sync(FULL_MASK, here) && threadIdx.x == 0) s.bin = BINS;
  }
  __syncthreads();
}

// The key down to which tokens are kept, s.thr (every kept key >= it), and the
// mass of those, s.z: the first `target` keys from the top, or as many as it
// takes for their mass to reach it.  False: all that `lv` counts does not reach
// it (then s.total_m is its mass).
template <typename S>
__device__ bool select(const S& sl, Shared& s, cg::cluster_group& cluster, Level lv, bool by_mass, u64 target, int which,
                       bool& fresh, bool listed) {
  u64 above_c = 0, above_m = 0;
#pragma unroll 1
  for (int level = 0;; ++level) {
    cross(sl, s, cluster, lv, by_mass, target - (by_mass ? above_m : above_c), fresh && level == 0, listed);
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
    if (threadIdx.x < 32) {
      const unsigned base = __reduce_add_sync(
          FULL_MASK, static_cast<int>(threadIdx.x) < rank ? cluster.map_shared_rank(&s, threadIdx.x)->count[bin] : 0u);
      if (threadIdx.x == 0) s.slot = base;
    }
    __syncthreads();
    const float floor = lv.bin0 < 0 ? lv.low(sl, bin) : lv.floor, ceil = lv.bin0 < 0 ? lv.high(sl, bin) : lv.ceil;
    auto send = [&](u64 key) {
      const unsigned at = atomicAdd(&s.slot, 1u);
      if (at < LIST)
#pragma unroll 1
        for (int c = 0; c < C; ++c) cluster.map_shared_rank(&s, c)->list[which][at] = key;
    };
    if (s.count[bin] != 0u) {
      if (listed) {
#pragma unroll 1
        for (int i = threadIdx.x; i < static_cast<int>(s.listed); i += THREADS) {
          const int at = s.list_to[i];
          const float l = lm_float(sl.row[at]);
          if (lv.bin_of(sl, l, at) == bin) send(sl.key(l, at));
        }
      } else {
        sl.among(floor, ceil, [&](float l, int i) {
          if (lv.bin_of(sl, l, i) == bin) send(sl.key(l, i));
        });
      }
    }
    cluster.sync();
    // Rank of each key: the number of larger ones.  (Two at a time: an odd number
    // is followed by a 0.)
    const int m = static_cast<int>(in_c);
    u64* list = s.list[which];
    static_assert(LIST <= THREADS, "a key a thread");
    if (threadIdx.x == 0) list[m] = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < m) {
      const u64 mine = list[threadIdx.x];
      int above = 0;
#pragma unroll 2
      for (int i = 0; i < m; i += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(list + i);
        above += (o.x > mine) + (o.y > mine);
      }
      s.sorted[above] = mine;
    }
    __syncthreads();
    // The masses before each, in that order.
    const int at = threadIdx.x;
    const u64 mass = at < m ? sl.fixed(sl.weight(sl.logit_of(s.sorted[at]))) : 0;
    const u64 before = above_m + block_before64(mass, s.wm);
    const u64 b = by_mass ? before : above_c + at, w = b + (by_mass ? mass : 1);
    if (at < m && b < target && target <= w) {
      s.thr = s.sorted[at];
      s.z = before + mass;
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
#pragma unroll 1
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
  int log_split = 0;
#pragma unroll 1
  while (log_split < 3 && keys << (log_split + 1) <= THREADS) ++log_split;
  const int split = 1 << log_split, sub = threadIdx.x & (split - 1);
#pragma unroll 1
  for (int base = 0; base < keys; base += THREADS >> log_split) {
    const int i = base + (threadIdx.x >> log_split);
    const u64 mine = i < keys ? s.candidates[i] : ~u64(0);
    const auto what = begin(i < keys && sub == 0, i, mine);
    int above = 0;
#pragma unroll 2
    for (int j = 2 * sub; j < keys; j += 2 * split) {
      const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(s.candidates + j);
      above += (o.x > mine) + (o.y > mine);
    }
#pragma unroll 1
    for (int d = split >> 1; d; d >>= 1) above += __shfl_xor_sync(FULL_MASK, above, d);
    if (i < keys && sub == 0) body(mine, above, what);
  }
}

// A higher limit for the slice's keys from `least` on, of which there are more
// than can be ranked: the want-th largest of an even share of them, one in so
// many in the order of the threads with a hit (flat: of the vectors).  (What the
// count that found them too many has stored by then depends on the order of the
// warps, and so would the limit.  64 x 131072 bfloat16 in ascending order, k = 50:
// 103 us, and 151 with the first that were stored.)
template <typename S>
__device__ __noinline__ float higher_limit(Shared& s, float least, bool flat, int shift, int want) {
  const S sl = *reinterpret_cast<const S*>(s.slice);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!flat) {  // s.hit in the threads' order
    if (threadIdx.x < WARPS) s.redk[threadIdx.x] = 0u;
    const int hits = static_cast<int>(s.hits), mine = static_cast<int>(threadIdx.x) < hits ? s.hit[threadIdx.x] : 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < hits) atomicOr(&s.redk[mine >> 5], 1u << (mine & 31));
    __syncthreads();
    const unsigned before = s.redk[warp] & ((1u << lane) - 1u);
    if (s.redk[warp] >> lane & 1u) {
      unsigned at = __popc(before);
#pragma unroll 1
      for (int w = 0; w < warp; ++w) at += __popc(s.redk[w]);
      s.hit[at] = static_cast<unsigned short>(threadIdx.x);
    }
    __syncthreads();
  }
  const int vectors = flat ? sl.nv : static_cast<int>(s.hits) << shift;
  auto vector = [&](int i) {
    return i >= vectors ? sl.nv : flat ? i : s.hit[i >> shift] + (i & ((1 << shift) - 1)) * THREADS;
  };
  auto marks = [&](int v) {
    unsigned some = 0;
    if (v < sl.nv) {
      float x[S::VEC];
      sl.load(v, x);
#pragma unroll
      for (int j = 0; j < S::VEC; ++j) some |= x[j] >= least ? 1u << j : 0u;
    }
    return some;
  };
  int mine = 0;
#pragma unroll 1
  for (int i = threadIdx.x; i < vectors; i += THREADS) mine += __popc(marks(vector(i)));
  mine = __reduce_add_sync(FULL_MASK, mine);
  if (lane == 0) s.redk[warp] = mine;
  __syncthreads();
  unsigned rank = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) rank += s.redk[w];
    all += s.redk[w];
  }
  const unsigned step = (all + CANDIDATES - 1) / CANDIDATES;
#pragma unroll 1
  for (int base = threadIdx.x - lane; base < vectors; base += THREADS) {
    const int v = vector(base + lane);
    unsigned some = marks(v);
    const int n = __popc(some);
    int with = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(FULL_MASK, with, d);
      if (lane >= d) with += o;
    }
    unsigned at = rank + with - n;
    rank += __shfl_sync(FULL_MASK, with, 31);
#pragma unroll 1
    for (; some; some &= some - 1, ++at)
      if (at % step == 0) s.candidates[at / step] = sl.key(sl.one(v, __ffs(some) - 1), sl.element(v) + __ffs(some) - 1);
    __syncwarp();
  }
  const int stored = static_cast<int>((all + step - 1) / step);
  if (threadIdx.x == 0) s.candidates[stored] = 0;
  __syncthreads();
  rank_candidates(
      s, stored, [](bool, int, u64) { return 0; },
      [&](u64 key, int place, int) {
        if (place == want - 1) s.thr = key;
      });
  __syncthreads();
  return sl.logit_of(s.thr);
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
  *logprob = greedy ? 0.f : sl.x(best.logit) - logf(static_cast<float>(kept) * sl.unit);
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
  if (threadIdx.x < 32) {
    best = s.best[threadIdx.x & (WARPS - 1)];
    warp_best(best);
    if (threadIdx.x == 0) {
      Shared* leader = cluster.map_shared_rank(&s, 0);
      leader->ex_best[rank] = best;
      leader->ex_kept[rank] = kept;
    }
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
#pragma unroll 1
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
  lv.x_per = fmaxf(reach - lv.x0, 1e-4f) * (1.f / BINS);
  lv.per_x = lm_rcp(lv.x_per);
  return lv;
}

// Where (in x below the maximum) the slices' samples put the point under which
// `left` of mass lies: s.likely[0] surely further than that, and, where the
// tokens above are many, s.likely[1] surely nearer (else 0); s.likely[2] the
// number of tokens above.  Surely: by four standard deviations of the sample's
// sum below the point.
template <typename S>
__device__ __forceinline__ void sample_point(const S& sl, Shared& s, float left) {
  const float every = static_cast<float>(1 << sl.sample_shift);
  constexpr int EACH = SAMPLE_BINS / 32;
  const int C = cg::this_cluster().num_blocks();
  if (threadIdx.x < SAMPLE_BINS) {
    unsigned sum = 0;
#pragma unroll 1
    for (int c = 0; c < C; ++c) {
      // Bins of a slice count from its own maximum.
      const int b = static_cast<int>(threadIdx.x) -
                    static_cast<int>(fminf(-SAMPLE_SCALE * sl.x(s.part[c].top), SAMPLE_BINS) + 0.5f);
      if (b >= 0) sum += s.sample[c][b];
    }
    s.row_sample[threadIdx.x] = static_cast<float>(sum);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const float4 four = reinterpret_cast<const float4*>(s.row_sample)[lane];
    static_assert(EACH == 4, "four bins a lane");
    const float count[EACH] = {four.x, four.y, four.z, four.w};
    // Mass and its variance, of a lane's bins and all below; tokens, of those above.
    float weight[EACH], mass[EACH], tail = 0.f, var = 0.f, tokens = 0.f;
#pragma unroll
    for (int j = 0; j < EACH; ++j) {
      weight[j] = every * __expf(-(EACH * lane + j + 0.5f) / SAMPLE_SCALE);
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
    float far = -1.f, near = 0.f, above = 0.f;
#pragma unroll
    for (int j = EACH - 1; j >= 0; --j) {
      if (tail <= left && left < tail + mass[j]) {
        const float point = (EACH * lane + j + 1 - __fdividef(left - tail, mass[j])) / SAMPLE_SCALE;
        const float blur = 0.02f + __fdividef(4.f * lm_sqrt(var + weight[j] * mass[j]), mass[j] * SAMPLE_SCALE);
        far = point + blur;
        above = tokens;
#pragma unroll
        for (int i = 0; i < j; ++i) above += count[i];
        above *= every;
        near = above > static_cast<float>(C * (s.room / 2)) ? fmaxf(point - blur, 0.f) : 0.f;
      }
      tail += mass[j];
      var += mass[j] * weight[j];
    }
    const unsigned which = __ballot_sync(FULL_MASK, far >= 0.f);
    if (which == 0u) far = INFINITY;  // the sample has no answer
    if (which == 0u ? lane == 0 : lane == __ffs(which) - 1) {
      s.likely[0] = far;
      s.likely[1] = near;
      s.likely[2] = above;
    }
  }
  __syncthreads();
}

// The slice's tokens in [floor, inf], to the list (s.listed counts them, and is 0
// before).  The lanes first mark those of several vectors.
template <typename S>
__device__ __forceinline__ void list_row(const S& sl, Shared& s, float floor) {
  constexpr int VEC = S::VEC, GROUP = 32 / VEC;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int base = threadIdx.x - lane; base < sl.nv; base += GROUP * THREADS) {
    unsigned hits = 0;
#pragma unroll 2
    for (int g = 0; g < GROUP; ++g) {
      const int u = base + lane + g * THREADS;
      if (u < sl.nv) {
        float x[VEC];
        sl.load(u, x);
#pragma unroll
        for (int j = 0; j < VEC; ++j) hits |= x[j] >= floor ? 1u << (g * VEC + j) : 0u;
      }
    }
    unsigned at = warp_reserve(&s.listed, __popc(hits));
#pragma unroll 1
    for (; hits; hits &= hits - 1, ++at) {
      const int b = __ffs(hits) - 1, u = base + lane + b / VEC * THREADS;
      if (at < s.room) s.list_to[at] = sl.element(u) + b % VEC;
    }
    __syncwarp();
  }
}

// One pass over the slice and its noise: the race of the tokens above `cut` (its
// copies up to cut_index included: none if that is NO_COPY) with a weight of floor_w or more, and a
// list of those in [floor, cut] that are not above.  The noise is read for
// all, not to wait for the logits first: where a tenth is kept every sector of
// it is touched anyway.  Scores are in units of log 2; the best of four
// elements is looked for where it beats the thread's.  (Four at a time: eight
// need more registers than there are.)
constexpr int NO_COPY = INT_MIN;  // below every position: a row that starts off the 16-byte boundary has some below 0
template <typename S>
__device__ __noinline__ Scan scan_row(Shared& s, float cut, int cut_index, float floor) {
  constexpr int VEC = S::VEC, PARTS = VEC / 4;
  const S sl = *reinterpret_cast<const S*>(s.slice);
  const float* noise = s.late.noise + sl.first;
  const float floor_w = s.late.floor_w;
  const bool draw = s.late.temperature != 0.f;
  const bool vec = reinterpret_cast<uintptr_t>(noise) % 16 == 0;
  const int lane = threadIdx.x & 31;
  const float next = key_to_float(ord_key(cut) + 1u);  // (NaN above +inf)
  if (cut == -INFINITY) cut_index = NO_COPY;           // what is not allowed
  Best best{-INFINITY, 0.f, NONE};
  u64 mass = 0, kept = 0;
  float sum = 0.f, sum_kept = 0.f;
  int turn = 0;
#pragma unroll 1
  for (int base = threadIdx.x - lane; base < sl.nv; base += THREADS) {
    const int v = base + lane, at = v * VEC;
    const bool some_here = v < sl.nv, in = some_here && sl.inside(v);
    float4 q[PARTS];
    uint4 bits;
    if (!draw) {
#pragma unroll
      for (int h = 0; h < PARTS; ++h) q[h] = make_float4(1.f, 1.f, 1.f, 1.f);
    } else if (in && vec) {
#pragma unroll
      for (int h = 0; h < PARTS; ++h) q[h] = __ldcs(reinterpret_cast<const float4*>(noise + at) + h);
    } else {
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        float* to = &q[h].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = sl.first + at + 4 * h + j;
          to[j] = some_here && i >= 0 && i < sl.n ? noise[at + 4 * h + j] : 1.f;
        }
      }
    }
    if (some_here) bits = in ? sl.whole(v) : sl.edge[v < sl.in0 ? 0 : 1];
    unsigned list = 0;
    if (!some_here) bits = make_uint4(S::NOTHING, S::NOTHING, S::NOTHING, S::NOTHING);
#pragma unroll 1
    for (int h = 0; h < PARTS; ++h) {
      float x[4];
      sl.unpack4(bits, x);
      const float qs[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
      const int first = sl.first + at + 4 * h;
      // Above: from the cut on up to its index, from the next value on after it.
      const float least = first <= cut_index ? cut : next;
      float y[4], w[4], score[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = x[j] >= least ? fminf((x[j] - sl.m) * sl.inv2, 0.f) : -INFINITY;
        list |= x[j] >= floor && !(x[j] >= least) ? 1u << (4 * h + j) : 0u;
      }
      if (first <= cut_index && cut_index < first + 3) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (first + j > cut_index && x[j] == cut) y[j] = -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = lm_exp2(y[j]);
        score[j] = y[j] - lm_log2_normal(qs[j]);
      }
      sum += (w[0] + w[1]) + (w[2] + w[3]);
      if (floor_w > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum_kept += w[j] >= floor_w ? w[j] : 0.f;
          if (w[j] < floor_w) y[j] = score[j] = -INFINITY;
        }
      }
      const float most = fmaxf(fmaxf(score[0], score[1]), fmaxf(score[2], score[3]));  // (NaN noise is never ahead)
      const float least_q = fminf(fminf(qs[0], qs[1]), fminf(qs[2], qs[3]));
      if (least_q < FLT_MIN || (most == -INFINITY && best.index == NONE)) {
        // Noise below the normal range, or a first token that is behind all others.
        if (fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) > -INFINITY) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float exact = fmaxf(y[j] - lm_log2(qs[j]), -INFINITY);
            if (y[j] > -INFINITY && (exact > best.score || best.index == NONE))
              best = Best{exact, x[j], static_cast<unsigned>(first + j)};
          }
        }
      } else if (most > best.score) {
        int which = 3;
        float l = x[3];
#pragma unroll
        for (int j = 2; j >= 0; --j)
          if (score[j] == most) {
            which = j;
            l = x[j];
          }
        best = Best{most, l, static_cast<unsigned>(first + which)};
      }
      if constexpr (PARTS > 1) {
        bits.x = bits.z;
        bits.y = bits.w;
        q[0] = q[PARTS - 1];
      }
    }
    if (__any_sync(FULL_MASK, list != 0u)) {
      unsigned place = warp_reserve(&s.listed, __popc(list));
#pragma unroll 1
      for (; list; list &= list - 1, ++place)
        if (place < s.room) s.list_to[place] = sl.first + at + __ffs(list) - 1;
      __syncwarp();
    }
    if (++turn % 16 == 0) {
      mass += sl.fixed(sum);
      kept += sl.fixed(sum_kept);
      sum = sum_kept = 0.f;
    }
  }
  mass += sl.fixed(sum);
  return Scan{best, mass, floor_w > 0.f ? kept + sl.fixed(sum_kept) : mass};
}

// 4. A list of the tokens among which the cuts lie: for top-k from a value that
// k keys of one slice reach; for top-p from the sample's, or from the one at
// which n tokens together weigh less than what may be left out.  The cuts are
// found in it, and what they leave joins the race.  Where the sample says that
// the tokens above its point are too many for a list, the pass that makes it
// races over them at once.  A list that is too long all the same is done
// without: then each step reads the slice.  (A function of its own: the
// registers that it needs would be spilled by rows that never come here, at a
// microsecond a row.)
template <typename S>
__device__ __noinline__ void late_row(Shared& s) {
  static_assert(sizeof(S) <= sizeof(s.slice), "room for the slice");
  const S sl = *reinterpret_cast<const S*>(s.slice);
  const Late& late = s.late;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks();
  const float temperature = late.temperature, top = sl.m, floor_w = late.floor_w;
  const bool greedy = temperature == 0.f, cuts = late.by_k || late.by_p, sampled = late.by_p && !late.by_k;
  u64 Z = late.Z;
  u64 thr = 0;
  // The least logit that min-p can keep (with room for its and the weights' roundings).
  const float lowest = greedy          ? top
                       : floor_w > 0.f ? fminf(top, top + temperature * (1.001f * __logf(floor_w) - 1e-3f))
                                       : -INFINITY;
  const float left = (1.f - fmaxf(late.p, 0.f)) * (static_cast<float>(Z) * sl.unit);
  const float sure = !cuts ? lowest
                     : !sampled
                         ? late.tau
                         : top - temperature * __logf(__fdividef(static_cast<float>(sl.n), 0.99f * left));
  const float far = sampled ? top - temperature * s.likely[0] : sure;
  const float ceil = sampled && s.likely[1] > 0.f ? top - temperature * s.likely[1] : top;
  // From the narrowest range to the widest, tried one after another.
  Level lv = far <= top && far > sure ? level_between(sl, far, ceil) : level_between(sl, sure, top);
  if (lv.floor == -FLT_MAX) lv = level_between(sl, -INFINITY, top);
  const bool dense = greedy || lv.ceil < top, list = !greedy && lv.floor > -FLT_MAX;
  if (threadIdx.x == 0) s.listed = 0;
  __syncthreads();
  Scan scan{Best{-INFINITY, 0.f, NONE}, 0, 0};
  if (dense) {
    // The noise is on its way to L2 before the loads ask for it.  (512 x 65536 float32,
    // p = 0.9: 125 us, and 128 without.)
    const float* noise = late.noise;
#pragma unroll 1
    for (int i = max(sl.first, 0) + 32 * static_cast<int>(threadIdx.x); i < min(sl.first + sl.nv * S::VEC, sl.n); i += 32 * THREADS)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(noise + i));
    scan = scan_row<S>(s, greedy ? top : lv.ceil, greedy ? sl.n : NO_COPY, greedy ? INFINITY : lv.floor);
  } else if (list) {  // (from the row's bottom on it would be too long)
    list_row(sl, s, lv.floor);
  }
  bool listed = list;
  if (list) {
    const u64 mass = block_sum64(scan.mass, s);
    if (threadIdx.x < C) {
      Shared* to = cluster.map_shared_rank(&s, threadIdx.x);
      to->beyond[cluster.block_rank()] = mass;
      to->lists[cluster.block_rank()] = s.listed;
    }
    cluster.sync();
#pragma unroll 1
    for (int c = 0; c < C; ++c) listed = listed && s.lists[c] <= s.room;
  }
  if (cuts) {
    bool fresh = false;
#pragma unroll 1
    for (int turn = late.by_k ? 0 : 1; turn < (late.by_p ? 2 : 1); ++turn) {  // the first k, then their share p
      const u64 target = turn ? mass_target(late.p, Z) : static_cast<u64>(late.k);
      bool cut;
#pragma unroll 1
      for (;;) {
        __syncthreads();  // what the turn before left in s has been read
        cut = select(sl, s, cluster, lv, turn == 1, target, turn, fresh, listed);
        if (cut || turn == 0 || lv.floor == -FLT_MAX) break;
        // The sample's answer was wrong, or roundings used up what the sure floor
        // leaves out.
        lv = level_between(sl, lv.floor > sure ? sure : -INFINITY, top);
        fresh = listed = false;
      }
      // Without a cut: there are no more than k, or Z's rounding asks for more
      // mass than there is, so that everything stays.
      if (turn == 0) Z = cut ? s.z : s.total_m;
      if (cut && s.thr > thr) thr = s.thr;
    }
  }
  if (listed) {
#pragma unroll 2
    for (int i = threadIdx.x; i < static_cast<int>(s.listed); i += THREADS) {
      const int at = s.list_to[i];
      const float l = lm_float(sl.row[at]), q = late.noise[at], w = sl.weight(l), x2 = fminf((l - sl.m) * sl.inv2, 0.f);
      if (sl.key(l, at) < thr || w < floor_w || x2 == -INFINITY) continue;
      scan.kept += sl.fixed(w);
      better(scan.best, Best{fmaxf(x2 - lm_log2(q), -INFINITY), l, static_cast<unsigned>(at)});
    }
  } else if (!greedy) {
    const float end = thr ? sl.logit_of(thr) : -INFINITY;
    const bool by_thr = end >= lowest;
    scan = scan_row<S>(s, by_thr ? end : lowest, by_thr && thr ? sl.index_of(thr) : sl.n, INFINITY);
  }
  finish(sl, s, cluster, scan.best, scan.kept, greedy, late.token, late.logprob);
}

// The first `want` keys of the cluster's lists into s.sorted.  (The lists'
// shares of `want` reach the least of them, so no key below it counts.)
__device__ __forceinline__ void merge_keys(Shared& s, int C, int want) {
  const int each = (want + C - 1) >> (__ffs(C) - 1);
  u64 least = ~u64(0);
#pragma unroll 1
  for (int c = 0; c < C; ++c) {
    const u64 key = s.sent[c].keys >= each ? s.tops[c][each - 1] : 0;
    least = key < least ? key : least;
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < C * TOP_SHARED; i += THREADS) {
    const int c = i / TOP_SHARED, j = i % TOP_SHARED;
    if (j >= s.sent[c].keys || s.tops[c][j] < least) continue;
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
}

// The race over the list s.sorted[0 .. got) (one warp): the tokens before which
// the mass is below the target, and whose weight is at least floor_w.  False,
// without a race, if the list does not hold all of them: `whole` says that
// it does in any case; otherwise it has to reach the mass or to fall below
// floor_w.  by_k: the mass is the list's.
template <typename S>
__device__ __forceinline__ bool race_list(const S& sl, const Shared& s, int got, bool whole, bool by_k, bool by_p, float p,
                                          u64 Z, float floor_w, bool greedy, int64_t* token, float* logprob) {
  // A lane takes neighbouring keys, so that one scan over the lanes does.
  const int lane = threadIdx.x & 31, each = (got + 31) >> 5, first = lane * each, end = min(first + each, got);
  u64 mine = 0;
#pragma unroll 1
  for (int at = first; at < end; ++at) mine += sl.fixed(sl.weight(sl.logit_of(s.sorted[at])));
  u64 above = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const u64 o = __shfl_up_sync(FULL_MASK, above, d);
    if (lane >= d) above += o;
  }
  const u64 total = __shfl_sync(FULL_MASK, above, 31);
  above -= mine;
  const u64 target = by_p ? mass_target(p, by_k ? total : Z) : ~u64(0);
  const float last = got ? sl.weight(sl.logit_of(s.sorted[got - 1])) : 0.f;
  if (!whole && !(by_p && total >= target) && !(last < floor_w)) return false;
  u64 kept = 0;
  Best best{-INFINITY, 0.f, NONE};
#pragma unroll 1
  for (int at = first; at < end && (above < target || at == 0); ++at) {
    const u64 key = s.sorted[at];
    const float l = sl.logit_of(key), w = sl.weight(l), x = sl.x(l);
    const u64 part = sl.fixed(w);
    above += part;
    if (!(w >= floor_w) || x == -INFINITY) continue;
    kept += part;
    better(best, Best{greedy ? 0.f : race(x, s.sorted_q[at]), l, static_cast<unsigned>(sl.index_of(key))});
  }
  kept = warp_sum64(kept);
  warp_best(best);
  if (lane == 0) write_row(sl, best, kept, greedy, token, logprob);
  return true;
}

// Running maximum (NaN if there is one) over whole vectors of logits.
template <typename T>
struct VectorMax {
  static_assert(sizeof(T) == 4);
  float m = -INFINITY;
  __device__ __forceinline__ void take(uint4 b) {
    m = max_nan(max_nan(m, max_nan(__uint_as_float(b.x), __uint_as_float(b.y))),
                max_nan(__uint_as_float(b.z), __uint_as_float(b.w)));
  }
  __device__ __forceinline__ float get() const { return m; }
};
__device__ __forceinline__ __nv_bfloat162 pair_max(__nv_bfloat162 a, unsigned b) {
  return __hmax2_nan(a, *reinterpret_cast<__nv_bfloat162*>(&b));
}
__device__ __forceinline__ __half2 pair_max(__half2 a, unsigned b) { return __hmax2_nan(a, *reinterpret_cast<__half2*>(&b)); }
template <typename P>
struct PairMax {  // two 16-bit values at a time
  P m;
  __device__ __forceinline__ PairMax(P lowest) : m(lowest) {}
  __device__ __forceinline__ void take(uint4 b) { m = pair_max(pair_max(pair_max(pair_max(m, b.x), b.y), b.z), b.w); }
  __device__ __forceinline__ float get() const { return max_nan(lm_float(m.x), lm_float(m.y)); }
};
template <>
struct VectorMax<__nv_bfloat16> : PairMax<__nv_bfloat162> {
  __device__ __forceinline__ VectorMax() : PairMax(__float2bfloat162_rn(-INFINITY)) {}
};
template <>
struct VectorMax<__half> : PairMax<__half2> {
  __device__ __forceinline__ VectorMax() : PairMax(__float2half2_rn(-INFINITY)) {}
};

// A row without filters, in one pass: a thread's mass and best score stand
// relative to the largest of its logits so far, `ref`; when that moves, the
// mass is scaled, and the best's score is computed anew from its logit and
// noise, so that all scores come from one formula and at last from the row's
// maximum.
// MASKED: the row has a mask.  (Asked of each vector instead, it lets the compiler
// put the waits for the logits between their loads: 512 x 65536 float32 took 51 or
// 65 us, as other code of the kernel changed.)
template <bool MASKED, typename S, typename Started>
__device__ __forceinline__ void free_row(S& sl, Shared& s, cg::cluster_group& cluster, Started&& started,
                                         const float* noise, float temperature, bool refused, int64_t* token,
                                         float* logprob) {
  constexpr int VEC = S::VEC, AHEAD = 16 / VEC;  // vectors under way a thread
  const int C = cluster.num_blocks(), rank = cluster.block_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool vec = reinterpret_cast<uintptr_t>(noise + sl.first) % 16 == 0;
  float ref = -INFINITY, top = -INFINITY, best_lq = 0.f;
  LongSum mass;
  Best best{-INFINITY, 0.f, NONE};
  auto x2 = [&](float l) { return fminf((l - ref) * sl.inv2, 0.f); };
  auto move = [&](float to) {
    mass.scale(lm_exp2(fminf((ref - to) * sl.inv2, 0.f)));
    ref = to;
    const float y = x2(best.logit);
    if (y == -INFINITY) best.index = NONE;  // it weighs nothing beside `to`
    best.score = best.index == NONE ? -INFINITY : fmaxf(y - best_lq, -INFINITY);
  };
  auto one = [&](int i) {  // an element by itself: a row's ends, and what the vectors leave
    if (!sl.is_allowed(i)) return;
    const float l = lm_float(sl.row[i]);
    top = max_nan(top, l);
    if (!(l > -INFINITY)) return;
    if (l > ref) move(l);
    const float y = x2(l);
    if (y == -INFINITY) return;  // it weighs nothing
    mass.add(lm_exp2(y));
    const float lq = lm_log2(noise[i]), score = fmaxf(y - lq, -INFINITY);  // NaN noise is never ahead
    if (score > best.score || best.index == NONE || (score == best.score && static_cast<unsigned>(i) < best.index)) {
      best = Best{score, l, static_cast<unsigned>(i)};
      best_lq = isnan(lq) ? INFINITY : lq;
    }
  };
#pragma unroll 1
  for (int v = threadIdx.x; v < sl.nv; v += AHEAD * THREADS) {
    uint4 bits[AHEAD];
    float q[AHEAD][VEC];
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
      const int u = v + g * THREADS;
      if (!sl.inside(u)) continue;
      bits[g] = MASKED ? sl.hide(sl.element(u), __ldg(sl.base + u)) : __ldg(sl.base + u);
      const float* from = noise + sl.element(u);
      if (vec) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const float4 f = __ldcs(reinterpret_cast<const float4*>(from + j));
          q[g][j] = f.x;
          q[g][j + 1] = f.y;
          q[g][j + 2] = f.z;
          q[g][j + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[g][j] = __ldcs(from + j);
      }
    }
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) {
      const int u = v + g * THREADS;
      if (!sl.inside(u)) continue;
      float x[VEC], most = -INFINITY, least_q = FLT_MAX, peak = -INFINITY;
      sl.unpack(bits[g], x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        peak = max_nan(peak, x[j]);
        least_q = fminf(least_q, q[g][j]);
      }
      top = max_nan(top, peak);
      if (peak > ref) move(peak);
      if (ref == -INFINITY) continue;
      float w[VEC], score[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float y = x2(x[j]);
        w[j] = lm_exp2(y);
        score[j] = y - lm_log2_normal(q[g][j]);
        most = fmaxf(most, score[j]);
      }
#pragma unroll
      for (int d = VEC / 2; d; d >>= 1)
#pragma unroll
        for (int j = 0; j < d; ++j) w[j] += w[j + d];
      if (least_q < FLT_MIN || (best.index == NONE && most == -INFINITY)) {
        // Noise below the normal range, or a first token that is behind all others.
#pragma unroll 1
        for (int j = 0; j < VEC; ++j) one(sl.element(u) + j);
        continue;
      }
      mass.add(w[0]);
      if (most > best.score) {
        int at = VEC - 1;
        float l = x[VEC - 1], noise_there = q[g][VEC - 1];
#pragma unroll
        for (int j = VEC - 2; j >= 0; --j)
          if (score[j] == most) {
            at = j;
            l = x[j];
            noise_there = q[g][j];
          }
        best = Best{most, l, static_cast<unsigned>(sl.element(u) + at)};
        best_lq = lm_log2_normal(noise_there);
      }
    }
    mass.turn(v, AHEAD * THREADS);
  }
  if (threadIdx.x < 2 * VEC) {
    const int which = threadIdx.x / VEC, v = which ? sl.nv - 1 : 0, i = sl.element(v) + static_cast<int>(threadIdx.x % VEC);
    if (sl.nv > 0 && !sl.inside(v) && (which == 0 ? sl.element(v) < 0 : sl.element(v) >= 0) && i >= 0 && i < sl.n) one(i);
  }
  // The row's maximum.
  top = warp_max_nan(top);
  if (lane == 0) s.redf[warp] = top;
  __syncthreads();
  top = warp_max_nan(s.redf[lane & (WARPS - 1)]);
  cluster.barrier_wait(std::move(started));
  if (threadIdx.x < C) cluster.map_shared_rank(&s, threadIdx.x)->part[rank] = Part{top, 0.f};
  cluster.sync();
#pragma unroll 1
  for (int i = 0; i < C; ++i) top = max_nan(top, s.part[i].top);
  const bool bad = refused || isnan(top) || !(temperature >= 0.f);
  if (bad || top == -INFINITY) {
    if (rank == 0 && threadIdx.x == 0) {
      *token = -1;
      *logprob = bad ? __int_as_float(0x7fc00000) : -INFINITY;
    }
    return;
  }
  sl.m = top;
  if (ref > -INFINITY) move(top);
  finish(sl, s, cluster, best, __float2ull_rn(mass.get() * sl.scale), false, token, logprob);
}

template <typename T>
__device__ __forceinline__ void sample_row(const TokenArgs& a, int64_t r, int per_cta, Shared& s) {
  using S = Slice<T>;
  constexpr int VEC = S::VEC;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = cluster.num_blocks(), rank = cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s.slot = s.merged = s.hits = 0;
  if (threadIdx.x < SAMPLE_BINS) s.own_sample[threadIdx.x] = 0u;
  auto started = cluster.barrier_arrive();  // waited for before the first write to another CTA
  const float temperature = a.temperature ? a.temperature[r] : a.all_temperature;
  const int32_t k = a.top_k ? a.top_k[r] : a.all_top_k;
  const float p = a.top_p ? a.top_p[r] : a.all_top_p;
  const float min_p = a.min_p ? a.min_p[r] : a.all_min_p;
  const bool greedy = temperature == 0.f;
  const bool by_k = !greedy && k > 0 && k < a.n, by_p = !greedy && p < 1.f;
  const bool need_mass = by_p && !by_k, alone = C == 1;
  // Keys that step 2 sorts (0: it would not help); for top-p in a CTA alone the sample may say otherwise.
  int want = greedy ? 1 : by_k ? (k <= (alone ? TOP : TOP_SHARED) ? k : 0) : min_p > 0.f ? TOP_MIN_P : by_p ? TOP_SHARED : 0;
  S sl;
  sl.row = static_cast<const T*>(a.logits) + r * a.ld;
  sl.mask = a.mask ? a.mask + r * a.mask_ld : nullptr;
  sl.edge = s.edge;
  sl.n = static_cast<int>(a.n);
  const int phase_of_row = static_cast<int>(reinterpret_cast<uintptr_t>(sl.row) % 16 / sizeof(T));
  const int all = (sl.n + phase_of_row + VEC - 1) / VEC, v0 = rank * per_cta;
  sl.nv = max(min(all - v0, per_cta), 0);
  sl.first = v0 * VEC - phase_of_row;
  sl.base = reinterpret_cast<const uint4*>(sl.row - phase_of_row) + v0;
  sl.in0 = sl.first < 0 ? 1 : 0;
  sl.in1 = min(sl.nv, (sl.n - sl.first) / VEC);
  // An infinite T: the smallest number, so that -inf stays -inf.
  sl.T_ = temperature;
  sl.inv = fmaxf(lm_rcp(temperature), __int_as_float(1));
  sl.inv2 = sl.inv * LOG2E;
  sl.index_bits = 32 - __clz(sl.n - 1);
  sl.sample_shift = min(max(sl.index_bits - 14, 0), 6);  // 8192 to 16384 elements of the row, where it has them
  const int e = min(62 - sl.index_bits, 44);
  sl.scale = __int_as_float((127 + e) << 23);
  sl.unit = __int_as_float((127 - e) << 23);
  const float* noise = a.noise + r * a.noise_ld;
  if (!greedy && !by_k && !by_p && !(min_p > 0.f)) {
    const bool refused = isnan(p) || isnan(min_p);
    if (sl.mask)
      free_row<true>(sl, s, cluster, std::move(started), noise, temperature, refused, a.out_tokens + r, a.out_logprobs + r);
    else
      free_row<false>(sl, s, cluster, std::move(started), noise, temperature, refused, a.out_tokens + r, a.out_logprobs + r);
    return;
  }

  // 1. The slice's largest logit (NaN if it holds one) and, for top-p, its
  // mass: a thread's sum of exp((l - ref) / T), ref being the largest of its
  // logits so far.
  float top = -INFINITY, mass = 0.f, own;  // own: of the thread's whole vectors
  {
    LongSum sum;
    VectorMax<T> packed;
    auto rescale = [&](float before) {
      sl.m = top;
      sum.scale(sl.weight(before));
    };
    constexpr int AHEAD = 4;  // loads under way a thread
#pragma unroll 1
    for (int v = threadIdx.x; v < sl.nv; v += AHEAD * THREADS) {
      uint4 bits[AHEAD];
      bool in[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int u = v + i * THREADS;
        in[i] = u < sl.nv && sl.inside(u);
        if (in[i]) bits[i] = sl.whole(u);
      }
      if (!need_mass) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (in[i]) packed.take(bits[i]);
      } else {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (!in[i]) continue;
          VectorMax<T> peak;
          peak.take(bits[i]);
          const float before = top;
          top = max_nan(top, peak.get());
          if (top != before) rescale(before);
          if (top == -INFINITY) continue;
          float x[VEC];
          sl.unpack(bits[i], x);
          sum.add(top < INFINITY && sl.inv2 < INFINITY ? sl.finite_weights(x) : sl.weights(x));
        }
        sum.turn(v, AHEAD * THREADS);
      }
    }
    own = top = max_nan(top, packed.get());
    // The row's ends, an element a thread; whose vectors they are in will find them in shared memory.
    if (threadIdx.x < 2 * VEC) {
      const int which = threadIdx.x / VEC, v = which ? sl.nv - 1 : 0;
      float x = -INFINITY;
      if (sl.nv > 0 && !sl.inside(v) && (which == 0 ? sl.element(v) < 0 : sl.element(v) >= 0)) {
        const int i = sl.element(v) + threadIdx.x % VEC;
        if (i >= 0 && i < sl.n && sl.is_allowed(i)) x = lm_float(sl.row[i]);
        const float before = top;
        top = max_nan(top, x);
        if (need_mass && top > -INFINITY) {
          rescale(before);
          sum.add(sl.weight(x));
        }
      }
      reinterpret_cast<T*>(s.edge)[threadIdx.x] = lm_cast<T>(x);
    }
    mass = sum.get();
  }
  const float ref = top;
  float all_top = -INFINITY;  // the row's maximum, where it is known before step 3
  float widest = warp_max_nan(top);
  if (lane == 0) s.redf[warp] = widest;
  __syncthreads();
  widest = warp_max_nan(s.redf[lane & (WARPS - 1)]);
  sl.m = widest;
  cluster.barrier_wait(std::move(started));
  u64 Z = 0;
  if (need_mass) {
    // (A thread without a logit has no mass; nor has a slice, and its maximum is -inf.)
    mass = warp_sum(mass > 0.f ? mass * sl.weight(ref) : 0.f);
    if (lane == 0) s.mass[warp] = mass;
    // The sample: one vector in 2^sample_shift.  (What lies beyond the bins weighs
    // nothing.  64 x 131072, p = 0.9: 47 us; 52 with half as many elements, 48 with twice.)
#pragma unroll 1
    for (int q = threadIdx.x; q < sl.nv >> sl.sample_shift; q += THREADS) {
      float x[VEC];
      sl.load(q << sl.sample_shift, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float at = -SAMPLE_SCALE * sl.x(x[j]);
        if (at < SAMPLE_BINS) atomicAdd(&s.own_sample[static_cast<int>(at)], 1u);
      }
    }
    __syncthreads();
    mass = s.mass[lane & (WARPS - 1)];
#pragma unroll
    for (int d = WARPS / 2; d; d >>= 1) mass += __shfl_xor_sync(FULL_MASK, mass, d);
#pragma unroll 1
    for (int i = threadIdx.x; i < SAMPLE_BINS * C; i += THREADS)
      cluster.map_shared_rank(&s, i / SAMPLE_BINS)->sample[rank][i % SAMPLE_BINS] = s.own_sample[i % SAMPLE_BINS];
    if (threadIdx.x < C) cluster.map_shared_rank(&s, threadIdx.x)->part[rank] = Part{widest, mass};
    cluster.sync();
    float m = s.part[0].top;
#pragma unroll 1
    for (int i = 1; i < C; ++i) m = max_nan(m, s.part[i].top);
    all_top = m;
    if (m > -INFINITY) {
      sl.m = m;
#pragma unroll 1
      for (int i = 0; i < C; ++i) Z += sl.fixed(s.part[i].mass * sl.weight(s.part[i].top));
      sample_point(sl, s, (1.f - fmaxf(p, 0.f)) * (static_cast<float>(Z) * sl.unit));
      if (want) {
        // How many keys should reach the mass: three standard deviations of a
        // count of one in 2^sample_shift more, and a few.  Worth a try where one
        // of them more does not pass the limit.  (With the limit at the count
        // itself rows are tried that then need step 4: 256 x 131072, p = 0.9, T = 0.7, took
        // 74 us in the median of 24 inputs, against 61; at three of them 59, but too few
        // are tried at T = 1: 64 rows took 54 us, against 53.)
        const float tokens = s.likely[2], deviation = lm_sqrt(static_cast<float>(1 << sl.sample_shift) * (tokens + 16.f));
        const float limit = alone ? TOP : TOP_SHARED;
        // (With min-p the tokens may end long before the mass.)
        want = tokens + deviation > limit ? (min_p > 0.f ? TOP_MIN_P : 0)
                                          : static_cast<int>(fminf(32.f + tokens + 3.f * deviation, limit));
      }
    } else {
      want = 0;  // a NaN, or nothing to choose
    }
  }
  if (sl.nv > 0) {
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int v = which ? sl.nv - 1 : 0;
      if (sl.inside(v) || static_cast<int>(threadIdx.x) != v % THREADS) continue;
      float x[VEC];
      sl.load(v, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) own = fmaxf(own, x[j]);
    }
  }
  // A value that as many keys reach as step 2 sorts, or as top-k keeps.
  const int reach = want ? want : by_k && k <= THREADS ? k : 0;
  const bool flat = sl.nv < THREADS;
  float tau = reach == 1 ? widest : -INFINITY;
  if (reach > 1 && !isnan(widest)) {
    if (flat) {
      // Fewer vectors than threads: the threads' maxima of single elements instead.
      own = -INFINITY;
#pragma unroll 1
      for (int i = threadIdx.x; i < sl.nv * VEC; i += THREADS) {
        const int at = sl.element(0) + i;
        if (at >= 0 && at < sl.n && sl.is_allowed(at)) own = fmaxf(own, lm_float(sl.row[at]));
      }
    }
    tau = block_tau(own, widest, reach, s);
  }

  // 2. The slice's first keys.
  int keys = 0;
  if (want && !isnan(widest)) {
    // The threads whose maximum reaches tau; their vectors are shared out over all.
    if (!flat && own >= fmaxf(tau, -FLT_MAX)) s.hit[atomicAdd(&s.hits, 1u)] = static_cast<unsigned short>(threadIdx.x);
    __syncthreads();
    const int per_thread = (sl.nv + THREADS - 1) / THREADS, shift = per_thread > 1 ? 32 - __clz(per_thread - 1) : 0;
#pragma unroll 1
    for (int turn = 0;; ++turn) {
      const float least = fmaxf(tau, -FLT_MAX);
      const int vectors = flat ? sl.nv : static_cast<int>(s.hits) << shift;
#pragma unroll 1
      for (int base = threadIdx.x - lane; base < vectors; base += THREADS) {
        // Too many already: the count alone says so.  (Other warps add to it: one
        // lane reads, so that the warp leaves as a whole.)
        const unsigned so_far = lane == 0 ? *reinterpret_cast<volatile unsigned*>(&s.slot) : 0u;
        if (__shfl_sync(FULL_MASK, so_far, 0) > CANDIDATES) break;
        const int i = base + lane, v = i >= vectors ? sl.nv : flat ? i : s.hit[i >> shift] + (i & ((1 << shift) - 1)) * THREADS;
        unsigned some = 0;
        if (v < sl.nv) {
          float x[VEC];
          sl.load(v, x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) some |= x[j] >= least ? 1u << j : 0u;
        }
        if (__any_sync(FULL_MASK, some != 0u)) {
          unsigned at = warp_reserve(&s.slot, __popc(some));
#pragma unroll 1
          for (; some; some &= some - 1, ++at)
            if (at < CANDIDATES) s.candidates[at] = sl.key(sl.one(v, __ffs(some) - 1), sl.element(v) + __ffs(some) - 1);
        }
        __syncwarp();
      }
      __syncthreads();
      keys = static_cast<int>(s.slot);
      if (keys <= CANDIDATES || turn == 2) break;
      // Too many (neighbours are alike, so that a thread holds several): again
      // from a higher limit, if there is one.
      if (threadIdx.x == 0) *reinterpret_cast<S*>(s.slice) = sl;
      __syncthreads();
      const float higher = higher_limit<S>(s, least, flat, shift, want);
      if (!(higher > least)) break;
      tau = higher;
      if (threadIdx.x == 0) s.slot = 0;
      __syncthreads();
    }
    if (threadIdx.x == 0 && keys <= CANDIDATES) s.candidates[keys] = 0;
    __syncthreads();
  }
  if (keys > CANDIDATES) {  // copies of one value
    keys = -1;
  } else if (keys > 0) {
    // The first `want`, with their noise: to the row's list, or to the cluster's first CTA.
    Shared* leader = cluster.map_shared_rank(&s, 0);
    u64* to = alone ? s.sorted : leader->tops[rank];
    float* to_q = alone ? s.sorted_q : leader->tops_q[rank];
    rank_candidates(
        s, keys, [&](bool some, int, u64 key) { return some && !greedy ? noise[sl.index_of(key)] : 1.f; },
        [&](u64 key, int place, float q) {
          if (place < want) {
            to[place] = key;
            to_q[place] = q;
          }
        });
    keys = keys < want ? keys : want;
  }

  // 3. The row's maximum and first keys (nothing to tell where step 2 was left out
  // and the maximum is known).
  int found = 0;  // keys of all CTAs, or -1
  if (want || !need_mass) {
    if (threadIdx.x < C) cluster.map_shared_rank(&s, threadIdx.x)->sent[rank] = Sent{widest, tau, keys};
    cluster.sync();
    top = s.sent[0].top;
    tau = s.sent[0].tau;
    found = s.sent[0].keys;
#pragma unroll 1
    for (int i = 1; i < C; ++i) {
      top = max_nan(top, s.sent[i].top);
      tau = fmaxf(tau, s.sent[i].tau);
      found = found < 0 || s.sent[i].keys < 0 ? -1 : found + s.sent[i].keys;
    }
  } else {
    top = all_top;
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
  const float floor_w = fminf(min_p, 1.f);
  if (want && found >= 0) {
    const bool decide = !by_k && !greedy;  // whether these keys are enough is not known beforehand
    if (rank == 0) {
      const int got = found < want ? found : want;
      if (!alone) merge_keys(s, C, want);
      if (warp == 0) {
        const bool enough = race_list(sl, s, got, !decide || found < want, by_k, by_p, p, Z, floor_w, greedy,
                                      a.out_tokens + r, a.out_logprobs + r);
        if (decide && lane < C) cluster.map_shared_rank(&s, lane)->enough = enough;
      }
    }
    if (!decide) return;
    cluster.sync();  // the first CTA has written `enough`
    if (s.enough) return;
  }
  if (threadIdx.x == 0) {
    *reinterpret_cast<S*>(s.slice) = sl;
    s.late = Late{noise, a.out_tokens + r, a.out_logprobs + r, Z, k, p, temperature, floor_w, tau, by_k, by_p};
  }
  __syncthreads();
  late_row<S>(s);
}

template <typename T>
__global__ void __launch_bounds__(THREADS, 2) k_sample_tokens(TokenArgs a, int per_cta, bool long_lists) {
  __shared__ Shared s;
  extern __shared__ int long_list[];
  const int log_c = __ffs(cg::this_cluster().num_blocks()) - 1;
  if (threadIdx.x == 0) {  // (read after many barriers)
    s.list_to = long_lists ? long_list : s.list_at;
    s.room = long_lists ? LISTED_ALONE : LISTED;
  }
  pdl_wait();
  pdl_trigger();
  sample_row<T>(a, blockIdx.x >> log_c, per_cta, s);
}

// CTAs of a row's cluster: as many as the SMs have room for at once (two an SM),
// while each still has a slice of some size.  (64 x 131072 bfloat16 without filters
// and with p = 0.9: 15.6 and 47 us with four CTAs, 18 and 60 with two, 27 and 92 with
// one, 21 and 62 with eight, whose CTAs do not all fit.  304 x 65536, p = 0.9: 72 us
// with one and 79 with two, at T = 0.7 40 and 49.)
int cluster_of(int64_t rows, int64_t bytes) {
  int c = 1;
  while (c < MAX_CLUSTER && rows * c * 2 <= 2 * sms() && bytes / (2 * c) >= SLICE_LEAST) c *= 2;
  return c;
}

template <typename T>
cudaError_t launch_typed(const TokenArgs& a, cudaStream_t stream) {
  constexpr int VEC = 16 / int(sizeof(T));
  const int64_t vectors = (a.n + 2 * VEC - 2) / VEC;  // at any alignment of the row
  const int c = cluster_of(a.rows, vectors * 16);
  // One CTA for a row whose slice would be worth several.
  const bool long_lists = c == 1 && vectors * 16 > 2 * SLICE_LEAST;
  size_t dynamic = 0;
  if (long_lists) {
    dynamic = LISTED_ALONE * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(k_sample_tokens<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(dynamic));
    if (e != cudaSuccess) return e;
  }
  return launch_clusters(k_sample_tokens<T>, a.rows * c, THREADS, c, dynamic, stream, a,
                         static_cast<int>((vectors + c - 1) / c), long_lists);
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
