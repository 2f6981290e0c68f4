// Choice of each token's experts, and its gradient.
//
// A token t has one logit z_e per expert.  With y = z (softmax scores) or
// y = log sigmoid(z) (sigmoid scores), p = softmax(y) over the experts.  The
// choice is the first k experts in the library order of z + bias (descending,
// ties by lower index, -inf and NaN never).  Gates: over the chosen,
// softmax(y) when normalized, else p (softmax) or sigmoid(z).  Balance loss:
//   loss = E sum_e (counts_e / N) P_e,  P_e = sum_t n_t p_te / N,
// counts_e the slots given to expert e, n_t those token t filled, N = sum n_t.
#include "lm.cuh"
#include "lm.h"
#include "../../include/profk.h"

namespace profk {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// log sigmoid(z), exact for large |z|.
__device__ __forceinline__ float log_sigmoid(float z) { return fminf(z, 0.f) - log1pf(expf(-fabsf(z))); }

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// The token's p, unnormalized, into s, and its sum (over the warp).  Softmax:
// s = exp(z - max).  Sigmoid: s = sigmoid(z) exp(-c), c = min(max z, 0), so
// that a token whose scores all underflow keeps their ratios.
template <int NPL>
__device__ __forceinline__ float token_scores(const float (&z)[NPL], float (&s)[NPL], int E, bool sig) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
#pragma unroll
  for (int r = 0; r < NPL; ++r)
    if (lane + 32 * r < E) m = fmaxf(m, z[r]);
  m = warp_max(m);
  const float c = fminf(m, 0.f), ec = expf(c);
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < NPL; ++r) {
    s[r] = 0.f;
    if (lane + 32 * r < E) {
      if (sig) {
        const bool pos = z[r] >= 0.f;
        const float u = z[r] == -INFINITY ? 0.f : expf(pos ? -z[r] : z[r] - c);
        s[r] = (pos ? 1.f : u) / (1.f + (pos ? u : u * ec));
      } else {
        s[r] = z[r] == m ? 1.f : expf(z[r] - m);
      }
      sum += s[r];
    }
  }
  return warp_sum(sum);
}

// The gate of lane j's chosen expert (logit zc; ok: the slot is filled), given
// the token's softmax maximum and sum for the form that needs them.
__device__ __forceinline__ float slot_gate(float zc, bool ok, bool sig, bool normalize, float p) {
  if (!normalize) return !ok ? 0.f : sig ? sigmoid(zc) : p;
  const float y = ok ? (sig ? log_sigmoid(zc) : zc) : -INFINITY;
  const float top = warp_max(y);
  const float e = ok ? (y == top ? 1.f : expf(y - top)) : 0.f;
  const float sum = warp_sum(e);
  return ok ? e / sum : 0.f;
}

// One warp per token; the lane holds the logits of experts lane, lane + 32,
// ...  Per CTA: the counts in shared memory (integers), the probabilities in
// registers, joined warp by warp in a fixed order and written to `part`.
template <typename T, int NPL>
__global__ void __launch_bounds__(THREADS) k_route(RouteArgs a, float* part_p, unsigned* part_c) {
  extern __shared__ unsigned char smem[];
  unsigned* cnt = reinterpret_cast<unsigned*>(smem);  // E
  float* sp = reinterpret_cast<float*>(cnt + a.experts);  // WARPS x E
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
  for (int e = threadIdx.x; e < E; e += THREADS) cnt[e] = 0u;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  float acc[NPL];
#pragma unroll
  for (int r = 0; r < NPL; ++r) acc[r] = 0.f;
  const T* logits = static_cast<const T*>(a.logits);
  for (int64_t t = int64_t(blockIdx.x) * WARPS + warp; t < a.tokens; t += int64_t(gridDim.x) * WARPS) {
    const T* row = logits + t * a.ld;
    int mine = -1;  // lane j: the expert of slot j
    int filled = 0;
    float gate = 0.f;
    if (!a.mask || a.mask[t]) {
      float z[NPL], s[NPL];
      uint32_t key[NPL];
#pragma unroll
      for (int r = 0; r < NPL; ++r) {
        const int e = lane + 32 * r;
        z[r] = e < E ? lm_float(row[e]) : -INFINITY;
        key[r] = e < E ? choice_key(a.bias ? z[r] + a.bias[e] : z[r]) : 0u;
      }
      for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int r = 0; r < NPL; ++r)
          if (key[r] > best) {
            best = key[r];
            at = r;
          }
        const uint32_t top = __reduce_max_sync(FULL_MASK, best);
        if (top == 0u) break;
        const unsigned e = __reduce_min_sync(FULL_MASK, best == top ? unsigned(lane + 32 * at) : 0xFFFFFFFFu);
#pragma unroll
        for (int r = 0; r < NPL; ++r)
          if (lane + 32 * r == int(e)) key[r] = 0u;
        if (lane == j) mine = int(e);
        ++filled;
      }
      const bool ok = mine >= 0;
      const float zc = ok ? lm_float(row[mine]) : -INFINITY;
      float sum = 0.f, m = 0.f;
      if (a.loss || (!a.normalize && !a.sigmoid)) {
        sum = token_scores<NPL>(z, s, E, a.sigmoid);
        if (filled) {
          const float scale = float(filled) / sum;
#pragma unroll
          for (int r = 0; r < NPL; ++r) acc[r] += s[r] * scale;
        }
        m = -INFINITY;
#pragma unroll
        for (int r = 0; r < NPL; ++r) m = fmaxf(m, z[r]);
        m = warp_max(m);
      }
      gate = slot_gate(zc, ok, a.sigmoid, a.normalize, (zc == m ? 1.f : expf(zc - m)) / sum);
      bool nan = false;
#pragma unroll
      for (int r = 0; r < NPL; ++r) nan |= isnan(z[r]);
      if (__any_sync(FULL_MASK, nan) && ok) gate = __int_as_float(0x7fc00000);
      if (ok) atomicAdd(cnt + mine, 1u);
    }
    if (lane < a.k) {
      a.gates[t * a.k + lane] = gate;
      a.chosen[t * a.k + lane] = mine;
    }
  }
#pragma unroll
  for (int r = 0; r < NPL; ++r)
    if (lane + 32 * r < E) sp[warp * E + lane + 32 * r] = acc[r];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += sp[w * E + e];
    part_p[int64_t(blockIdx.x) * E + e] = sum;
    part_c[int64_t(blockIdx.x) * E + e] = cnt[e];
  }
}

// Joins the CTAs' counts and probabilities in CTA order; one CTA.
__global__ void __launch_bounds__(1024) k_route_join(int parts, int E, const float* part_p, const unsigned* part_c,
                                                     int64_t* counts, float* loss) {
  __shared__ float sf[32];
  __shared__ unsigned long long sn[32];
  __shared__ unsigned long long total;
  pdl_wait();
  pdl_trigger();
  const int e = threadIdx.x, lane = e & 31, warp = e >> 5;
  unsigned long long c = 0;
  float p = 0.f;
  if (e < E)
    for (int i = 0; i < parts; ++i) {
      c += part_c[int64_t(i) * E + e];
      p += part_p[int64_t(i) * E + e];
    }
  if (e < E) counts[e] = static_cast<int64_t>(c);
  if (!loss) return;
  unsigned long long n = c;
#pragma unroll
  for (int d = 16; d; d >>= 1) n += __shfl_xor_sync(FULL_MASK, n, d);
  if (lane == 0) sn[warp] = n;
  __syncthreads();
  if (e == 0) {
    n = 0;
    for (int w = 0; w < 32; ++w) n += sn[w];
    total = n;
  }
  __syncthreads();
  const float N = total ? static_cast<float>(total) : 1.f;
  const float v = warp_sum((static_cast<float>(c) / N) * (p / N));
  if (lane == 0) sf[warp] = v;
  __syncthreads();
  if (e == 0) {
    float sum = 0.f;
    for (int w = 0; w < 32; ++w) sum += sf[w];
    *loss = static_cast<float>(E) * sum;
  }
}

// Gradient of the gates and of the balance loss, one warp per token; the
// choice and the counts are constants.  dy as in the header's formulas, then
// dz = dy (softmax) or dy sigmoid(-z).
template <typename T, int NPL>
__global__ void __launch_bounds__(THREADS) k_route_backward(RouteBackwardArgs a) {
  extern __shared__ unsigned char smem[];
  __shared__ unsigned long long total;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.experts;
  float* extra = reinterpret_cast<float*>(smem) + warp * E;  // the chosen experts' part of dy
  if (threadIdx.x == 0) total = 0;
  for (int e = lane; e < E; e += 32) extra[e] = 0.f;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  float share[NPL];  // dL E counts_e / N^2
#pragma unroll
  for (int r = 0; r < NPL; ++r) share[r] = 0.f;
  if (a.grad_loss) {
    unsigned long long n = 0;
    for (int e = threadIdx.x; e < E; e += THREADS) n += static_cast<unsigned long long>(a.counts[e]);
    if (n) atomicAdd(&total, n);
    __syncthreads();
    const float N = total ? static_cast<float>(total) : 1.f;
    const float f = *a.grad_loss * static_cast<float>(E) / N;
#pragma unroll
    for (int r = 0; r < NPL; ++r)
      if (lane + 32 * r < E) share[r] = f * (static_cast<float>(a.counts[lane + 32 * r]) / N);
  }
  const T* logits = static_cast<const T*>(a.logits);
  T* grad = static_cast<T*>(a.grad_logits);
  for (int64_t t = int64_t(blockIdx.x) * WARPS + warp; t < a.tokens; t += int64_t(gridDim.x) * WARPS) {
    const T* row = logits + t * a.ld;
    T* out = grad + t * a.grad_ld;
    int64_t mine = lane < a.k ? a.chosen[t * a.k + lane] : -1;
    const bool ok = mine >= 0 && mine < E;
    const int filled = __popc(__ballot_sync(FULL_MASK, ok));
    if (!filled) {  // masked, or nothing to choose: no gradient
      for (int e = lane; e < E; e += 32) out[e] = lm_cast<T>(0.f);
      continue;
    }
    float z[NPL], s[NPL];
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < NPL; ++r) {
      const int e = lane + 32 * r;
      z[r] = e < E ? lm_float(row[e]) : -INFINITY;
      m = fmaxf(m, z[r]);
    }
    m = warp_max(m);
    const float inv = 1.f / token_scores<NPL>(z, s, E, a.sigmoid);
    float dot = 0.f;
#pragma unroll
    for (int r = 0; r < NPL; ++r) {
      s[r] *= inv;  // p
      dot += s[r] * share[r];
    }
    dot = warp_sum(dot) * filled;
    if (a.grad_gates) {
      const float zc = ok ? lm_float(row[mine]) : -INFINITY;
      const float g = slot_gate(zc, ok, a.sigmoid, a.normalize, (zc == m ? 1.f : expf(zc - m)) * inv);
      const float dg = ok ? a.grad_gates[t * a.k + lane] : 0.f;
      const float gd = warp_sum(g * dg);
      float d = g * dg;
      if (a.normalize)
        d = g * (dg - gd);
      else if (!a.sigmoid)
        dot += gd;
      if (ok) extra[mine] = d;
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < NPL; ++r) {
      const int e = lane + 32 * r;
      if (e < E) {
        float dy = s[r] * (share[r] * filled - dot) + extra[e];
        if (a.sigmoid) dy *= sigmoid(-z[r]);
        out[e] = lm_cast<T>(dy);
      }
    }
    __syncwarp();
    if (ok) extra[mine] = 0.f;
    __syncwarp();
  }
}

template <typename F>
cudaError_t by_type(int type, F&& f) {
  switch (type) {
    case PROFK_F32: return f(float{});
    case PROFK_BF16: return f(__nv_bfloat16{});
    default: return f(__half{});
  }
}

// The smallest NPL with 32 NPL >= E.
template <typename F>
cudaError_t by_width(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 1>{});
  if (E <= 64) return f(std::integral_constant<int, 2>{});
  if (E <= 128) return f(std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

int route_grid(int64_t tokens) {
  const int64_t need = (tokens + WARPS - 1) / WARPS;
  const int64_t most = 2 * static_cast<int64_t>(sms());
  return static_cast<int>(need < most ? need : most);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  const int grid = route_grid(a.tokens);
  if (grid == 0)  // no tokens: zero counts and loss
    return launch_kernel(k_route_join, dim3(1), dim3(1024), 0, stream, 0, a.experts, static_cast<const float*>(nullptr),
                         static_cast<const unsigned*>(nullptr), a.counts, a.loss);
  cudaMemPool_t pool;
  cudaError_t err = library_pool(&pool);
  if (err != cudaSuccess) return err;
  void* part = nullptr;
  const size_t each = size_t(grid) * a.experts * 4;
  err = cudaMallocFromPoolAsync(&part, 2 * each, pool, stream);
  if (err != cudaSuccess) return err;
  float* part_p = static_cast<float*>(part);
  unsigned* part_c = reinterpret_cast<unsigned*>(static_cast<char*>(part) + each);
  err = by_type(a.type, [&](auto t) {
    return by_width(a.experts, [&](auto w) {
      const size_t smem = size_t(1 + WARPS) * a.experts * 4;
      return launch_kernel(k_route<decltype(t), decltype(w)::value>, dim3(grid), dim3(THREADS), smem, stream, a, part_p,
                           part_c);
    });
  });
  if (err == cudaSuccess)
    err = launch_kernel(k_route_join, dim3(1), dim3(1024), 0, stream, grid, a.experts, part_p, part_c, a.counts, a.loss);
  const cudaError_t freed = cudaFreeAsync(part, stream);
  return err != cudaSuccess ? err : freed;
}

cudaError_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t stream) {
  return by_type(a.type, [&](auto t) {
    return by_width(a.experts, [&](auto w) {
      return launch_kernel(k_route_backward<decltype(t), decltype(w)::value>, dim3(route_grid(a.tokens)), dim3(THREADS),
                           size_t(WARPS) * a.experts * 4, stream, a);
    });
  });
}

}  // namespace profk
