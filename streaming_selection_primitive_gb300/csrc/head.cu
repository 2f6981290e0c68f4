// Log-probabilities of given tokens from hidden states and the output matrix: a product
// whose result, the logits, is turned into row maxima and sums tile by tile and never
// leaves the chip.
#include "../../include/profk.h"
#include "lm.h"
#include "logprobs.cuh"

namespace profk {
namespace {

constexpr int TILE = 64;        // rows and tokens of a tile
constexpr int DEPTH = 32;       // of the product at a time
constexpr int THREADS = 256;

template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(THREADS) k_head(HeadArgs a, float4* parts, float* logits) {
  pdl_wait();
  __shared__ float h[DEPTH][TILE + 1], w[DEPTH][TILE + 1], l[TILE][TILE + 1];
  const int64_t row0 = int64_t(blockIdx.y) * TILE, col0 = int64_t(blockIdx.x) * TILE;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < a.width; k0 += DEPTH) {
    __syncthreads();
    for (int i = threadIdx.x; i < TILE * DEPTH; i += THREADS) {
      const int k = i % DEPTH, r = i / DEPTH;
      const bool in = k0 + k < a.width;
      h[k][r] = in && row0 + r < a.rows ? lm_float(static_cast<const T*>(a.hidden)[(row0 + r) * a.hidden_ld + k0 + k]) : 0.f;
      w[k][r] = in && col0 + r < a.n ? lm_float(static_cast<const T*>(a.weight)[(col0 + r) * a.weight_ld + k0 + k]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < DEPTH; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(h[k][ty + 16 * i], w[k][tx + 16 * j], acc[i][j]);
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) l[ty + 16 * i][tx + 16 * j] = acc[i][j];
  __syncthreads();
  const int64_t row = row0 + threadIdx.x;
  if (threadIdx.x < TILE && row < a.rows) {
    const float c = inverse_temperature(a.temperature ? a.temperature[row] : a.all_temperature);
    const int64_t token = a.tokens[row];
    const int cols = static_cast<int>(min(int64_t(TILE), a.n - col0));
    float m = -INFINITY, s = 0.f, t = 0.f;
    for (int j = 0; j < cols; ++j) m = fmaxf(m, l[threadIdx.x][j]);
    for (int j = 0; j < cols; ++j) {
      const float x = (l[threadIdx.x][j] - reference(m)) * c, e = lm_exp2(x);
      s += e;
      t = fmaf(fmaxf(x, NO_MASS), e, t);
    }
    parts[int64_t(blockIdx.x) * a.rows + row] = make_float4(m, s, t, 0.f);
    if (token >= col0 && token < col0 + cols) logits[row] = l[threadIdx.x][token - col0];
  }
}

constexpr int JOIN_ROWS = 32, JOIN_WARPS = 16;

// A row's parts joined: a lane has a row, a warp every JOIN_WARPS-th part.
__global__ void __launch_bounds__(JOIN_ROWS * JOIN_WARPS) k_head_join(HeadArgs a, const float4* parts, const float* logits, int tiles) {
  pdl_wait();
  __shared__ RowSum sums[JOIN_WARPS][JOIN_ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = int64_t(blockIdx.x) * JOIN_ROWS + lane;
  const float temperature = row < a.rows ? (a.temperature ? a.temperature[row] : a.all_temperature) : 1.f;
  const float c = inverse_temperature(temperature);
  RowSum y{-INFINITY, 0.f, 0.f};
  if (row < a.rows)
    for (int i = warp; i < tiles; i += JOIN_WARPS) {
      const float4 z = parts[int64_t(i) * a.rows + row];
      y = joined(y, RowSum{z.x, z.y, z.z}, c);
    }
  sums[warp][lane] = y;
  __syncthreads();
  if (warp != 0 || row >= a.rows) return;
  for (int i = 1; i < JOIN_WARPS; ++i) y = joined(y, sums[i][lane], c);
  if (!(c > 0.f)) y.s = NAN;
  const int64_t token = a.tokens[row];
  const bool live = token >= 0;
  a.logprobs[row] = live ? row_logprob(y, token < a.n ? logits[row] : NAN, temperature) : 0.f;
  if (a.entropies) a.entropies[row] = live ? row_entropy(y) : 0.f;
}

}  // namespace

cudaError_t launch_head_logprobs(const HeadArgs& a, cudaStream_t stream) {
  cudaMemPool_t pool;
  cudaError_t err = library_pool(&pool);
  if (err != cudaSuccess) return err;
  const int tiles = static_cast<int>((a.n + TILE - 1) / TILE);
  const size_t part_bytes = size_t(tiles) * a.rows * sizeof(float4);
  char* work = nullptr;
  err = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&work), part_bytes + a.rows * 4, pool, stream);
  if (err != cudaSuccess) return err;
  float4* parts = reinterpret_cast<float4*>(work);
  float* logits = reinterpret_cast<float*>(work + part_bytes);
  const dim3 grid(tiles, static_cast<unsigned>((a.rows + TILE - 1) / TILE));
  err = a.type == PROFK_BF16 ? launch_kernel(k_head<__nv_bfloat16, true>, grid, dim3(THREADS), 0, stream, a, parts, logits)
                             : launch_kernel(k_head<__half, true>, grid, dim3(THREADS), 0, stream, a, parts, logits);
  if (err == cudaSuccess)
    err = launch_kernel(k_head_join, dim3(static_cast<unsigned>((a.rows + JOIN_ROWS - 1) / JOIN_ROWS)), dim3(JOIN_ROWS * JOIN_WARPS), 0, stream,
                        a, parts, logits, tiles);
  const cudaError_t freed = cudaFreeAsync(work, stream);
  return err != cudaSuccess ? err : freed;
}

}  // namespace profk
