// Log-probabilities of given tokens from hidden states and the output matrix: a product
// on the tensor cores whose result, the logits, is turned into row maxima and sums tile
// by tile and never leaves the chip.
//
// A tile is 128 rows of hidden states by 256 tokens of the vocabulary.  A CTA (one an SM)
// has a warp that copies pieces of both, 64 deep, into a ring in shared memory, a warp
// that issues the products into one half of the tensor memory, and eight warps that
// meanwhile take the finished tile in the other half: a thread has half of a row's
// tokens, and carries the row's running maximum and sums over a run of tiles.  The runs'
// sums are joined by a second kernel.
//
// What bounds it: 4096 x 2048 x 131072 bfloat16 takes 1161 us (1.89 PFLOP/s, what the library's product
// reaches in a short run) to 1310 in a long one (1.68, under the power limit); its logits alone
// would be 2.1 GB to write and to read.  Of 5 rows it takes 172 us for 1.07 GB of matrix (6.2 TB/s; 215 while
// 128 rows were copied for the 5), and 18.6 for 67 MB: launch, first piece, last tile and join are half of it.
// 777 x 1000 x 50001 float16 takes 98 us, 0.41 of the tensor cores' time: a row of 2000 bytes has its 128 bytes
// of a piece in two lines of L2, and the copies of 384 such rows take a CTA 1.5 times the 512 cycles
// of their products (width 1024: 68 us).  Not adopted: tiles of 128 to 224 tokens (the same or slower everywhere),
// CTAs in pairs that share the products' second operand (2.4 times slower as written: the second
// one's copies were announced to the first by a warp, one exchange more a piece) or copy half
// of it for both (777 x 1000 x 50001 86 us, 300 x 1024 x 20000 30 instead of 23).
//
// Rows that are left out are copied and multiplied like others (4096 x 2048 x 131072 takes the same with half of
// them left out, by themselves the other half would take 657 us): give only the rows that count where many do not.
//
// Every wait is bounded; a CTA whose wait ends without its barrier writes NaN for all rows of
// its remaining work, and leaves when its copies and products are done.
#include <cuda.h>

#include <algorithm>

#include "../../include/profk.h"
#include "lm.h"
#include "logprobs.cuh"
#include "ring.h"
#include "tcgen05.cuh"

namespace profk {
namespace {

constexpr int TILE_ROWS = 128;
constexpr int TILE_TOKENS = 256;
constexpr int DEPTH = 64;   // of a piece: 128 bytes a row, the widest swizzle
constexpr int MAX_STAGES = 5;  // pieces in the ring: of 128 rows 4
constexpr int TAKERS = 8;   // warps that take tiles: two for each quarter of the lanes
constexpr int COPIER = TAKERS, MULTIPLIER = TAKERS + 1;  // the other two warps
constexpr int THREADS = 32 * (TAKERS + 4);  // (two warps have nothing to do: registers are handed over by groups of four)
// Registers a thread where a tile has segments: of 168 at the launch the takers, who hold 128 sums each,
// get more from the others.  (256 * 232 + 128 * 40 = 384 * 168.)  It is not enough for 32 columns just loaded beside the
// sums and the row's state: 312 bytes a thread are spilled (with entropies 324), with 224 registers 376.
constexpr int TAKER_REGISTERS = 232, OTHER_REGISTERS = 40;
constexpr int TENSOR_COLUMNS = 2 * TILE_TOKENS;  // all there are: two accumulators
// Pieces whose products the tensor cores add up at a temperature of 1 or more (segment_pieces).  They cut their sums
// off instead of rounding them, and what that takes away grows with the depth: 3453 deep it put log-probabilities off
// by 1.6e-6 of themselves, in two segments by 7e-7 (a float32 product: 5e-7).  The takers add the segments, which costs
// 4096 x 4096 x 32768 640 us instead of 604; with segments of half as much 2048 x 131072 would take 1285 instead of 1161.
constexpr int SEGMENT = 32, LEAST_SEGMENT = 8;
constexpr int PARTS = 2;    // a row's columns are taken by two threads, 32 by 32 in turn

constexpr int ROWS_BYTES = TILE_ROWS * DEPTH * 2;
constexpr int RING_BYTES = 4 * (ROWS_BYTES + TILE_TOKENS * DEPTH * 2);
// The ring begins at a multiple of 1024 bytes.  16 KB more than that are never touched: a launch with 213 KB takes
// 777 x 1000 x 50001 97.2 us, with 197 KB 100.6.
constexpr int SHARED_BYTES = RING_BYTES + ROWS_BYTES + 1024;
// A product takes its first operand from a whole tile of rows, whatever has been copied: it stays within its stage.
static_assert(8 * DEPTH * 2 + TILE_TOKENS * DEPTH * 2 >= ROWS_BYTES);

// How the work is cut: run r is row tile r % row_tiles and the vocabulary's tiles
// (r / row_tiles) * run and on, `run` of them, so that CTAs that work at the same time share
// their tiles of the matrix in L2.
struct Plan {
  int rows;   // rows of hidden states that are copied for a tile: a multiple of 8
  int row_tiles, token_tiles, run, runs, pieces, stages;
  int segments;  // of a tile
  // A stage: the rows, then the tokens.  Of fewer rows than a tile has the product takes what comes
  // behind them for the others (whose results nobody looks at).
  __host__ __device__ int rows_bytes() const { return rows * DEPTH * 2; }
  __host__ __device__ int stage_bytes() const { return rows_bytes() + TILE_TOKENS * DEPTH * 2; }
};

struct Barriers {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];  // of the ring
  uint64_t done[2], taken[2];            // of the accumulators
  uint32_t tensor;                       // address of the tensor memory
  int given_up;
};

// The pieces of a tile up to the end of a segment (whose lengths differ by one at most).
__device__ __forceinline__ int segment_end(const Plan& plan, int segment) { return plan.pieces * (segment + 1) / plan.segments; }

template <bool ENTROPY>
__device__ __forceinline__ void take_columns(RowSum& r, float (&v)[32], float c) {
  float m = r.m;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, v[i]);
  // (Not only where m has grown: 32 lanes with a row each are never of one mind, and the branch
  // cost 2048 x 64 x 131072 96 us instead of 88.)
  const float d = shrink(r.m, m, c), f = lm_exp2(d);
  if (ENTROPY) r.t = f * (r.t + d * r.s);
  r.s *= f;
  r.m = m;
  const Centre at(m, c);
  Pair s[2] = {0, 0}, t[2] = {0, 0};
  const Pair by = pair(at.by, at.by), cc = pair(c, c);
  const auto add = [&](Pair x, int i) {
    float x0, x1;
    split(x, x0, x1);
    const Pair e = pair(lm_exp2(x0), lm_exp2(x1));
    s[i & 1] = add2(s[i & 1], e);
    if (ENTROPY) t[i & 1] = fma2(pair(fmaxf(x0, NO_MASS), fmaxf(x1, NO_MASS)), e, t[i & 1]);
  };
  if (at.fused) {
#pragma unroll
    for (int i = 0; i < 16; ++i) add(fma2(pair(v[2 * i], v[2 * i + 1]), cc, by), i);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) add(mul2(add2(pair(v[2 * i], v[2 * i + 1]), by), cc), i);
  }
  float a, b;
  if (ENTROPY) {
    split(add2(t[0], t[1]), a, b);
    r.t += a + b;
  }
  split(add2(s[0], s[1]), a, b);
  r.s += a + b;
}

// SEGMENTS: a tile has more than one.
template <bool ENTROPY, bool SEGMENTS>
__global__ void __launch_bounds__(THREADS, 1)
    k_head(const __grid_constant__ CUtensorMap hidden, const __grid_constant__ CUtensorMap weight, HeadArgs a, Plan plan, uint32_t product,
           float4* parts, int count, float* logits, WaitCfg waits) {
  extern __shared__ uint8_t raw[];
  __shared__ Barriers sync;
  uint8_t* ring = raw + (1024 - shared_address(raw) % 1024) % 1024;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int limit = wait_limit(waits), stages = plan.stages, stage_bytes = plan.stage_bytes(), rows_bytes = plan.rows_bytes();
  if (threadIdx.x == 0) {
    for (int i = 0; i < plan.stages; ++i) {
      barrier_init(&sync.full[i], 1);
      barrier_init(&sync.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      barrier_init(&sync.done[i], 1 + waits.skew);
      barrier_init(&sync.taken[i], TAKERS);
    }
    barrier_init_done();
    sync.given_up = 0;
  }
  if (warp == MULTIPLIER) tensor_alloc<TENSOR_COLUMNS>(&sync.tensor);
  before_barrier();
  __syncthreads();
  after_barrier();
  const uint32_t tensor = sync.tensor;
  pdl_wait();
  pdl_trigger();  // (behind it: what follows may read what this reads)

  if (warp >= TAKERS) {
    if constexpr (SEGMENTS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(OTHER_REGISTERS));
    if (warp == COPIER) {
      if (lane == 0) {
        RingPlace at;
        int issued = 0;  // copies that may still be on their way: the last one to each stage
        for (int run = blockIdx.x; run < plan.runs && !sync.given_up; run += gridDim.x) {
          const int row0 = run % plan.row_tiles * TILE_ROWS, first = run / plan.row_tiles * plan.run;
          const int last = min(first + plan.run, plan.token_tiles);
          bool ok = true;
          for (int tile = first; tile < last && ok; ++tile)
            for (int piece = 0; piece < plan.pieces; ++piece) {
              ok = barrier_wait(&sync.empty[at.stage], at.empty(), &sync.given_up, limit);
              if (!ok) break;
              uint8_t* to = ring + at.stage * stage_bytes;
              barrier_arrive_expect(&sync.full[at.stage], stage_bytes);
              copy_tile(to, &hidden, piece * DEPTH, row0, &sync.full[at.stage]);
              copy_tile(to + rows_bytes, &weight, piece * DEPTH, tile * TILE_TOKENS, &sync.full[at.stage]);
              issued = min(issued + 1, stages);
              at.next(stages);
            }
        }
        // Whoever gives up sets the flag, which the waits for what is still being copied are not to look at.
        leave_ring(
            at, issued, stages, [&](RingPlace p) { return barrier_wait(&sync.empty[p.stage], p.empty(), &sync.given_up, limit); },
            [&](RingPlace p) {
              int nobody = 0;
              barrier_wait(&sync.full[p.stage], p.full(), &nobody, WAIT_POLLS);
            });
      }
    } else if (warp == MULTIPLIER) {
      if (lane == 0) {
        RingPlace at;
        int half = 0;
        unsigned taken = 1;  // (both accumulators begin free)
        bool ok = true;
        for (int run = blockIdx.x; run < plan.runs && ok; run += gridDim.x) {
          const int first = run / plan.row_tiles * plan.run, last = min(first + plan.run, plan.token_tiles);
          for (int tile = first; tile < last && ok; ++tile) {
            for (int segment = 0, piece = 0; segment < plan.segments && ok; ++segment) {
              const int end = SEGMENTS ? segment_end(plan, segment) : plan.pieces;
              ok = barrier_wait(&sync.taken[half], taken, &sync.given_up, limit);
              if (!ok) break;
              after_barrier();
              const uint32_t to = tensor + half * TILE_TOKENS;
              for (int first_piece = piece; piece < end; ++piece) {
                ok = barrier_wait(&sync.full[at.stage], at.full(), &sync.given_up, limit);
                if (!ok) break;
                after_barrier();
                const uint64_t x = tile_descriptor(ring + at.stage * stage_bytes), w = tile_descriptor(ring + at.stage * stage_bytes + rows_bytes);
#pragma unroll
                for (int k = 0; k < DEPTH / 16; ++k)  // 32 bytes on along the rows: 2 in the descriptor's units
                  multiply(to, x + 2 * k, w + 2 * k, product, piece - first_piece + k > 0);
                products_arrive(&sync.empty[at.stage]);
                at.next(stages);
              }
              if (!ok) break;
              products_arrive(&sync.done[half]);
              half ^= 1;
              if (half == 0) taken ^= 1;
            }
          }
        }
      }
    }
  } else {
    if constexpr (SEGMENTS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TAKER_REGISTERS));
    const int quarter = warp & 3, side = warp >> 2;
    int half = 0;
    unsigned done = 0;
    bool ok = true;
    for (int run = blockIdx.x; run < plan.runs; run += gridDim.x) {
      const int index = run / plan.row_tiles, first = index * plan.run, last = min(first + plan.run, plan.token_tiles);
      const int64_t row = int64_t(run % plan.row_tiles) * TILE_ROWS + quarter * 32 + lane;
      const bool in = row < a.rows;
      const float c = inverse_temperature(in && a.temperature ? a.temperature[row] : a.all_temperature);
      const int64_t token = in ? a.tokens[row] : -1;
      RowSum sum{-INFINITY, 0.f, 0.f, 0.f};
      for (int tile = first; tile < last && ok; ++tile) {
        const int64_t column0 = int64_t(tile) * TILE_TOKENS;
        const auto take = [&](float(&v)[32], int i) {
          const int64_t column = column0 + i;
          if (column + 32 > a.n) {  // behind the vocabulary
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (column + j >= a.n) v[j] = -INFINITY;
          }
          const int64_t at = token - column;
          if (__any_sync(FULL_MASK, at >= 0 && at < 32)) {
            float logit = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (at == j) logit = v[j];
            if (at >= 0 && at < 32 && token < a.n) logits[row] = logit;
          }
          take_columns<ENTROPY>(sum, v, c);
        };
        const uint32_t lanes = tensor + (uint32_t(quarter * 32) << 16) + side * 32;
        const auto wait_done = [&] {
          ok = __all_sync(FULL_MASK, barrier_wait(&sync.done[half], done, &sync.given_up, limit));
          after_barrier();
          return ok;
        };
        const auto have_taken = [&] {
          before_barrier();
          __syncwarp();
          if (lane == 0) barrier_arrive(&sync.taken[half]);
          half ^= 1;
          if (half == 0) done ^= 1;
        };
        constexpr int STEP = 32 * PARTS, MINE = TILE_TOKENS / STEP;  // this side's columns, 32 at a time
        if constexpr (SEGMENTS) {
          float v[MINE][32];
          for (int segment = 0; segment < plan.segments; ++segment) {
            if (!wait_done()) break;
#pragma unroll
            for (int i = 0; i < MINE; ++i) {
              float w[32];
              tensor_load(w, lanes + half * TILE_TOKENS + i * STEP);
              tensor_loaded();
#pragma unroll
              for (int j = 0; j < 32; ++j) v[i][j] = segment == 0 ? w[j] : v[i][j] + w[j];
            }
            have_taken();
          }
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < MINE; ++i) take(v[i], side * 32 + i * STEP);
        } else {
          if (!wait_done()) break;
#pragma unroll 1
          for (int i = 0; i < MINE; ++i) {
            float v[32];
            tensor_load(v, lanes + half * TILE_TOKENS + i * STEP);
            tensor_loaded();
            take(v, side * 32 + i * STEP);
          }
          have_taken();
        }
      }
      if (!ok) sum.s = NAN;
      if (in) parts[(row * count + index) * PARTS + side] = make_float4(sum.m, sum.s, sum.t, 0.f);
    }
  }
  // The products in flight are waited for, by a barrier that nothing else can make give up: where the takers' waits
  // run out, that may be behind the multiplier's last look at the flag.  (Otherwise they are done when the takers are.)
  if (warp == MULTIPLIER && lane == 0) {
    int nobody = 0;
    __shared__ uint64_t last;
    barrier_init(&last, 1);
    barrier_init_done();
    products_arrive(&last);
    barrier_wait(&last, 0, &nobody, WAIT_POLLS);
  }
  __syncwarp();
  before_barrier();
  __syncthreads();
  after_barrier();
  if (warp == MULTIPLIER) tensor_free<TENSOR_COLUMNS>(tensor);
}

constexpr int JOIN_THREADS = 128;

// A row's parts joined, by a warp.  (Parts of a row one behind the other: with those of a part, which the
// kernel before would write in one piece, and a row a lane, 5 x 1024 x 32768 took 22.2 us in all, not 18.5.)
__global__ void __launch_bounds__(JOIN_THREADS) k_head_join(HeadArgs a, const float4* parts, const float* logits, int count) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
  // (The kernel before lets this one start once all before it is done: what the user gave can be read.)
  const int64_t token = row < a.rows ? a.tokens[row] : -1;
  const float temperature = row < a.rows && a.temperature ? a.temperature[row] : a.all_temperature;
  const float c = inverse_temperature(temperature);
  pdl_wait();
  pdl_trigger();
  if (row >= a.rows) return;
  const bool live = token >= 0;
  const float logit = live && token < a.n ? logits[row] : NAN;
  RowSum y{-INFINITY, 0.f, 0.f, 0.f};
  if (live)
#pragma unroll 4
    for (int i = lane; i < count; i += 32) {
      const float4 z = parts[row * count + i];
      y = joined(y, RowSum{z.x, z.y, z.z, 0.f}, c);
    }
  y = centred(warp_join<true>(y, c), c);
  if (!(c > 0.f)) y.s = NAN;
  if (lane == 0) {
    a.logprobs[row] = live ? row_logprob(y, logit, temperature) : 0.f;
    if (a.entropies) a.entropies[row] = live ? row_entropy(y) : 0.f;
  }
}

// A matrix of `rows` rows as the copies see it: tiles of 64 values by `tile_rows`, zero outside.
bool describe(CUtensorMap* map, const void* p, bool bf16, int64_t rows, int64_t width, int64_t ld, int tile_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t size[2] = {cuuint64_t(width), cuuint64_t(rows)}, stride[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {DEPTH, cuuint32_t(tile_rows)}, step[2] = {1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(p), size, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a logit lacks counts 1 / T times in a log-probability (of rows with temperatures of their own: twice), and
// twice as much in an entropy: 1502 deep at 0.556, entropies were off by 2.1e-6 of themselves in one segment (a
// float32 product: 7.5e-7).
int segment_pieces(const HeadArgs& a) {
  const float part = (a.temperature ? 0.5f : std::min(a.all_temperature, 1.f)) * (a.entropies ? 0.5f : 1.f);
  return std::max(static_cast<int>(SEGMENT * part), LEAST_SEGMENT);
}

Plan plan_for(const HeadArgs& a) {
  Plan p;
  p.row_tiles = static_cast<int>((a.rows + TILE_ROWS - 1) / TILE_ROWS);
  p.rows = static_cast<int>(std::min<int64_t>(TILE_ROWS, (a.rows + 7) / 8 * 8));
  p.pieces = static_cast<int>((a.width + DEPTH - 1) / DEPTH);
  p.token_tiles = static_cast<int>((a.n + TILE_TOKENS - 1) / TILE_TOKENS);
  const int most = segment_pieces(a);
  p.segments = (p.pieces + most - 1) / most;
  p.stages = std::min(MAX_STAGES, RING_BYTES / p.stage_bytes());
  // Runs of up to 4 tiles, while there are 8 runs or more for each SM.
  const int64_t tiles = int64_t(p.row_tiles) * p.token_tiles;
  p.run = static_cast<int>(std::clamp<int64_t>(tiles / (8 * sms()), 1, 4));
  p.runs = p.row_tiles * ((p.token_tiles + p.run - 1) / p.run);
  return p;
}

}  // namespace

cudaError_t launch_head_logprobs(const HeadArgs& a, cudaStream_t stream) {
  const bool bf16 = a.type == PROFK_BF16;
  const Plan plan = plan_for(a);
  CUtensorMap hidden, weight;
  if (!describe(&hidden, a.hidden, bf16, a.rows, a.width, a.hidden_ld, plan.rows) ||
      !describe(&weight, a.weight, bf16, a.n, a.width, a.weight_ld, TILE_TOKENS))
    return cudaErrorInvalidValue;
  const int runs = (plan.token_tiles + plan.run - 1) / plan.run, count = runs * PARTS;
  cudaMemPool_t pool;
  cudaError_t err = library_pool(&pool);
  if (err != cudaSuccess) return err;
  const size_t part_bytes = size_t(count) * a.rows * sizeof(float4);
  char* work = nullptr;
  err = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&work), part_bytes + a.rows * sizeof(float), pool, stream);
  if (err != cudaSuccess) return err;
  float4* parts = reinterpret_cast<float4*>(work);
  float* logits = reinterpret_cast<float*>(work + part_bytes);
  const bool segments = plan.segments > 1;
  const auto kernel = a.entropies ? (segments ? k_head<true, true> : k_head<true, false>) : (segments ? k_head<false, true> : k_head<false, false>);
  const unsigned grid = std::min(plan.runs, sms());
  err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SHARED_BYTES);
  if (err == cudaSuccess)
    err = launch_kernel(kernel, dim3(grid), dim3(THREADS), size_t(SHARED_BYTES), stream, hidden, weight, a, plan,
                        product_descriptor(bf16, TILE_ROWS, TILE_TOKENS), parts, runs, logits, head_wait());
  if (err == cudaSuccess)
    err = launch_kernel(k_head_join, dim3(static_cast<unsigned>((a.rows + JOIN_THREADS / 32 - 1) / (JOIN_THREADS / 32))), dim3(JOIN_THREADS), 0,
                        stream, a, parts, logits, count);
  const cudaError_t freed = cudaFreeAsync(work, stream);
  return err != cudaSuccess ? err : freed;
}

}  // namespace profk
