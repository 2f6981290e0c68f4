// Shared device pieces of the language-model selections (tokens.cu, route.cuh).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"

namespace profk {

__device__ __forceinline__ float lm_float(float v) { return v; }
__device__ __forceinline__ float lm_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float lm_float(__half v) { return __half2float(v); }

// One rounding, to the caller's type, at the end of a computation in float32.
template <typename T>
__device__ __forceinline__ T lm_cast(float v);
template <>
__device__ __forceinline__ float lm_cast<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 lm_cast<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half lm_cast<__half>(float v) { return __float2half_rn(v); }

// Order key of a value that may be chosen: ord_key, whose smallest value (ord
// of -inf) is above zero; 0 for what may not be chosen (-inf and NaN).
__device__ __forceinline__ uint32_t choice_key(float v) { return v > -INFINITY ? ord_key(v) : 0u; }

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

// 2^x by the hardware's approximation (two ulps; results below the normal
// range are zero).
__device__ __forceinline__ float lm_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float lm_sqrt(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x by the hardware's approximation (one ulp; x or results below the
// normal range count as zero).  What it divides carries two ulps of an
// exponential already.
__device__ __forceinline__ float lm_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The line of p to L2.
__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL_MASK, v, d));
  return v;
}

// Static shared memory of a kernel that is launched by launch_clusters_most with a few KB of dynamic one
// below 48 KB: no more than this.
constexpr size_t STATIC_ROOM = 8 * 1024;

// Launches a kernel whose CTAs form clusters of `cluster`, as launch_kernel does, with `smem`
// bytes of dynamic shared memory, `most` being what any call of it asks for.  (The
// limit is the kernel's, for all host threads: it is set to the same number whatever the call.)
template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters_most(void (*kernel)(KArgs...), int64_t grid, int threads, int cluster, size_t smem,
                                        size_t most, cudaStream_t stream, Args... args) {
  if (smem + STATIC_ROOM > 48 * 1024) {  // (what a launch has without asking holds static and dynamic memory together)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
  }
  ++launch_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... KArgs, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(KArgs...), int64_t grid, int threads, int cluster, size_t smem,
                                   cudaStream_t stream, Args... args) {
  return launch_clusters_most(kernel, grid, threads, cluster, smem, smem, stream, args...);
}

}  // namespace profk
