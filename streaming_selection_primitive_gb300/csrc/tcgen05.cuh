// Instructions of the asynchronous units, as logprobs.cu and head.cu use them: barriers in
// shared memory whose waits are bounded, copies that count on them, stores to other CTAs of
// a cluster, and (head.cu) products on the tensor cores with their accumulators in tensor memory.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace profk {

__device__ __forceinline__ uint32_t shared_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// ---- barriers in shared memory ----

__device__ __forceinline__ void barrier_init(uint64_t* b, unsigned arrivals) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(shared_address(b)), "r"(arrivals) : "memory");
}
// Makes the initialised barriers visible to the copies and products that arrive on them.
__device__ __forceinline__ void barrier_init_done() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

__device__ __forceinline__ void barrier_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(shared_address(b)) : "memory");
}
__device__ __forceinline__ void barrier_arrive_expect(uint64_t* b, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(shared_address(b)), "r"(bytes) : "memory");
}

// CLUSTER: what other CTAs of the cluster wrote before their arrivals is seen, too.
template <bool CLUSTER>
__device__ __forceinline__ bool barrier_passed(uint64_t* b, unsigned parity) {
  unsigned ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(shared_address(b)), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(shared_address(b)), "r"(parity)
        : "memory");
  return ok != 0;
}

// Waits for the phase of that parity; false if it did not come within `limit` polls or
// another warp of the CTA has given up (*given_up, in shared memory, which this sets too).
template <bool CLUSTER = false>
__device__ __forceinline__ bool barrier_wait(uint64_t* b, unsigned parity, volatile int* given_up, int limit) {
  for (int poll = 0; poll < limit; ++poll) {
    if (barrier_passed<CLUSTER>(b, parity)) return true;
    if (*given_up) return false;
  }
  *given_up = 1;
  return false;
}

// ---- clusters ----

// The cluster's first barrier in two halves, without a fence (fence.mbarrier_init orders the
// barriers' beginnings): behind the second one every CTA of the cluster runs.
__device__ __forceinline__ void cluster_begin() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_begun() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 16 bytes to the same place of CTA `rank`'s shared memory, counted on its barrier.  Only in kernels that
// are launched as clusters, of one CTA too: without the launch's attribute this is an illegal instruction.
__device__ __forceinline__ void store_remote(void* to, float4 v, uint64_t* counted_on, int rank) {
  uint32_t a, b;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(shared_address(to)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(shared_address(counted_on)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w), "r"(b)
               : "memory");
}

// ---- tile copies ----

__device__ __forceinline__ void copy_tile(void* to, const void* map, int x, int y, uint64_t* done) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(shared_address(to)),
      "l"(map), "r"(x), "r"(y), "r"(shared_address(done))
      : "memory");
}

// A run of bytes: both addresses and the length are multiples of 16.
__device__ __forceinline__ void copy_bytes(void* to, const void* from, unsigned bytes, uint64_t* done) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(shared_address(to)), "l"(from),
               "r"(bytes), "r"(shared_address(done))
               : "memory");
}

// ---- products ----

// A tile of rows of 128 bytes, swizzled as the copies write it (atoms of 8 rows, 1024
// bytes), its first element at `p`: 16-bit values along a row are the product's depth.
__device__ __forceinline__ uint64_t tile_descriptor(const void* p) {
  constexpr uint64_t ATOM = 1024 >> 4, VERSION = 1, SWIZZLE_128 = 2;
  return (static_cast<uint64_t>(shared_address(p) >> 4) & 0x3fff) | (uint64_t(1) << 16) | (ATOM << 32) | (VERSION << 46) | (SWIZZLE_128 << 61);
}

// D (float32, m rows in the lanes of tensor memory, n columns) of A and B, both bfloat16
// or both float16, both with their depth along the rows of their tiles.
__host__ __device__ constexpr uint32_t product_descriptor(bool bf16, int m, int n) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

__device__ __forceinline__ void multiply(uint32_t d, uint64_t a, uint64_t b, uint32_t how, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(how), "r"(uint32_t(add))
      : "memory");
}
// The barrier gets an arrival when the products issued so far by this thread are done.
__device__ __forceinline__ void products_arrive(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(shared_address(b)) : "memory");
}

__device__ __forceinline__ void before_barrier() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_barrier() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- tensor memory ----

// By a whole warp; the address goes to *at in shared memory.
template <int COLUMNS>
__device__ __forceinline__ void tensor_alloc(uint32_t* at) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(shared_address(at)), "n"(COLUMNS) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
template <int COLUMNS>
__device__ __forceinline__ void tensor_free(uint32_t at) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "n"(COLUMNS));
}

// 32 columns of this warp's quarter of the lanes: a thread has its lane's.
__device__ __forceinline__ void tensor_load(float (&v)[32], uint32_t at) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tensor_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

}  // namespace profk
