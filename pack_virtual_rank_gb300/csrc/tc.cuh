// tc.cuh -- the sm_103a primitives of the head's products: mbarriers with bounded waits, tensor
// map loads and stores, tcgen05 (tensor memory, descriptors, matrix products).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace relay {
namespace {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// ------------------------------------------------------------------- barriers --

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n.reg .b64 s;\nmbarrier.arrive.expect_tx.shared::cta.b64 s, [%0], %1;\n}" ::"r"(bar), "r"(bytes)
               : "memory");
}
// Arrival at a barrier of either CTA of the pair (an address from pair_addr).
__device__ __forceinline__ void bar_arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// PAIR: what ordinary stores of the other CTA wrote before its arrival is seen, too. Where a barrier stands for loads by tensor
// maps, products or this CTA's own stores, that is not needed.
template <bool PAIR = true>
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (!PAIR) {
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  }
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Every wait of a product ends: when its barrier completes, when another warp of the CTA gave
// up, or after kWaitNs. The slowest wait of a healthy run is one tile's products.
constexpr uint64_t kWaitNs = 500000000ull;
template <bool PAIR = true>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* gave_up) {
  if (bar_try<PAIR>(bar, parity)) return true;
  uint64_t start = 0;  // the clock is read once a wait has become a long one
  for (uint32_t i = 1;; ++i) {
    if (bar_try<PAIR>(bar, parity)) return true;
    if (i % 64 == 0) {
      if (*gave_up) return false;
      const uint64_t now = global_ns();
      if (start == 0) start = now;
      if (now - start > kWaitNs) {
        *gave_up = 1;
        return false;
      }
    }
  }
}

// --------------------------------------------------------------- pairs of CTAs --

__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// The address, in CTA `rank` of the pair, of a shared memory address of this CTA.
__device__ __forceinline__ uint32_t pair_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Every thread of both CTAs calls it; there is no way around it in either.
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ----------------------------------------------------------------- tensor maps --

// Into this CTA's shared memory; the bytes are counted at a barrier of either CTA of the pair.
template <int CTAS>
__device__ __forceinline__ void map_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void map_prefetch(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void map_store(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(y), "r"(src)
               : "memory");
}
// Adds the box to what memory holds (fp32).
__device__ __forceinline__ void map_add(const CUtensorMap* map, int x, int y, uint32_t src) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(PENDING) : "memory");
}
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// --------------------------------------------------------------------- tcgen05 --
// CTAS 2: a pair of CTAs makes one product: tensor memory is allocated by both, one thread of the first
// issues, each CTA holds half the rows of A and of B, and gets half the rows of the result.

template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  if constexpr (CTAS == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t cols) {
  if constexpr (CTAS == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The barrier at this address in every CTA of the product gets one arrival when every product issued
// before by this thread is done.
template <int CTAS>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CTAS == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 32 lanes x 16 columns of fp32: lane i of the warp gets row i's columns. The whole warp calls it;
// the load and its wait are one statement, so that nothing reads v in between.
__device__ __forceinline__ void tmem_load16(uint32_t tmem, float* v) {
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(tmem)
      : "memory");
}

// Shared memory descriptors of bf16 operands, K inner elements of them to a stage (tiles at 1024-byte addresses).
//  inner dimension contiguous: rows of K elements with a swizzle of their width (128 or 64 bytes), groups
//  of 8 rows one behind the other.
//  outer dimension contiguous: boxes of 64 outer elements (128-byte rows and swizzle) by K inner rows;
//  groups of 8 inner rows 1024 bytes apart, boxes of 64 outer elements 128 K bytes apart.
template <int K>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool outer_contiguous) {
  static_assert(K == 64 || K == 32, "128 or 64 bytes");
  uint64_t d = (uint64_t)((addr & 0x3ffffu) >> 4);
  d |= (uint64_t)(outer_contiguous ? 128 * K >> 4 : 1) << 16;
  d |= (uint64_t)(outer_contiguous ? 1024 >> 4 : 16 * K >> 4) << 32;
  d |= 1ull << 46;
  d |= (outer_contiguous || K == 64 ? 2ull : 4ull) << 61;
  return d;
}
// Descriptor advance (16-byte units) for the next 16 elements of the inner dimension.
__device__ __forceinline__ constexpr uint32_t operand_step(bool outer_contiguous) {
  return outer_contiguous ? 2048 >> 4 : 32 >> 4;
}
// fp32 accumulator, bf16 operands, M x N.
__host__ __device__ constexpr uint32_t product_desc(int m, int n, bool a_outer, bool b_outer) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_outer << 15) | ((uint32_t)b_outer << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
template <int CTAS>
__device__ __forceinline__ void tc_product(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  if constexpr (CTAS == 2)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

}  // namespace
}  // namespace relay
