// Tensor memory, the tensor cores' asynchronous products and tensor copies (PTX ISA: tcgen05, cp.async.bulk.tensor) for
// kernels of one CTA per SM, by itself (G = 1) or in pairs (G = 2: clusters of two CTAs whose tensor cores work on one
// product; the CTA of rank 0 issues it), and waits that give up.
#pragma once

#include <cuda.h>

#include "vsamp_device.cuh"

namespace vsamp {

// A box of a 2-D tensor map at element (x, y), x * element size a multiple of 16 bytes; elements outside the tensor are 0.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// The same by one CTA of a pair: the bytes are counted on a barrier of either CTA (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A box of shared memory (128-byte swizzle as the map says) to a 3-D tensor at element (x, y, z), none negative, x * element
// size a multiple of 16 bytes; what lies outside the tensor is not written. add: fp32 values are added in memory (those
// below 2^-126 too, as measured; red.global takes them for zeros). The box may be written again after bulk_read_done, and is in
// memory after bulk_done (both by the storing thread).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int32_t x, int32_t y, int32_t z, uint32_t src, bool add) {
  if (add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_read_done() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Registers per thread of this warpgroup from here on; the warpgroups' shares together stay within the launch's.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Bytes that were expected on a barrier of this CTA and will not come.
__device__ __forceinline__ void mbar_complete_tx(void* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// An arrival on a barrier of either CTA of a pair (a shared::cluster address) after tensor memory has been read. It carries
// no ordinary memory, so it has no cluster scope, whose release and acquire would cost hundreds of cycles.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Columns of tensor memory (a power of two from 32): called by one whole warp (of each CTA of a pair), which also frees them.
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t result, uint32_t columns) {
  if constexpr (G == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
  if constexpr (G == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

// True in one lane of a whole warp. What stands behind it may take its operands from the warp's uniform registers, as the
// instructions on tensor maps and descriptors want them: behind a comparison of the lane's number each operand is moved
// there by itself (a loop of four products 202 cycles instead of a few).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tcgen05_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tcgen05_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand of rows of 128 bytes along the inner dimension, 128-byte swizzle, in groups of eight rows (1024
// bytes, on such a boundary). A step of 32 bytes along the inner dimension adds 2 to the descriptor.
__device__ __forceinline__ uint64_t umma_operand(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// e4m3 x e4m3 -> fp32, both operands with the inner dimension contiguous, M x N results.
__host__ __device__ constexpr uint32_t umma_e4m3(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }

// One product over 32 elements of the inner dimension, added to what tensor memory holds unless `add` is 0. One thread. In
// a pair each CTA holds half of a's rows, which are its lanes of tensor memory, and half of b's.
template <int G>
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
  if constexpr (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}
// An arrival on `bar`, in a pair on both CTAs' barriers at that offset, once this thread's products so far are done.
template <int G>
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  if constexpr (G == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((unsigned short)3)
        : "memory");
}

// 16 or 32 columns of the warp's 32 lanes, waited for: load and wait are one statement, so that nothing reads the registers
// in between and none is copied.
__device__ __forceinline__ void tmem_read(uint32_t at, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(at)
      : "memory");
}

// 16 lanes of tensor memory, 32 columns: a thread gets of lane t / 4 the columns 8 k + 2 (t % 4) and the next one in r[4 k],
// r[4 k + 1], of lane t / 4 + 8 the same in r[4 k + 2], r[4 k + 3].
__device__ __forceinline__ void tmem_read_16(uint32_t at, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(at)
      : "memory");
}

// What this thread wrote to the other CTA's shared memory, and its arrivals there, are in place before anything that it does next
// (cluster_barrier_shared by itself publishes a thread's writes to its own CTA's shared memory alone).
__device__ __forceinline__ void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }

__device__ __forceinline__ void dsmem_publish_u32(uint32_t addr, uint32_t v) {
  dsmem_store_u32(addr, v);
  fence_cluster();
}

// Marks this CTA, and in a pair the other one too, as one of whose waits gave up. The marks are in place before anything that
// the thread does next: what it passes on without having waited for it is passed on to CTAs that are marked.
template <int G>
__device__ __forceinline__ void mark_dead(volatile int* dead) {
  if constexpr (G == 2) {
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    dsmem_publish_u32(dsmem_map(const_cast<int*>(dead), rank ^ 1), 1u);
  }
  *dead = 1;
}

// Waits for a phase of `bar`, until `limit` clock cycles have passed or the CTA is marked; then it, and a pair's other CTA, are
// marked and the answer is false.
template <int G>
__device__ __forceinline__ bool wait_alive(void* bar, uint32_t parity, volatile int* dead, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*dead || clock64() - t0 > limit) {
      mark_dead<G>(dead);
      return false;
    }
  }
}

}  // namespace vsamp
