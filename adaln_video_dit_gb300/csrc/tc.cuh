// Wrappers of the tensor-core instructions (tcgen05, tensor memory) and of the
// tensor (TMA) copies that feed them.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace adaln {

// ----- cluster ------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the same shared variable in another CTA of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Relaxed: for hand-overs of tensor memory, which tcgen05.wait::ld and the
// tcgen05 fences order.  A release at cluster scope would wait here until this
// thread's global stores are performed.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t mapped) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapped)
               : "memory");
}

// One lane of a converged warp.  Copies and matrix instructions are issued by
// a whole warp walking the loop with one lane elected at each issue, not by a
// lane on its own: their operands live in uniform registers, which the compiler
// can only use where control flow is uniform (a lone lane's TMA issue measured
// 235 cycles, half of what a stage's products take).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ----- TMA ----------------------------------------------------------------------
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Box of a 2-D tensor map at (x, y) into this CTA's shared memory; completion
// on barrier `bar` of this CTA.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int x, int y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// As above, for a CTA pair: completion on the pair's even CTA's barrier (bit 24
// of a shared-window address is the rank within the pair).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* m, int x, int y,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(bar & 0xFEFFFFFFu)
      : "memory");
}

// Box of shared memory to a 2-D tensor map at (x, y); what lies outside the
// tensor is not written.  Grouped per issuing thread: bulk_commit closes a
// group; bulk_wait_read<N> waits until the shared memory of all groups but the
// last N may be reused, bulk_wait until all are written.
__device__ __forceinline__ void tma_store(const CUtensorMap* m, int x, int y, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(m),
               "r"(x), "r"(y), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Make this thread's shared-memory writes visible to the copies.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// ----- tensor memory --------------------------------------------------------------
template <int G>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_out, uint32_t cols) {
  if (G == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (G == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// 32 lanes x 32 columns of 32 bits: register i of lane l is column i of lane l.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}

// ----- matrix instructions ----------------------------------------------------------
// Operand tiles live in shared memory as 128-byte-swizzled atoms of 8 rows x
// 128 bytes (1024-byte aligned), as a TMA box of 64 bf16 in x writes them.
//   rows of 64 k values ("K-major"):  8-row groups 1024 bytes apart;
//   rows of 64 m or n values ("MN-major"): 8-k groups 1024 bytes apart, the
//     next 64 m or n values `chunk` bytes on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major, uint32_t chunk) {
  const uint64_t lbo = mn_major ? chunk >> 4 : 1, sbo = 1024 >> 4;
  return (uint64_t)((addr >> 4) & 0x3FFF) | lbo << 16 | sbo << 32 | 1ull << 46 | 2ull << 61;
}
// Bytes from one 16-k step of a tile to the next.
__device__ __forceinline__ uint32_t k_step_bytes(bool mn_major) { return mn_major ? 2048 : 32; }

// bf16 x bf16 -> fp32, an M x N tile.
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, bool a_mn, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

template <int G>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  const uint32_t acc = accumulate;
  if (G == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Arrive on `bar` once the matrix instructions issued so far are done (G = 2:
// on that barrier of both CTAs of the pair).
template <int G>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if (G == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     bar)
                 : "memory");
}

}  // namespace adaln
