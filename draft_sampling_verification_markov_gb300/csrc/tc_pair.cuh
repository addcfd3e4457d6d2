// tc_pair.cuh -- inline-PTX wrappers of what the vocabulary product (mx_logits.cu) uses beside
// tc_ptx.cuh: block-scaled MMAs of CTA pairs, scale copies into tensor memory, copies and arrivals
// across a cluster, and forms of these for warps whose lanes run a loop together.
#pragma once

#include "tc_ptx.cuh"

namespace spec {
namespace tc {

// Whether the phase of `parity` is complete, without waiting (try_wait may suspend the thread).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by a converged warp, with one answer for all its lanes (the votes keep the warp's
// control flow uniform, which its uniform registers need).
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               volatile int* abort, uint32_t* status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// Named barrier `id` of `threads` threads; whether `ok` holds in all of them.
__device__ __forceinline__ bool all_of(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.aligned.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------------------ block scaling

// Instruction descriptor, kind::mxf8f6f4 with E8M0 scales: element formats af / bf (0 = E4M3,
// 5 = E2M1), both operands K-major, fp32 accumulate, M x N. block_scale_ids adds which byte of a
// scale word (which 32-element block of a 128-element group) the instruction uses.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, int af, int bf) {
  return ((uint32_t)af << 7) | ((uint32_t)bf << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27);
}
__host__ __device__ constexpr uint32_t block_scale_ids(int b) {
  return ((uint32_t)b << 29) | ((uint32_t)b << 4);
}

// 1 in one lane of a converged warp, 0 in the others. A warp whose lanes all run an issue loop,
// with only the asynchronous instructions predicated on this, keeps their operands in uniform
// registers.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

// ---- CTA pairs (cta_group::2): the even CTA of a two-CTA cluster issues for both.

// D (+)= (A * sA) x (B * sB)^T, 32 elements of K, M = 256: each CTA holds its 128 rows of A and of
// D, half the rows of B, and one scale a row of its A and of all of B in tensor memory (lane =
// row % 32, column = row / 32). `lead`: issue from this lane.
__device__ __forceinline__ void mma_mx_pair(uint32_t lead, uint32_t d_tmem, uint64_t a_desc,
                                            uint64_t b_desc, uint32_t idesc, uint32_t sa_tmem,
                                            uint32_t sb_tmem, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.ne.b32 q, %7, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sa_tmem), "r"(sb_tmem), "r"(accumulate), "r"(lead)
      : "memory");
}

// Shared-memory descriptor of a scale tile for tcgen05.cp: 32 rows of 16 bytes, contiguous (no
// swizzle, 8-row groups 128 B apart).
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 16) |
         ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

// 512 bytes of each CTA's shared memory to four columns of its tensor memory: row i to lane i of
// each of the four lane quarters.
__device__ __forceinline__ void copy_scales_pair(uint32_t lead, uint32_t taddr, uint64_t desc) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc), "r"(lead)
      : "memory");
}

// Arrive on the barrier at this offset in the CTAs of `mask` once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t lead, uint64_t* bar, uint16_t mask = 3) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
      ".multicast::cluster.b64 [%0], %2;\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead), "h"(mask)
      : "memory");
}

// The cluster address of a local shared-memory object in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// Tile copy into this CTA that reports to a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t lead, void* dst, const CUtensorMap* map,
                                                 int c0, int c1, uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar), "l"(policy), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void expect_tx_if(uint32_t lead, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(lead)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace tc
}  // namespace spec
