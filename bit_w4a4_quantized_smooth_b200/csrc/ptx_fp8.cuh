// PTX wrappers that the 8-bit kernels alone use, beside those of ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace svdq {

// Counts this warp in at a named barrier without waiting.
__device__ __forceinline__ void named_bar_arrive(uint32_t id, uint32_t count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// warp_wait with one test and one vote where the phase is already complete.
__device__ __forceinline__ bool warp_wait_ready(uint32_t bar, uint32_t parity, uint64_t timeout_ns,
                                                unsigned int where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, timeout_ns, where);
}

// The four block-scaled FP8 MMAs (E4M3 operands, K = 32 each, one UE8M0 scale
// per 32 along K read from tmem; idesc chooses the byte of each scale word) of
// a 128-column stage, then the arrival on `bar` when they are complete: one
// election for all five.  (Elected one by one the four MMAs took a warp 186
// cycles to issue on B200, measured with the cycle counter.)  The descriptors
// advance by 32 bytes an MMA; the first MMA starts the accumulator when
// `accumulate` is 0.
#define SVDQ_MXF8_STAGE(group, commit)                                                                              \
  SVDQ_ELECT_BEGIN ".reg .pred p, t;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"        \
  "@e tcgen05.mma.cta_group::" group ".kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t"      \
  "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"                                                                     \
  "@e tcgen05.mma.cta_group::" group ".kind::mxf8f6f4.block_scale.block32 [%0], a, b, %3, [%5], [%6], t;\n\t"        \
  "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"                                                                     \
  "@e tcgen05.mma.cta_group::" group ".kind::mxf8f6f4.block_scale.block32 [%0], a, b, %3, [%5], [%6], t;\n\t"        \
  "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"                                                                     \
  "@e tcgen05.mma.cta_group::" group ".kind::mxf8f6f4.block_scale.block32 [%0], a, b, %3, [%5], [%6], t;\n\t"        \
  commit SVDQ_ELECT_END

__device__ __forceinline__ void e_stage_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate, uint32_t bar) {
  asm volatile(SVDQ_MXF8_STAGE("1", "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];") ::
                   "r"(d_tmem),
               "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem), "r"(bar)
               : "memory");
}

// Across the CTA pair (issued by the even CTA); the arrival goes to the barrier
// at the same offset in both CTAs.
__device__ __forceinline__ void e_stage_mxf8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                  uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate,
                                                  uint32_t bar) {
  asm volatile(
      SVDQ_MXF8_STAGE("2",
                      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                      " [%7], %8;") ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem), "r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// A stage's expected bytes and its two 2-D loads, one election for the three.
__device__ __forceinline__ void e_stage_load(uint32_t bar, uint32_t tx, uint32_t dst0, const void* tmap0, int y0,
                                             uint32_t dst1, const void* tmap1, int y1, int x) {
  asm volatile(SVDQ_ELECT_BEGIN
               "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
               "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
               " [%2], [%3, {%8, %4}], [%0];\n\t"
               "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
               " [%5], [%6, {%8, %7}], [%0];" SVDQ_ELECT_END ::"r"(bar),
               "r"(tx), "r"(dst0), "l"(tmap0), "r"(y0), "r"(dst1), "l"(tmap1), "r"(y1), "r"(x)
               : "memory");
}

// The same in a CTA pair: both CTAs' loads complete on the even CTA's barrier
// `bar_cluster`, which the even CTA (`arms` = 1, its own address `bar`) arms.
__device__ __forceinline__ void e_stage_load_pair(uint32_t bar_cluster, uint32_t arms, uint32_t bar, uint32_t tx,
                                                  uint32_t dst0, const void* tmap0, int y0, uint32_t dst1,
                                                  const void* tmap1, int y1, int x) {
  asm volatile(SVDQ_ELECT_BEGIN ".reg .pred q;\n\tsetp.ne.b32 q, %9, 0;\n\tand.pred q, q, e;\n\t"
               "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%10], %1;\n\t"
               "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
               " [%2], [%3, {%8, %4}], [%0];\n\t"
               "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
               " [%5], [%6, {%8, %7}], [%0];" SVDQ_ELECT_END ::"r"(bar_cluster),
               "r"(tx), "r"(dst0), "l"(tmap0), "r"(y0), "r"(dst1), "l"(tmap1), "r"(y1), "r"(x), "r"(arms), "r"(bar)
               : "memory");
}

}  // namespace svdq
