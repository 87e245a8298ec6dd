// tcgen05 and TMA instructions issued by one elected lane of a converged warp.
//
// These instructions take their operands from uniform registers.  Where the
// issuing lane is picked by a predicate or a branch on the thread index, the
// operands are not known to be uniform and each MMA costs about 110 cycles to
// issue, whatever its size (measured: M 128, K 16, N 16 to 128).  With the
// lane elected inside the instruction's own block, in a warp whose index came
// through a shuffle, it is 39 cycles for N = 16 and 64 for N = 128, the
// tensor core's own time; votes and exits between the MMAs add to that (four
// MMAs, N = 128, with two waits and two commits: 411 cycles in a loop that
// leaves on a failed wait, 260 unrolled with waits that do not).
#pragma once
#include "tc_utils.cuh"

namespace mla {
namespace tc {

// The index of this thread's warp, known to be the same in all of its lanes.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one != 0;
}

// Bounded wait of a converged warp, without the vote and the early return of
// mbar_wait_warp: code after it stays one straight line, in which the operands
// of the instructions below are known to be uniform.  False when the wait ran
// out or another role gave up (the caller goes on to its next check).
template <bool kCluster>
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !(kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)); ++i) {
    if ((i & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) *abort_flag = 1;
      if (*abort_flag) return false;
    }
  }
  return true;
}

// A word of a CTA of the cluster's shared memory (address from map_to_rank).
__device__ __forceinline__ void st_cluster_u32(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void pause_ns(uint64_t ns) {
  for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < ns;) __nanosleep(1000);
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f16.
__device__ __forceinline__ void mma_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrive on the mbarrier when every MMA issued so far has completed.
__device__ __forceinline__ void mma_commit_elect(uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}\n" ::"r"(bar)
      : "memory");
}
// The same, if the elected lane says so.
__device__ __forceinline__ void mma_commit_elect_if(uint32_t bar, bool yes) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.and.b32 p, %1, 0, q;\n"
      "@p tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n"
      "}\n" ::"r"(bar),
      "r"(static_cast<uint32_t>(yes))
      : "memory");
}
// Load the 3-D box at {x, y, z}, completing on the mbarrier.
__device__ __forceinline__ void tma_load_3d_elect(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                                  uint32_t bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n"
      "}\n" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// The same over a CTA pair (cta_group::2), issued in its even CTA.
__device__ __forceinline__ void mma_pair_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrive on the mbarrier at this offset in the CTAs of the pair that `ctas`
// has a bit for.
__device__ __forceinline__ void commit_pair_elect(uint32_t bar, int ctas) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
      "}\n" ::"r"(bar),
      "h"(static_cast<uint16_t>(ctas))
      : "memory");
}
// The same, if the elected lane says so.
__device__ __forceinline__ void commit_pair_elect_if(uint32_t bar, int ctas, bool yes) {
  asm volatile(
      "{\n"
      ".reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.and.b32 p, %2, 0, q;\n"
      "@p tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
      "}\n" ::"r"(bar),
      "h"(static_cast<uint16_t>(ctas)), "r"(static_cast<uint32_t>(yes))
      : "memory");
}
// Load the 3-D box at {x, y, z}, completing on an mbarrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_3d_pair_elect(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                                       uint32_t cluster_bar) {
  asm volatile(
      "{\n"
      ".reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];\n"
      "}\n" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
      : "memory");
}

}  // namespace tc
}  // namespace mla
