// elect.cuh -- one thread of a converged warp, for instructions that a single
// thread issues (tcgen05.mma and commit, TMA).
//
// The loops around such instructions are run by the whole warp, and only the
// instructions themselves sit behind elect_one(): everything they take
// (descriptors, addresses, coordinates) is then known to be the same in every
// lane and lives in uniform registers. In a loop that one lane runs alone, each
// operand is moved from a lane's register first: 0.33 us per k-block of four
// 256 x 256 x 16 pair MMAs and 0.32 of four 256 x 128 x 16 ones, against 0.29
// and 0.22 (T = H = F = 4096, one GEMM: 1488 and 1676 TFLOP/s).
#pragma once

#include "common.cuh"

// The same lane every time, as the commits must come from the thread whose MMAs they follow.
MOE_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
// mbar_wait by a whole warp.
MOE_DEV bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, code));
}
// The same for a barrier on which another CTA of the cluster arrives with relaxed.cluster after
// release_smem_cluster(): that CTA's ordinary stores to its shared memory are visible after it. The phase is observed at
// the cluster's scope, and the acquire is restricted to shared memory, so that it waits for no access to global memory.
MOE_DEV bool mbar_wait_warp_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int* status, int code) {
  uint32_t ok = 0;
  uint64_t t0 = 0;
  while (true) {
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) break;
    if (*abort) break;
    if (t0 == 0) t0 = globaltimer_ns();
    if (globaltimer_ns() - t0 > MOE_WAIT_NS) {
      *abort = 1;
      record_status(status, code);
      break;
    }
  }
  asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
  return __all_sync(0xffffffffu, ok != 0);
}
// Before a relaxed.cluster arrival: this thread's stores to its CTA's shared memory (and those it has observed) come
// before the arrival for whoever waits for it with mbar_wait_warp_cluster.
MOE_DEV void release_smem_cluster() {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
