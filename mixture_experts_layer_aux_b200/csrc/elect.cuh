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
