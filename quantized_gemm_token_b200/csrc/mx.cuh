// mx.cuh -- device helpers of the microscaled kernels: the converged issuing
// warp, barrier tests ahead of time, and small shared-memory accesses.
#pragma once

#include <cstdint>

#include "pipeline.cuh"
#include "sm100.cuh"

namespace dq {

// One lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0;
}

// Whether the phase with the given parity of `bar` has completed (no waiting).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait by a whole converged warp; the result is the warp's.  An issuing
// warp that stays converged (this wait, and elect_one() around the
// instructions that one thread issues) keeps its descriptors and addresses in
// uniform registers, where tcgen05 instructions take them from; issued from a
// branch of a single lane each tcgen05 instruction took 60 - 100 cycles (the
// 4-bit product of 8192^3: 483 us so, 273 us converged).
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, const WaitCtl& ctl,
                                               volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, abort));
}

// The same for two phases that were tested (mbar_test) earlier: a test's
// answer takes about 100 cycles, so a loop that feeds the tensor core asks for
// the next step's before it issues the present one's MMAs (two waits and two
// commits per 512-cycle step: 661 cycles per step without, 515 with).
__device__ __forceinline__ bool mbar_wait_warp2(bool tested, uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                                uint32_t parity1, const WaitCtl& ctl, volatile int* abort) {
  if (__all_sync(0xffffffffu, tested)) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar0, parity0, ctl, abort) && mbar_wait(bar1, parity1, ctl, abort));
}

// Brings a tile towards L2 only: no shared memory, nothing to wait for.  L2 is
// where all writers of the tile meet, so unlike a load it may be issued before
// the kernels ahead in the stream have completed.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y)
               : "memory");
}

namespace pipe {

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Barrier `id` over `nthreads` threads (all of them converged warps) that
// returns whether all of them passed true: roles that leave together on a
// failed wait.
__device__ __forceinline__ bool bar_and(int id, int nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\tbarrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

}  // namespace pipe
}  // namespace dq
