// Tensor maps, TMA loads and bounded waits for them.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "spec_device.cuh"

namespace specv {

using TensorMapEncode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                     const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                     CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Lets a kernel have `bytes` of shared memory, once a device; `done` is the kernel's own.
inline bool allow_shared(const void* kernel, int bytes, std::atomic<unsigned long long>* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done->load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done->fetch_or(bit);
  return true;
}

// cuTensorMapEncodeTiled, looked up once (the library does not link the driver); null where there is none.
TensorMapEncode tensor_map_encoder();

__device__ __forceinline__ void tma_load_3d(uint32_t smem, const CUtensorMap* map, int x, int y, int z, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t smem, const CUtensorMap* map, int x, int y, int z, int w,
                                            unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// How long a wait may take before its call is flagged, and how much longer before
// it is given up.  (A variable of the build, so that a wait can be made to run out.)
#ifndef SPEC_WAIT_NS
#define SPEC_WAIT_NS 2000000000ull
#endif
constexpr unsigned long long kWaitNs = SPEC_WAIT_NS, kGiveUpNs = kWaitNs + 2000000000ull;
constexpr int kLate = 1, kGivenUp = 2;

// One try that lets the thread sleep for a while (none for 0 ns): threads that poll
// take issue slots from those that they wait for.
__device__ __forceinline__ bool mbar_sleep_wait(unsigned long long* bar, uint32_t parity, unsigned ns) {
  uint32_t ok;
  if (ns == 0) {
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
  }
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(ns) : "memory");
  return ok != 0;
}

// Waits for the phase.  Where it does not come in time *failed becomes kLate and the
// wait goes on, since what is on its way still lands here; where it does not come at
// all, kGivenUp, from when on no wait of this CTA waits and nothing more is begun: a
// barrier takes no arrival for the next phase before the last has ended.
__device__ __forceinline__ void mbar_await(unsigned long long* bar, uint32_t parity, int* failed) {
  constexpr unsigned nap = kWaitNs < 100000 ? (unsigned)kWaitNs : 100000;
  if (mbar_sleep_wait(bar, parity, nap)) return;
  const unsigned long long began = global_ns();
  while (!mbar_sleep_wait(bar, parity, nap)) {
    if (*(volatile int*)failed == kGivenUp) return;
    const unsigned long long waited = global_ns() - began;
    if (waited >= kWaitNs) atomicMax(failed, waited >= kGiveUpNs ? kGivenUp : kLate);
  }
}
__device__ __forceinline__ bool mbar_given_up(const int* failed) { return *(const volatile int*)failed == kGivenUp; }

// The end of a CTA that has given up: a second in which what is still on its way to
// its memory lands there.
__device__ __forceinline__ void mbar_settle(const int* failed) {
  if (!mbar_given_up(failed)) return;
  const unsigned long long began = global_ns();
  for (int i = 0; i < 2000 && global_ns() - began < 1000000000ull; ++i) __nanosleep(1000000);
}

}  // namespace specv
