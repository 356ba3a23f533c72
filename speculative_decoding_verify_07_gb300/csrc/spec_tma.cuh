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

// One try that lets the thread sleep for up to a millisecond: threads that poll
// take issue slots from those that they wait for.
__device__ __forceinline__ bool mbar_sleep_wait(unsigned long long* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u) : "memory");
  return ok != 0;
}

// Waits for the phase; sets *failed and returns when it does not come within
// two seconds, or when another wait of this CTA has given up.
__device__ __forceinline__ void mbar_await(unsigned long long* bar, uint32_t parity, volatile int* failed) {
  if (mbar_sleep_wait(bar, parity)) return;
  const unsigned long long began = global_ns();
  while (!mbar_sleep_wait(bar, parity)) {
    if (*failed) return;
    if (global_ns() - began > 2000000000ull) *failed = 1;
  }
}

}  // namespace specv
