// What the convolution and the scan share: a row's length and states, elements of
// either type, the gate.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_device.cuh"
#include "spec_host.h"
#include "spec_paged.cuh"

namespace specv {

// A row's length, its initial state's slot (-1: zeros) and that of its last state (-1:
// none).  A row with a slot out of range has no tokens and no states.
struct MixerRow {
  int len;
  int from, to;
};

template <class T>
__device__ __forceinline__ MixerRow mixer_row(const T& A, int r, bool flag) {
  MixerRow R;
  R.len = A.lens ? min(max(__ldg(A.lens + r), 0), A.T) : A.T;
  const int s = A.slot ? __ldg(A.slot + r) : r, o = A.last_slot ? __ldg(A.last_slot + r) : r;
  R.from = A.state ? s : -1;
  R.to = A.last ? o : -1;
  if ((A.state && (s < 0 || s >= A.slots)) || (A.last && (o < 0 || o >= A.last_slots))) {
    R.len = 0;
    R.from = R.to = -1;
    if (flag && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
  }
  return R;
}

template <bool BF16>
__device__ __forceinline__ float load_one(const void* p, long long i) {
  if (BF16) return __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + i) << 16);
  return __ldg(static_cast<const float*>(p) + i);
}
template <bool BF16>
__device__ __forceinline__ void store_one(void* p, long long i, float x) {
  if (BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(x, 0.f);
  else static_cast<float*>(p)[i] = x;
}

// v / (1 + exp(-v)), with an error of a few units of 2^-24 (-0 from -87 down, where it is below 2^-119).
__device__ __forceinline__ float silu(float v) {
  float by;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(1.f + exp2_fast(-v * kLog2e)));
  return v * by;
}

// The checks of rows and slots that both calls share.
template <class T>
inline int mixer_check(const T& A) {
  if (A.B < 0 || A.B > 65535 || A.T < 0 || A.T > SPEC_MAX_LENGTH || A.slots < 0 || A.last_slots < 0) return SPEC_E_DIM;
  if (A.dtype != SPEC_F32 && A.dtype != SPEC_BF16) return SPEC_E_DTYPE;
  if ((A.state && !A.slot && A.slots < A.B) || (A.last && !A.last_slot && A.last_slots < A.B)) return SPEC_E_DIM;
  if (!paged_aligned(A.slot, 4) || !paged_aligned(A.last_slot, 4) || !paged_aligned(A.lens, 4) || !paged_aligned(A.flags, 4))
    return SPEC_E_ALIGN;
  return SPEC_OK;
}

}  // namespace specv
