// spec_recur: h_t = exp(g_t) h_{t-1} + x_t, channel by channel, and its backward
// pass.  One thread a channel walks its row's tokens in order.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_host.h"
#include "spec_paged.cuh"

namespace specv {

struct RecurArgs {
  const unsigned char* g;
  const unsigned char* x;      // forward: x; backward: dh
  const unsigned char* hin;    // backward: h
  unsigned char* h;            // forward: h; backward: dx
  unsigned char* dg;
  const float* state;
  const int32_t* slot;
  const int32_t* lens;
  float* last;                 // forward: the last states; backward: d_state
  const int32_t* last_slot;
  const float* d_last;
  uint32_t* flags;
  long long g_row, g_tok, x_row, x_tok;   // elements
  int B, T, D, slots, last_slots;
};

template <bool BF16>
__device__ __forceinline__ float elem(const unsigned char* p, long long i) {
  if (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
  return reinterpret_cast<const float*>(p)[i];
}

template <bool BF16>
__device__ __forceinline__ void put(unsigned char* p, long long i, float x) {
  if (BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(x, 0.f);
  else reinterpret_cast<float*>(p)[i] = x;
}

// A row's length, its initial state's place (-1: zeros) and that of its last
// state (-1: none); false (and flagged) where a slot is out of range.
__device__ __forceinline__ bool recur_row(const RecurArgs& A, int r, int* len, long long* from, long long* to) {
  *len = A.lens ? min(max(A.lens[r], 0), A.T) : A.T;
  const int s = A.slot ? A.slot[r] : r, o = A.last_slot ? A.last_slot[r] : r;
  const bool ok = (!A.state || (s >= 0 && s < A.slots)) && (!A.last || (o >= 0 && o < A.last_slots));
  *from = A.state && ok ? (long long)s * A.D : -1;
  *to = A.last && ok ? (long long)o * A.D : -1;
  return ok;
}

template <bool BF16, bool HBF16>
__global__ void recur_kernel(const RecurArgs A) {
  const int r = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= A.D) return;
  int len;
  long long from, to;
  const bool ok = recur_row(A, r, &len, &from, &to);
  if (!ok) {
    if (c == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
    len = 0;
  }
  float h = from >= 0 ? A.state[from + c] : 0.f;
  const long long base = (long long)r * A.T * A.D + c;
  for (int t = 0; t < len; ++t) {
    const float a = expf(elem<BF16>(A.g, r * A.g_row + t * A.g_tok + c));
    h = fmaf(a, h, elem<BF16>(A.x, r * A.x_row + t * A.x_tok + c));
    put<HBF16>(A.h, base + (long long)t * A.D, h);
  }
  for (int t = len; t < A.T; ++t) put<HBF16>(A.h, base + (long long)t * A.D, 0.f);
  if (to >= 0) A.last[to + c] = h;
}

template <bool BF16, bool HBF16>
__global__ void recur_backward_kernel(const RecurArgs A) {
  const int r = blockIdx.y, c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= A.D) return;
  int len;
  long long from, to;
  const bool ok = recur_row(A, r, &len, &from, &to);
  if (!ok) {
    if (c == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
    len = 0;
  }
  const long long base = (long long)r * A.T * A.D + c;
  for (int t = len; t < A.T; ++t) {
    put<BF16>(A.h, base + (long long)t * A.D, 0.f);
    put<BF16>(A.dg, base + (long long)t * A.D, 0.f);
  }
  float carry = A.d_last && ok ? A.d_last[(long long)r * A.D + c] : 0.f;
  for (int t = len - 1; t >= 0; --t) {
    const float a = expf(elem<BF16>(A.g, r * A.g_row + t * A.g_tok + c));
    const float lam = elem<BF16>(A.x, base + (long long)t * A.D) + carry;
    const float before = t ? elem<HBF16>(A.hin, base + (long long)(t - 1) * A.D) : from >= 0 ? A.state[from + c] : 0.f;
    carry = a * lam;
    put<BF16>(A.h, base + (long long)t * A.D, lam);
    put<BF16>(A.dg, base + (long long)t * A.D, carry * before);
  }
  if (A.last) A.last[(long long)r * A.D + c] = carry;
}

template <bool BWD>
static int recur_launch(RecurArgs& A, int dtype, int h_dtype, cudaStream_t st) {
  const dim3 grid((A.D + 127) / 128, A.B);
  const bool b = dtype == SPEC_BF16, hb = h_dtype == SPEC_BF16;
  if (BWD) {
    if (b) hb ? recur_backward_kernel<true, true><<<grid, 128, 0, st>>>(A) : recur_backward_kernel<true, false><<<grid, 128, 0, st>>>(A);
    else hb ? recur_backward_kernel<false, true><<<grid, 128, 0, st>>>(A) : recur_backward_kernel<false, false><<<grid, 128, 0, st>>>(A);
  } else {
    if (b) hb ? recur_kernel<true, true><<<grid, 128, 0, st>>>(A) : recur_kernel<true, false><<<grid, 128, 0, st>>>(A);
    else hb ? recur_kernel<false, true><<<grid, 128, 0, st>>>(A) : recur_kernel<false, false><<<grid, 128, 0, st>>>(A);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

static bool recur_dims(int B, int T, int D) { return B >= 0 && B <= 65535 && T >= 0 && D >= 1 && D <= (1 << 26); }

// The checks both passes share.
static int recur_check(int dtype, int h_dtype, int B, int T, int D, int slots, int last_slots, const int32_t* slot,
                       const int32_t* last_slot, const float* state, const float* last, const int32_t* lens,
                       const uint32_t* flags) {
  if (!recur_dims(B, T, D) || slots < 0 || last_slots < 0) return SPEC_E_DIM;
  if ((dtype != SPEC_F32 && dtype != SPEC_BF16) || (h_dtype != SPEC_F32 && h_dtype != SPEC_BF16)) return SPEC_E_DTYPE;
  if (state && !slot && slots < B) return SPEC_E_DIM;
  if (last && !last_slot && last_slots < B) return SPEC_E_DIM;
  if (!paged_aligned(slot, 4) || !paged_aligned(last_slot, 4) || !paged_aligned(state, 4) || !paged_aligned(last, 4) ||
      !paged_aligned(lens, 4) || !paged_aligned(flags, 4))
    return SPEC_E_ALIGN;
  return SPEC_OK;
}

}  // namespace specv

extern "C" size_t spec_recur_workspace_size(int B, int T, int D) {
  if (!specv::recur_dims(B, T, D)) return 0;
  return 256;
}

extern "C" int spec_recur(const void* g, int64_t g_row, int64_t g_tok, const void* x, int64_t x_row, int64_t x_tok,
                          int dtype, const float* state, const int32_t* slot, int slots, const int32_t* lens, int B,
                          int T, int D, void* h, int h_dtype, float* last, const int32_t* last_slot, int last_slots,
                          uint32_t* flags, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  using namespace specv;
  const int rc = recur_check(dtype, h_dtype, B, T, D, slots, last_slots, slot, last_slot, state, last, lens, flags);
  if (rc != SPEC_OK) return rc;
  if (B == 0) return SPEC_OK;
  if (T > 0 && (!g || !x || !h)) return SPEC_E_NULL;
  if (!workspace) return SPEC_E_NULL;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4, hs = h_dtype == SPEC_BF16 ? 2 : 4;
  if (!paged_aligned(g, es) || !paged_aligned(x, es) || !paged_aligned(h, hs) || !paged_aligned(workspace, 256))
    return SPEC_E_ALIGN;
  if (workspace_bytes < spec_recur_workspace_size(B, T, D)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  RecurArgs A = {};
  A.g = static_cast<const unsigned char*>(g);
  A.x = static_cast<const unsigned char*>(x);
  A.h = static_cast<unsigned char*>(h);
  A.state = state;
  A.slot = slot;
  A.lens = lens;
  A.last = last;
  A.last_slot = last_slot;
  A.flags = flags;
  A.g_row = g_row;
  A.g_tok = g_tok;
  A.x_row = x_row;
  A.x_tok = x_tok;
  A.B = B;
  A.T = T;
  A.D = D;
  A.slots = slots;
  A.last_slots = last_slots;
  return recur_launch<false>(A, dtype, h_dtype, reinterpret_cast<cudaStream_t>(cuda_stream));
}

extern "C" int spec_recur_backward(const void* g, int64_t g_row, int64_t g_tok, const void* h, int h_dtype,
                                   const void* dh, const float* d_last, int dtype, const float* state,
                                   const int32_t* slot, int slots, const int32_t* lens, int B, int T, int D, void* dg,
                                   void* dx, float* d_state, uint32_t* flags, void* workspace, size_t workspace_bytes,
                                   void* cuda_stream) {
  using namespace specv;
  const int rc = recur_check(dtype, h_dtype, B, T, D, slots, B, slot, nullptr, state, d_state, lens, flags);
  if (rc != SPEC_OK) return rc;
  if (B == 0) return SPEC_OK;
  if (T > 0 && (!g || !h || !dh || !dg || !dx)) return SPEC_E_NULL;
  if (!workspace) return SPEC_E_NULL;
  const size_t es = dtype == SPEC_BF16 ? 2 : 4, hs = h_dtype == SPEC_BF16 ? 2 : 4;
  if (!paged_aligned(g, es) || !paged_aligned(dh, es) || !paged_aligned(dg, es) || !paged_aligned(dx, es) ||
      !paged_aligned(h, hs) || !paged_aligned(d_last, 4) || !paged_aligned(workspace, 256))
    return SPEC_E_ALIGN;
  if (workspace_bytes < spec_recur_workspace_size(B, T, D)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  RecurArgs A = {};
  A.g = static_cast<const unsigned char*>(g);
  A.x = static_cast<const unsigned char*>(dh);
  A.hin = static_cast<const unsigned char*>(h);
  A.h = static_cast<unsigned char*>(dx);
  A.dg = static_cast<unsigned char*>(dg);
  A.state = state;
  A.slot = slot;
  A.lens = lens;
  A.last = d_state;
  A.d_last = d_last;
  A.flags = flags;
  A.g_row = g_row;
  A.g_tok = g_tok;
  A.B = B;
  A.T = T;
  A.D = D;
  A.slots = slots;
  A.last_slots = B;
  return recur_launch<true>(A, dtype, h_dtype, reinterpret_cast<cudaStream_t>(cuda_stream));
}
