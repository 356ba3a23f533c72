// spec_attend: attention of each row's new tokens over its paged cache.
//
// The plain form of the operator: one CTA a (token, query head).  Its warps
// take the visible positions in turn, each with a running maximum m, sum l and
// weighted sum of values (one pass: when m grows by d the sums shrink by
// exp(-d)); the warps' partials are joined at the end in a fixed order.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_host.h"
#include "spec_paged.cuh"

namespace specv {

struct AttendArgs {
  PagedCache C;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  uint32_t* flags;
  long long q_token;     // elements from token to token of q
  int N, group, hq;
  float scale;
};

constexpr int kAttendWarps = 4;

template <int PER>
__device__ __forceinline__ void load_vec(const unsigned char* pool, const uint8_t* exps, const PagedCache& C, bool e4m3,
                                         int page, int head, int slot, int lane, float* x) {
  const long long vec = (long long)head * C.page_size + slot;
  const unsigned char* p = pool + page * C.page_bytes;
  if (e4m3) {
    const float s = exp_value(exps[page * C.exp_bytes + vec]);
    if (PER == 4) {
      const float4 f = e4m3x4_float(*reinterpret_cast<const uint32_t*>(p + vec * C.D + lane * 4));
      x[0] = f.x * s, x[1] = f.y * s, x[PER - 2] = f.z * s, x[PER - 1] = f.w * s;
    } else {
      const float4 f = e4m3x4_float(*reinterpret_cast<const uint16_t*>(p + vec * C.D + lane * 2));
      x[0] = f.x * s, x[1] = f.y * s;
    }
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(p + (vec * C.D + lane * PER) * 2);
#pragma unroll
    for (int i = 0; i < PER / 2; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
  }
}

template <int D>
__global__ void __launch_bounds__(kAttendWarps * 32) attend_plain_kernel(const AttendArgs A, bool e4m3) {
  constexpr int PER = D / 32;
  const int token = blockIdx.x, hq = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __shared__ float sm_m[kAttendWarps], sm_l[kAttendWarps], sm_o[kAttendWarps][D];
  const int r = paged_row(A.C, token);
  if (r < 0) return;
  const int pos = A.C.kv_len[r] - (A.C.cu[r + 1] - token);
  const int head = hq / A.group;
  float q[PER], acc[PER], m = -INFINITY, l = 0.f;
  const uint32_t* qw = reinterpret_cast<const uint32_t*>(A.q + token * A.q_token + (long long)hq * D) + lane * PER / 2;
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) q[2 * i] = bf16_lo(qw[i]) * A.scale, q[2 * i + 1] = bf16_hi(qw[i]) * A.scale;
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  for (int j = warp; j <= pos; j += kAttendWarps) {
    int slot;
    const int page = paged_lookup(A.C, r, j, &slot);
    if (page < 0) {
      if (lane == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
      continue;
    }
    float x[PER], s = 0.f;
    load_vec<PER>(A.C.k, A.C.k_exp, A.C, e4m3, page, head, slot, lane, x);
#pragma unroll
    for (int i = 0; i < PER; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    load_vec<PER>(A.C.v, A.C.v_exp, A.C, e4m3, page, head, slot, lane, x);
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - base), p = expf(s - base);
    m = top;
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = acc[i] * keep + p * x[i];
  }
  if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
#pragma unroll
  for (int i = 0; i < PER; ++i) sm_o[warp][lane * PER + i] = acc[i];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
#pragma unroll
  for (int w = 0; w < kAttendWarps; ++w) top = fmaxf(top, sm_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int w = 0; w < kAttendWarps; ++w) total += sm_l[w] * expf(sm_m[w] - base);
  const long long row = (long long)token * A.hq + hq;
  for (int d = threadIdx.x; d < D; d += kAttendWarps * 32) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kAttendWarps; ++w) o += sm_o[w][d] * expf(sm_m[w] - base);
    if (total != 0.f) o /= total;
    A.out[row * D + d] = (uint16_t)pack_bf16(o, 0.f);
  }
  if (threadIdx.x == 0 && A.lse) A.lse[row] = total == 0.f ? -INFINITY : base + logf(total);
}

}  // namespace specv

extern "C" size_t spec_attend_workspace_size(int heads, int group, int head_dim) {
  if (heads < 1 || heads > 65535 || group < 1 || group > SPEC_MAX_GROUP || (head_dim != 64 && head_dim != 128)) return 0;
  return 256;
}

extern "C" int spec_attend(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens,
                           const spec_cache_t* cache, uint16_t* out, float* lse, uint32_t* flags, void* workspace,
                           size_t workspace_bytes, void* cuda_stream) {
  using namespace specv;
  AttendArgs A;
  const int rc = paged_check(cache, N, &A.C);
  if (rc != SPEC_OK) return rc;
  if (group < 1 || group > SPEC_MAX_GROUP || max_tokens < 0 || token_stride < 0) return SPEC_E_DIM;
  A.hq = A.C.heads * group;
  const long long dense = (long long)A.hq * A.C.D;
  if (A.hq > 65535 || (token_stride && token_stride < dense)) return SPEC_E_DIM;
  if (N == 0 || A.C.B == 0) return SPEC_OK;
  if (!q || !out || !workspace) return SPEC_E_NULL;
  A.q_token = token_stride ? token_stride : dense;
  if (!paged_aligned(q, 16) || !paged_aligned(out, 16) || A.q_token % 8 || (lse && !paged_aligned(lse, 4)) ||
      (flags && !paged_aligned(flags, 4)) || !paged_aligned(workspace, 256))
    return SPEC_E_ALIGN;
  if (workspace_bytes < spec_attend_workspace_size(A.C.heads, group, A.C.D)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  A.q = q;
  A.out = out;
  A.lse = lse;
  A.flags = flags;
  A.N = N;
  A.group = group;
  A.scale = scale;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const dim3 grid((unsigned)N, (unsigned)A.hq);
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  if (A.C.D == 128) attend_plain_kernel<128><<<grid, kAttendWarps * 32, 0, st>>>(A, e4m3);
  else attend_plain_kernel<64><<<grid, kAttendWarps * 32, 0, st>>>(A, e4m3);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}
