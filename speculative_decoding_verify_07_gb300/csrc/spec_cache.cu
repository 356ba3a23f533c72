// spec_cache_write and spec_cache_read: a token's keys and values into the
// paged cache, in 16 bits or quantised to 8, and back.
//
// A lane holds 8 consecutive elements of one head's vector, so D / 8 lanes
// hold the vector, a few shuffles find its largest magnitude, and the source
// is read once in 16-byte loads.  The scale is a power of two, 2^s with
// max|x| <= 448 * 2^s: x * 2^-s and c * 2^s are then exact, the one rounding
// is that to e4m3 (relative 2^-4, the same at every magnitude above 2^-6 of
// the code range, so the finest scale would gain nothing but sub-normal
// range), and what is read back is exact in bf16.  One exponent byte a
// vector costs 1/128 of an 8-bit cache.
//
// Both kernels are bound by memory (3 bytes an element for bf16 to e4m3).  A
// token's vectors, key and value of every head, take 2 * heads * D / 8 lanes; a
// thread keeps its place among them and takes U tokens, all of whose loads are
// begun before the first is used.  The tokens' places in the cache are looked up
// once a CTA, into shared memory, while the loads are in flight.  Measured, 8
// heads of 128, bf16 to e4m3: prompts of 25,000 tokens written at 4450 GB/s, 67 %
// of the copy bandwidth (issue slots 78 % busy: the conversion), 54,000 tokens
// read at 6020 GB/s (90 %), 64 rows of 3 tokens written in 4.1 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_host.h"
#include "spec_paged.cuh"

namespace specv {

constexpr int kCacheThreads = 256;

struct CacheIO {
  PagedCache C;
  unsigned char* kv[2];      // packed keys and values
  long long token_bytes;     // from one token to the next
  int N;
  int lanes;                 // of a token: 2 * heads * (D / 8)
  int across, at_once;       // of these, in a CTA; and tokens that it takes at a time
  uint32_t* flags;
};

// Where a token is in the cache.
struct TokenPlace {
  long long page;   // page index, or -1
  int slot;
  int row;
};

__device__ __forceinline__ TokenPlace find_place(const CacheIO& A, int token) {
  TokenPlace t;
  t.page = -1;
  t.slot = 0;
  t.row = paged_row(A.C, token);
  if (t.row < 0) return t;
  const int end = __ldg(A.C.cu + t.row + 1);
  const int pos = paged_kv_len(A.C, t.row) - (end - token);
  if (pos >= 0) t.page = paged_lookup(A.C, t.row, pos, &t.slot);
  if (t.page < 0 && A.flags) atomicOr(&A.flags[t.row], (uint32_t)SPEC_F_BAD_IDX);
  return t;
}

// A thread's place among a token's lanes, and its first token.
struct Place {
  int token, head, kv, lane;
  bool live;
};

template <int LPV, int U>
__device__ __forceinline__ Place thread_place(const CacheIO& A, TokenPlace* places) {
  const int first = blockIdx.x * U * A.at_once, count = min(U * A.at_once, A.N - first);
  for (int t = threadIdx.x; t < count; t += kCacheThreads) places[t] = find_place(A, first + t);
  Place p;
  const int turn = threadIdx.x / A.across, w = blockIdx.y * kCacheThreads + threadIdx.x - turn * A.across;
  p.live = turn < A.at_once && w < A.lanes;
  p.token = first + turn;
  p.lane = w % LPV;
  const int vec = w / LPV;
  p.kv = vec >= A.C.heads;
  p.head = vec - (p.kv ? A.C.heads : 0);
  return p;
}

template <bool F32, bool E4M3, int LPV, int U>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheIO A) {
  __shared__ TokenPlace places[kCacheThreads * U / (2 * LPV)];
  const Place P = thread_place<LPV, U>(A, places);
  const unsigned char* from = A.kv[P.kv] + P.token * A.token_bytes + ((long long)P.head * LPV + P.lane) * (F32 ? 32 : 16);
  const long long step = A.at_once * A.token_bytes;
  uint4 raw[U][F32 ? 2 : 1];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int w = 0; w < (F32 ? 2 : 1); ++w) {
      raw[u][w] = make_uint4(0, 0, 0, 0);
      if (P.live && P.token + u * A.at_once < A.N) raw[u][w] = __ldcs(reinterpret_cast<const uint4*>(from + u * step) + w);
    }
  __syncthreads();
  const int turn = P.token - blockIdx.x * U * A.at_once;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the largest magnitude as bits: NaN above infinity above every number
    uint32_t amax;
    if (F32) {
      const uint4 a = raw[u][0], b = raw[u][F32 ? 1 : 0];
      constexpr uint32_t m = 0x7fffffffu;
      amax = max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)), max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
#pragma unroll
      for (int o = LPV / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    } else {
      const uint4 a = raw[u][0];
      constexpr uint32_t m = 0x7fff7fffu;
      uint32_t two = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
#pragma unroll
      for (int o = LPV / 2; o; o >>= 1) two = __vmaxu2(two, __shfl_xor_sync(0xffffffffu, two, o));
      amax = max(two << 16, two & 0xffff0000u);
    }
    if (!P.live || P.token + u * A.at_once >= A.N) continue;
    const TokenPlace at = places[turn + u * A.at_once];
    if (P.lane == 0 && amax >= 0x7f800000u && A.flags && at.row >= 0) atomicOr(&A.flags[at.row], (uint32_t)SPEC_F_NAN);
    if (at.page < 0) continue;
    const long long vec = (long long)P.head * A.C.page_size + at.slot;
    unsigned char* const pool = (P.kv ? A.C.v : A.C.k) + at.page * A.C.page_bytes;
    float x[8];
    if (F32) {
      const uint4 a = raw[u][0], b = raw[u][F32 ? 1 : 0];
      x[0] = __uint_as_float(a.x), x[1] = __uint_as_float(a.y), x[2] = __uint_as_float(a.z), x[3] = __uint_as_float(a.w);
      x[4] = __uint_as_float(b.x), x[5] = __uint_as_float(b.y), x[6] = __uint_as_float(b.z), x[7] = __uint_as_float(b.w);
    } else {
      const uint4 a = raw[u][0];
      x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
      x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
    }
    if (!E4M3) {
      uint4 w = raw[u][0];
      if (F32)
        w = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
      *reinterpret_cast<uint4*>(pool + (vec * LPV + P.lane) * 16) = w;
    } else {
      // amax = 1.f * 2^E; 448 = 1.75 * 2^8
      const int s = max((int)(amax >> 23) - 127 - 8 + ((amax & 0x7fffffu) > 0x600000u), -126);
      const bool bad = amax >= 0x7f800000u;
      const float inv = __uint_as_float((uint32_t)(127 - s) << 23);
      uint16_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[e]) : "f"(x[2 * e + 1] * inv), "f"(x[2 * e] * inv));
      const uint2 codes = make_uint2((uint32_t)h[0] | (uint32_t)h[1] << 16, (uint32_t)h[2] | (uint32_t)h[3] << 16);
      *reinterpret_cast<uint2*>(pool + (vec * LPV + P.lane) * 8) = bad ? make_uint2(0, 0) : codes;
      if (P.lane == 0) (P.kv ? A.C.v_exp : A.C.k_exp)[at.page * A.C.exp_bytes + vec] = (uint8_t)(bad ? 255 : s + 127);
    }
  }
}

template <bool E4M3, int LPV, int U>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheIO A) {
  __shared__ TokenPlace places[kCacheThreads * U / (2 * LPV)];
  const Place P = thread_place<LPV, U>(A, places);
  __syncthreads();
  const int turn = P.token - blockIdx.x * U * A.at_once;
  uint4 raw[U];
  uint32_t e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    e[u] = 127;
    if (!P.live || P.token + u * A.at_once >= A.N) continue;
    const TokenPlace at = places[turn + u * A.at_once];
    if (at.page < 0) continue;
    const long long vec = (long long)P.head * A.C.page_size + at.slot;
    const unsigned char* p = (P.kv ? A.C.v : A.C.k) + at.page * A.C.page_bytes;
    if (E4M3) {
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(p + (vec * LPV + P.lane) * 8));
      raw[u].x = w.x;
      raw[u].y = w.y;
      e[u] = __ldg((P.kv ? A.C.v_exp : A.C.k_exp) + at.page * A.C.exp_bytes + vec);
    } else {
      raw[u] = __ldcs(reinterpret_cast<const uint4*>(p + (vec * LPV + P.lane) * 16));
    }
  }
  unsigned char* const to = A.kv[P.kv] + P.token * A.token_bytes + ((long long)P.head * LPV + P.lane) * 16;
  const long long step = A.at_once * A.token_bytes;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!P.live || P.token + u * A.at_once >= A.N) continue;
    uint4 w = raw[u];
    if (E4M3) {
      const float s = exp_value(e[u]);
      const float4 a = e4m3x4_float(raw[u].x), b = e4m3x4_float(raw[u].y);
      w = make_uint4(pack_bf16(a.x * s, a.y * s), pack_bf16(a.z * s, a.w * s), pack_bf16(b.x * s, b.y * s),
                     pack_bf16(b.z * s, b.w * s));
    }
    __stcs(reinterpret_cast<uint4*>(to + u * step), w);
  }
}

template <int LPV, int U>
static void launch_write(const CacheIO& A, bool f32, bool e4m3, cudaStream_t st) {
  const dim3 grid((A.N + U * A.at_once - 1) / (U * A.at_once), (A.lanes + kCacheThreads - 1) / kCacheThreads);
  if (f32) {
    if (e4m3) cache_write_kernel<true, true, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
    else cache_write_kernel<true, false, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
  } else {
    if (e4m3) cache_write_kernel<false, true, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
    else cache_write_kernel<false, false, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
  }
}

template <int LPV, int U>
static void launch_read(const CacheIO& A, bool e4m3, cudaStream_t st) {
  const dim3 grid((A.N + U * A.at_once - 1) / (U * A.at_once), (A.lanes + kCacheThreads - 1) / kCacheThreads);
  if (e4m3) cache_read_kernel<true, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
  else cache_read_kernel<false, LPV, U><<<grid, kCacheThreads, 0, st>>>(A);
}

static int cache_launch(bool write, void* k, void* v, int dtype, long long token_stride, int N, const spec_cache_t* cache,
                        uint32_t* flags, void* cuda_stream) {
  CacheIO A;
  const int rc = paged_check(cache, N, &A.C);
  if (rc != SPEC_OK) return rc;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_E_DTYPE;
  if (token_stride < 0) return SPEC_E_DIM;
  const int es = dtype == SPEC_F32 ? 4 : 2;
  const long long dense = (long long)A.C.heads * A.C.D;
  if (token_stride && token_stride < dense) return SPEC_E_DIM;
  if (N == 0 || A.C.B == 0) return SPEC_OK;
  if (!k || !v) return SPEC_E_NULL;
  A.token_bytes = (token_stride ? token_stride : dense) * es;
  if (!paged_aligned(k, 16) || !paged_aligned(v, 16) || A.token_bytes % 16 || (flags && !paged_aligned(flags, 4)))
    return SPEC_E_ALIGN;
  const int lpv = A.C.D / 8;
  A.lanes = 2 * A.C.heads * lpv;
  A.across = A.lanes < kCacheThreads ? A.lanes : kCacheThreads;
  A.at_once = kCacheThreads / A.across;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  A.kv[0] = static_cast<unsigned char*>(k);
  A.kv[1] = static_cast<unsigned char*>(v);
  A.N = N;
  A.flags = flags;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const bool e4m3 = cache->dtype == SPEC_E4M3, f32 = dtype == SPEC_F32;
  // Four tokens a thread keep four loads in flight (the long prompts 31.5 us, with one 46.1; 1500 tokens 4.9 and
  // 5.2); one where four would leave SMs without two CTAs (500 tokens 3.6 us, with four 4.1).
  const bool many = (long long)N * A.lanes >= 2LL * 152 * kCacheThreads * 4;
  if (write) {
    if (lpv == 16) many ? launch_write<16, 4>(A, f32, e4m3, st) : launch_write<16, 1>(A, f32, e4m3, st);
    else many ? launch_write<8, 4>(A, f32, e4m3, st) : launch_write<8, 1>(A, f32, e4m3, st);
  } else {
    if (lpv == 16) many ? launch_read<16, 4>(A, e4m3, st) : launch_read<16, 1>(A, e4m3, st);
    else many ? launch_read<8, 4>(A, e4m3, st) : launch_read<8, 1>(A, e4m3, st);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

}  // namespace specv

extern "C" int spec_cache_write(const void* k, const void* v, int dtype, int64_t token_stride, int N,
                                const spec_cache_t* cache, uint32_t* flags, void* cuda_stream) {
  return specv::cache_launch(true, const_cast<void*>(k), const_cast<void*>(v), dtype, token_stride, N, cache, flags,
                             cuda_stream);
}

extern "C" int spec_cache_read(uint16_t* k, uint16_t* v, int N, const spec_cache_t* cache, uint32_t* flags,
                               void* cuda_stream) {
  return specv::cache_launch(false, k, v, SPEC_BF16, 0, N, cache, flags, cuda_stream);
}
