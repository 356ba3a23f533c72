// The paged cache as kernels see it: argument checks, page lookup, e4m3 values, and the arithmetic the forward shares.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_device.cuh"

namespace specv {

struct PagedCache {
  unsigned char* k;
  unsigned char* v;
  uint8_t* k_exp;
  uint8_t* v_exp;
  const int32_t* table;
  const int32_t* cu;
  const int32_t* kv_len;
  long long page_bytes;   // from one page to the next
  long long exp_bytes;
  int B, max_pages, pages, heads, page_size, D;
  int page_shift;         // log2(page_size), or -1
};

inline bool paged_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Checks a spec_cache_t and lays it out for a kernel.  Enqueues nothing.
inline int paged_check(const spec_cache_t* c, int N, PagedCache* out) {
  if (!c) return SPEC_E_NULL;
  if (N < 0 || c->B < 0 || c->max_pages < 0 || c->pages < 0 || c->heads < 1 || c->heads > 65535) return SPEC_E_DIM;
  if (c->page_size < 1 || c->page_size > SPEC_MAX_PAGE) return SPEC_E_DIM;
  if (c->head_dim != 64 && c->head_dim != 128) return SPEC_E_DIM;
  // (the ends of the tiles that positions are counted in are held in 32 bits too)
  if ((long long)c->max_pages * c->page_size > SPEC_MAX_LENGTH) return SPEC_E_DIM;
  if (c->dtype != SPEC_BF16 && c->dtype != SPEC_E4M3) return SPEC_E_DTYPE;
  const bool e4m3 = c->dtype == SPEC_E4M3;
  const int es = e4m3 ? 1 : 2;
  const long long dense = (long long)c->heads * c->page_size * c->head_dim;
  const long long edense = (long long)c->heads * c->page_size;
  if (c->page_stride < 0 || (c->page_stride && c->page_stride < dense)) return SPEC_E_DIM;
  if (e4m3 && (c->exp_stride < 0 || (c->exp_stride && c->exp_stride < edense))) return SPEC_E_DIM;
  if (N > 0 && c->B > 0) {
    if (!c->cu_tokens || !c->kv_len) return SPEC_E_NULL;
    if (c->max_pages > 0 && !c->page_table) return SPEC_E_NULL;
    if (c->pages > 0 && (!c->k_pages || !c->v_pages || (e4m3 && (!c->k_exp || !c->v_exp)))) return SPEC_E_NULL;
    if (!paged_aligned(c->cu_tokens, 4) || !paged_aligned(c->kv_len, 4) || !paged_aligned(c->page_table, 4))
      return SPEC_E_ALIGN;
    if (!paged_aligned(c->k_pages, 16) || !paged_aligned(c->v_pages, 16) || (c->page_stride * es) % 16)
      return SPEC_E_ALIGN;
  }
  out->k = static_cast<unsigned char*>(c->k_pages);
  out->v = static_cast<unsigned char*>(c->v_pages);
  out->k_exp = c->k_exp;
  out->v_exp = c->v_exp;
  out->table = c->page_table;
  out->cu = c->cu_tokens;
  out->kv_len = c->kv_len;
  out->page_bytes = (c->page_stride ? c->page_stride : dense) * es;
  out->exp_bytes = c->exp_stride ? c->exp_stride : edense;
  out->B = c->B;
  out->max_pages = c->max_pages;
  out->pages = c->pages;
  out->heads = c->heads;
  out->page_size = c->page_size;
  out->D = c->head_dim;
  out->page_shift = -1;
  for (int s = 0; s < 13; ++s)
    if (c->page_size == 1 << s) out->page_shift = s;
  return SPEC_OK;
}

__device__ __forceinline__ int paged_index(const PagedCache& C, int pos) {
  return C.page_shift >= 0 ? pos >> C.page_shift : pos / C.page_size;
}

// What row r has cached.  A negative number places no token, as zero does, and
// taking tokens from the lowest would pass 32 bits.
__device__ __forceinline__ int paged_kv_len(const PagedCache& C, int r) { return max(__ldg(C.kv_len + r), 0); }

// The page of position pos >= 0 of row r, or -1 where there is none.
__device__ __forceinline__ int paged_lookup(const PagedCache& C, int r, int pos, int* slot) {
  const int i = paged_index(C, pos);
  *slot = pos - i * C.page_size;
  if (i >= C.max_pages) return -1;
  const int page = __ldg(C.table + (long long)r * C.max_pages + i);
  return page >= 0 && page < C.pages ? page : -1;
}

// The same in two steps, so that the table's entry can be on its way meanwhile:
// the entry as it stands (-1 beyond the table), and the page that it names or -1.
__device__ __forceinline__ int paged_entry(const PagedCache& C, int r, int pos, int* slot) {
  const int i = paged_index(C, pos);
  *slot = pos - i * C.page_size;
  return i < C.max_pages ? __ldg(C.table + (long long)r * C.max_pages + i) : -1;
}
__device__ __forceinline__ int paged_page(const PagedCache& C, int entry) {
  return entry >= 0 && entry < C.pages ? entry : -1;
}

// The row whose new tokens hold `token`, or -1: the last r with cu[r] <= token.
__device__ __forceinline__ int paged_row(const PagedCache& C, int token) {
  int lo = 0, hi = C.B;   // cu[lo] <= token < cu[hi] once the ends are checked
  if (token < __ldg(C.cu) || token >= __ldg(C.cu + C.B)) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(C.cu + mid) <= token) lo = mid; else hi = mid;
  }
  return lo;
}

// 2^(e - 127) for an exponent byte, NaN for 255 (bytes 0 and 1 both give 2^-126).
__device__ __forceinline__ float exp_value(uint32_t e) {
  return __uint_as_float(e >= 255u ? 0x7fc00000u : (e < 1u ? 1u : e) << 23);
}

// Two pairs of e4m3 codes as fp16.
__device__ __forceinline__ void e4m3_f16(uint32_t w, uint32_t* lo, uint32_t* hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(*lo), "=r"(*hi) : "r"(w));
}

// Four e4m3 codes as floats (exact).
__device__ __forceinline__ float4 e4m3x4_float(uint32_t w) {
  uint32_t lo, hi;
  e4m3_f16(w, &lo, &hi);
  float4 f;
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
      : "=f"(f.x), "=f"(f.y) : "r"(lo));
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.f32.f16 %0, a;\ncvt.f32.f16 %1, b;\n}"
      : "=f"(f.z), "=f"(f.w) : "r"(hi));
  return f;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)), "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 both_of(float x) { return make_float2(x, x); }

}  // namespace specv
