// spec_recur: h_t = exp(g_t) h_{t-1} + x_t, channel by channel, and its backward
// pass, the same recurrence from the last token to the first.
//
// Bound by memory (g, x, h once; backward g, h, dh, dx, dg).  A few tokens: a
// thread walks its channels' tokens.  More: a step s -> a s + b is joined with the
// next as (a2 a1, a2 b1 + b2), so tiles of tokens are reduced to one such pair,
// the pairs are handed along the row, and each tile is walked from the state that
// enters it.  Every sum is taken in the same order on every call.
//
// Measured: 1x65536x2048 bf16 184 us, 4380 GB/s (65 % of the copy bandwidth; issue
// slots are busy in 65 % of the cycles, the barriers of a tile and the chain along
// the row take the rest), its backward pass 267 us, 5030 GB/s (75 %); 8x4096x1024
// float32 5030 and 5350 GB/s; 64x3x4096 3.6 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_host.h"
#include "spec_paged.cuh"
#include "spec_tma.cuh"

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

// A row's length, its initial state's place (-1: zeros) and that of its last
// state (-1: none); false where a slot is out of range (d_state, by row, is
// zero there: the state has no part in the row's results).
template <bool BWD>
__device__ __forceinline__ bool recur_row(const RecurArgs& A, int r, int* len, long long* from, long long* to) {
  *len = A.lens ? min(max(A.lens[r], 0), A.T) : A.T;
  const int s = A.slot ? A.slot[r] : r, o = A.last_slot ? A.last_slot[r] : r;
  const bool ok = (!A.state || (s >= 0 && s < A.slots)) && (!A.last || (o >= 0 && o < A.last_slots));
  *from = A.state && ok ? (long long)s * A.D : -1;
  *to = A.last && (ok || BWD) ? (long long)(BWD ? r : o) * A.D : -1;
  return ok;
}

// VEC neighbouring channels of one token as they are in memory.
template <bool BF16, int VEC>
struct Channels {
  static constexpr int kBytes = VEC * (BF16 ? 2 : 4);
  uint32_t w[kBytes < 4 ? 1 : kBytes / 4];

  __device__ __forceinline__ void load(const unsigned char* p) {
    if (kBytes == 16) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p));
      w[0] = x.x, w[kBytes / 16] = x.y, w[kBytes / 8] = x.z, w[kBytes / 16 * 3] = x.w;
    } else if (kBytes == 8) {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(p));
      w[0] = x.x, w[kBytes / 8] = x.y;
    } else if (kBytes == 4) {
      w[0] = __ldcs(reinterpret_cast<const uint32_t*>(p));
    } else {
      w[0] = __ldcs(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ float get(int v) const {
    if (!BF16) return __uint_as_float(w[v]);
    return v % 2 ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
  }
  static __device__ __forceinline__ void store(unsigned char* p, const float* x) {
    uint32_t w[kBytes < 4 ? 1 : kBytes / 4];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (!BF16) w[v] = __float_as_uint(x[v]);
      else if (v % 2 == 0) w[v / 2] = pack_bf16(x[v], v + 1 < VEC ? x[v + 1 < VEC ? v + 1 : v] : 0.f);
    }
    if (kBytes == 16) {
      __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[kBytes / 16], w[kBytes / 8], w[kBytes / 16 * 3]));
    } else if (kBytes == 8) {
      __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[kBytes / 8]));
    } else if (kBytes == 4) {
      __stcs(reinterpret_cast<uint32_t*>(p), w[0]);
    } else {
      __stcs(reinterpret_cast<uint16_t*>(p), (uint16_t)w[0]);
    }
  }
};

// exp(g).  An error of the decay adds up over the tokens that the state
// remembers, 1 / (1 - exp(g)) of them, and that of ex2.approx leans to one side
// (by 2.5e-8 in the mean near 1, measured; over 400 tokens that is 1e-5).  So
// below |g| = 1/32 the series to g^3 is taken instead (mean 1e-10 up to 0.01,
// 1e-8 at the border); further out little is remembered.
__device__ __forceinline__ float decay(float g) {
  float a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(g * 1.4426950408889634f));
  const float near = fmaf(fmaf(fmaf(g, 1.f / 6.f, 0.5f), g, 1.f), g, 1.f);
  return fabsf(g) < 0.03125f ? near : a;
}

// decay() of two channels.
__device__ __forceinline__ float2 decay2(float2 g) {
  const float2 y = mul2(g, both_of(1.4426950408889634f));
  float2 a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(y.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(y.y));
  const float2 near = fma2(fma2(fma2(g, both_of(1.f / 6.f), both_of(0.5f)), g, both_of(1.f)), g, both_of(1.f));
  return make_float2(fabsf(g.x) < 0.03125f ? near.x : a.x, fabsf(g.y) < 0.03125f ? near.y : a.y);
}

// ---------------------------------------------------------------- few tokens

constexpr int kStepThreads = 256;
constexpr int kStepAhead = 4;     // tokens loaded ahead of the state's chain

template <bool BF16, bool HBF16, int VEC, bool BWD>
__global__ void __launch_bounds__(kStepThreads) recur_step_kernel(const RecurArgs A) {
  using In = Channels<BF16, VEC>;
  using H = Channels<HBF16, VEC>;
  using Out = Channels<BWD ? BF16 : HBF16, VEC>;
  constexpr int es = BF16 ? 2 : 4, hs = HBF16 ? 2 : 4, os = BWD ? es : hs;
  const int r = blockIdx.y, c = (blockIdx.x * kStepThreads + threadIdx.x) * VEC;
  if (c >= A.D) return;
  int len;
  long long from, to;
  const bool ok = recur_row<BWD>(A, r, &len, &from, &to);
  if (!ok) {
    if (c == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
    len = 0;
  }
  const long long base = (long long)r * A.T * A.D + c, gbase = r * A.g_row + c, xbase = BWD ? base : r * A.x_row + c;
  const long long x_tok = BWD ? A.D : A.x_tok;
  float first[VEC], s[VEC], zero[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    first[v] = from >= 0 ? A.state[from + c + v] : 0.f;
    s[v] = BWD ? (A.d_last && ok ? A.d_last[(long long)r * A.D + c + v] : 0.f) : first[v];
    zero[v] = 0.f;
  }
  for (int t = len; t < A.T; ++t) {
    Out::store(A.h + (base + (long long)t * A.D) * os, zero);
    if (BWD) In::store(A.dg + (base + (long long)t * A.D) * es, zero);
  }
  for (int t0 = 0; t0 < len; t0 += kStepAhead) {
    In g[kStepAhead], x[kStepAhead];
    H hb[BWD ? kStepAhead : 1];
#pragma unroll
    for (int i = 0; i < kStepAhead; ++i) {
      const int n = min(t0 + i, len - 1), t = BWD ? len - 1 - n : n;
      g[i].load(A.g + (gbase + t * A.g_tok) * es);
      x[i].load(A.x + (xbase + t * x_tok) * es);
      if (BWD && t) hb[BWD ? i : 0].load(A.hin + (base + (long long)(t - 1) * A.D) * hs);
    }
#pragma unroll
    for (int i = 0; i < kStepAhead; ++i) {
      if (t0 + i >= len) break;
      const int t = BWD ? len - 1 - t0 - i : t0 + i;
      float out[VEC], dg[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float a = decay(g[i].get(v));
        if (BWD) {
          out[v] = x[i].get(v) + s[v];
          s[v] = a * out[v];
          dg[v] = s[v] * (t ? hb[BWD ? i : 0].get(v) : first[v]);
        } else {
          out[v] = s[v] = fmaf(a, s[v], x[i].get(v));
        }
      }
      Out::store(A.h + (base + (long long)t * A.D) * os, out);
      if (BWD) In::store(A.dg + (base + (long long)t * A.D) * es, dg);
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v)
    if (to >= 0) A.last[to + c + v] = s[v];
}

// ---------------------------------------------------------------- many tokens

// Workspace: a header, then for each (tile, row, channel) the two words of its
// aggregate, then one of the state behind it.
struct ScanHeader {
  unsigned ticket, done, epoch, pad[61];
};

using Word = unsigned long long;   // the call's tag above a float: one access is whole

__device__ __forceinline__ Word tagged(float x, unsigned tag) { return (Word)tag << 32 | __float_as_uint(x); }
__device__ __forceinline__ void put_word(Word* p, Word w) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(w) : "memory");
}
__device__ __forceinline__ Word get_word(const Word* p) {
  Word w;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(w) : "l"(p) : "memory");
  return w;
}

constexpr int kScanWarps = 8;        // at most, one behind the other in time
constexpr int kScanCh = 64;          // channels of a tile, two a lane
constexpr int kScanGroupMost = 32;
constexpr int kScanSpins = 1 << 20;  // about a second of polling

// Tokens of a warp: a tile is 16 KB a tensor.
template <bool BF16>
constexpr int scan_steps() { return BF16 ? 16 : 8; }

// Waits for N words under the tag and returns their floats; zeros (and
// *gave_up) where they do not come.
template <int N>
__device__ __forceinline__ void await_words(const Word* p, unsigned tag, float* x, bool* gave_up) {
#pragma unroll
  for (int n = 0; n < N; ++n) x[n] = 0.f;
  for (int i = 0; i < kScanSpins && !*gave_up; ++i) {
    Word w[N];
    bool all = true;
#pragma unroll
    for (int n = 0; n < N; ++n) w[n] = get_word(p + n);
#pragma unroll
    for (int n = 0; n < N; ++n) all = all && (unsigned)(w[n] >> 32) == tag;
    if (all) {
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] = __uint_as_float((unsigned)w[n]);
      return;
    }
  }
  *gave_up = true;
}

// Two neighbouring channels in shared memory.
template <bool BF16>
__device__ __forceinline__ float2 lds_pair(uint32_t p) {
  if (BF16) {
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(p) : "memory");
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
  float2 x;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "r"(p) : "memory");
  return x;
}

// Two neighbouring channels of global memory, the second where `both`; PAIR: as one access.
template <bool BF16, bool PAIR>
__device__ __forceinline__ void store_pair(unsigned char* p, float2 x, bool both) {
  if (PAIR) {
    if (BF16) __stcs(reinterpret_cast<uint32_t*>(p), pack_bf16(x.x, x.y));
    else __stcs(reinterpret_cast<float2*>(p), x);
  } else if (BF16) {
    __stcs(reinterpret_cast<uint16_t*>(p), (uint16_t)pack_bf16(x.x, 0.f));
    if (both) __stcs(reinterpret_cast<uint16_t*>(p) + 1, (uint16_t)pack_bf16(x.y, 0.f));
  } else {
    __stcs(reinterpret_cast<float*>(p), x.x);
    if (both) __stcs(reinterpret_cast<float*>(p) + 1, x.y);
  }
}

// Fills a warp's rows of a tile from memory that TMA cannot read: by 4-byte copies
// that need no registers on the way, or, where 16-bit rows do not begin at 4-byte
// boundaries, element by element.  `p` is the first row's channel c0 of the tile,
// `left` the channels from there to D.
template <bool BF16>
__device__ __forceinline__ void fill_rows(unsigned char* to, const unsigned char* p, long long tok_bytes, int rows, int left) {
  constexpr int es = BF16 ? 2 : 4, row_bytes = kScanCh * es;
  const int lane = threadIdx.x % 32;
  if (!BF16 || (((uintptr_t)p | tok_bytes) & 3) == 0) {
#pragma unroll 4
    for (int i = 0; i < rows; ++i)
#pragma unroll
      for (int w = 0; w < row_bytes / 128; ++w) {
        const int c = (w * 32 + lane) * (4 / es);
        const unsigned char* g = p + i * tok_bytes;
        const int bytes = min(max(left - c, 0) * es, 4);          // (the rest of the word becomes zero)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(to + i * row_bytes + w * 128 + lane * 4)),
                     "l"(bytes ? g + c * es : g), "r"(bytes) : "memory");
      }
  } else {
    const int c = 2 * lane;
#pragma unroll 4
    for (int i = 0; i < rows; ++i) {
      const uint16_t* g = reinterpret_cast<const uint16_t*>(p + i * tok_bytes) + c;
      uint16_t x = 0, y = 0;
      if (c < left) x = __ldcs(g);
      if (c + 1 < left) y = __ldcs(g + 1);
      *reinterpret_cast<uint32_t*>(to + i * row_bytes + lane * 4) = (uint32_t)x | (uint32_t)y << 16;
    }
  }
}

struct ScanMaps {
  CUtensorMap g, x, h;      // backward: g, dh, h
};

// A CTA takes a tile of 64 channels x (warps * S tokens) of a row.  Tiles go by
// tickets, all channels of all rows before the next tokens, and a tile waits only
// for tiles of smaller tickets, whose CTAs have begun.
//
// The tile comes by TMA, past the load queue through which the small loads of
// the chain have to go.  Its tokens are read twice from shared memory, once to
// reduce them and once, when the state that enters is known, to walk them; the
// decay is computed both times, which leaves registers for four CTAs an SM (five
// forward: with four 10 % slower), and their loads and chain steps hide one another.
// Rows that do not begin at 16-byte boundaries are copied word by word (4x8192x1337
// float32 149 us forward, 3530 GB/s; 8x4096x1024 by TMA 5030 GB/s, by words 3400).
template <bool BF16, bool HBF16, bool BWD, bool TMA>
__global__ void __launch_bounds__(kScanWarps * 32, (TMA && !BWD ? 5 : 4)) recur_scan_kernel(const RecurArgs A, const __grid_constant__ ScanMaps maps,
                                                                         ScanHeader* W, Word* agg, Word* inc, int tiles, int blocks,
                                                                         int group) {
  constexpr int S = scan_steps<BF16>();
  constexpr int es = BF16 ? 2 : 4, hs = HBF16 ? 2 : 4, os = BWD ? es : hs, row_bytes = kScanCh * es, h_row = kScanCh * hs;
  extern __shared__ __align__(128) unsigned char staged[];       // g, x or dh, and for the gradients h, [token][channel]
  __shared__ float2 sm_a[kScanWarps][32], sm_b[kScanWarps][32], sm_in[32], sm_pa[kScanWarps][32], sm_pb[kScanWarps][32];
  __shared__ __align__(8) unsigned long long full;
  __shared__ unsigned sm_ticket, sm_tag;
  __shared__ int failed;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32, span = warps * S;
  if (threadIdx.x == 0) {
    sm_ticket = tiles > 1 ? atomicAdd(&W->ticket, 1u) : blockIdx.x;
    sm_tag = *(volatile unsigned*)&W->epoch + 1;
    failed = 0;
    if (TMA) {
      mbar_init(&full, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  }
  __syncthreads();
  const unsigned tag = sm_tag, ticket = sm_ticket;
  const unsigned per = (unsigned)A.B * (unsigned)blocks, nth = ticket / per, rest = ticket - nth * per, row = rest / (unsigned)blocks;
  const int r = (int)row, tile = BWD ? tiles - 1 - (int)nth : (int)nth, c0 = (int)(rest - row * (unsigned)blocks) * kScanCh;
  const int c = c0 + 2 * lane;
  const bool live = c < A.D, both = c + 1 < A.D;
  int len;
  long long from, to;
  const bool ok = recur_row<BWD>(A, r, &len, &from, &to);
  if (!ok) len = 0;
  if (!ok && tile == 0 && c == 0 && warp == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
  const int used = (len + span - 1) / span;                    // tiles of this row that hold tokens
  const int order = BWD ? used - 1 - tile : tile;              // this tile's place among them
  const int t0 = tile * span + warp * S;
  const long long base = ((long long)r * A.T + t0) * A.D + c;
  unsigned char* const out_p = A.h + base * os;
  unsigned char* const dg_p = BWD ? A.dg + base * es : nullptr;
  const long long out_tok = (long long)A.D * os, dg_tok = (long long)A.D * es;

  if (tile >= used) {
    // nothing but zeros here; a row without tokens hands its state on
    if (live) {
      for (int i = 0; i < S && t0 + i < A.T; ++i) {
        store_pair<BWD ? BF16 : HBF16, TMA>(out_p + i * out_tok, make_float2(0.f, 0.f), both);
        if (BWD) store_pair<BF16, TMA>(dg_p + i * dg_tok, make_float2(0.f, 0.f), both);
      }
      if (tile == 0 && warp == 0 && to >= 0)
        for (int v = 0; v < 1 + both; ++v)
          A.last[to + c + v] = BWD ? (A.d_last && ok ? A.d_last[(long long)r * A.D + c + v] : 0.f) : (from >= 0 ? A.state[from + c + v] : 0.f);
    }
  } else {
    unsigned char* const sm_x = staged + span * row_bytes;
    unsigned char* const sm_h = sm_x + span * row_bytes;
    if (TMA) {
      if (threadIdx.x == 0) {
        mbar_arrive_expect_tx(&full, span * (2 * row_bytes + (BWD ? h_row : 0)));
        tma_load_3d(smem_u32(staged), &maps.g, c0, tile * span, r, &full);
        tma_load_3d(smem_u32(sm_x), &maps.x, c0, tile * span, r, &full);
        if (BWD) tma_load_3d(smem_u32(sm_h), &maps.h, c0, tile * span - 1, r, &full);     // the states before
      }
    } else {
      const long long g_tok = A.g_tok * es, x_tok = (BWD ? (long long)A.D : A.x_tok) * es, h_tok = (long long)A.D * hs;
      const int rows = max(0, min(S, len - t0)), left = A.D - c0;
      const long long first = base - 2 * lane;                   // of channel c0
      fill_rows<BF16>(staged + warp * S * row_bytes, A.g + (r * A.g_row + c0) * es + t0 * g_tok, g_tok, rows, left);
      fill_rows<BF16>(sm_x + warp * S * row_bytes, A.x + (BWD ? first * es : (r * A.x_row + c0) * es + t0 * x_tok), x_tok, rows, left);
      if (BWD) {
        const int skip = t0 == 0;      // (before the first token there is the state)
        fill_rows<HBF16>(sm_h + (warp * S + skip) * h_row, A.hin + (first + (long long)(skip - 1) * A.D) * hs, h_tok, max(0, rows - skip), left);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
    const bool whole = t0 + S <= len;
    const uint32_t at_g = smem_u32(staged) + (warp * S * kScanCh + 2 * lane) * es, at_x = smem_u32(sm_x) + (warp * S * kScanCh + 2 * lane) * es;
    const uint32_t at_h = smem_u32(sm_h) + (warp * S * kScanCh + 2 * lane) * hs;
    if (TMA) mbar_await(&full, 0, &failed);
    // this warp's steps as one: s -> pa s + pb (a token beyond the row: s -> s)
    float2 pa = both_of(1.f), pb = both_of(0.f);
    auto reduce = [&](int n) {
      const float2 a = decay2(lds_pair<BF16>(at_g + n * row_bytes)), x = lds_pair<BF16>(at_x + n * row_bytes);
      pb = BWD ? mul2(a, add2(x, pb)) : fma2(a, pb, x);
      pa = mul2(pa, a);
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < S; ++i) reduce(BWD ? S - 1 - i : i);
    } else {
      const int rows = max(0, min(S, len - t0));
#pragma unroll 1
      for (int i = 0; i < rows; ++i) reduce(BWD ? rows - 1 - i : i);
    }
    sm_a[warp][lane] = pa;
    sm_b[warp][lane] = pb;
    __syncthreads();
    const int ahead = order % group;                             // tiles of this group that come first
    const bool ends = ahead == group - 1, hands_on = order < used - 1;
    const bool publishes = warp == (BWD ? 0 : warps - 1);        // the last in order
    const long long mine = ((long long)tile * A.B + r) * (blocks * kScanCh) + c;
    const long long back = (BWD ? 1LL : -1LL) * A.B * (blocks * kScanCh);       // to the tile before in order
    // what comes before this warp in the tile, and in the warp that publishes it the whole tile
    float2 fa = make_float2(1.f, 1.f), fb = make_float2(0.f, 0.f);
    for (int w = 0; w < (BWD ? warps - 1 - warp : warp); ++w) {
      const int n = BWD ? warps - 1 - w : w;
      const float2 wa = sm_a[n][lane], wb = sm_b[n][lane];
      fb = make_float2(fmaf(wa.x, fb.x, wb.x), fmaf(wa.y, fb.y, wb.y));
      fa = make_float2(fa.x * wa.x, fa.y * wa.y);
    }
    const float2 ta = make_float2(fa.x * pa.x, fa.y * pa.y), tb = make_float2(fmaf(pa.x, fb.x, pb.x), fmaf(pa.y, fb.y, pb.y));
    // The state that enters the row is read by its first tile alone, which hands on what is behind it: `last` may be the
    // same memory, and the tile that writes it has waited, through the tiles between, for words made of that read.
    float2 s = make_float2(0.f, 0.f);
    if (publishes && order == 0 && live) {
      const float* p = BWD ? (A.d_last ? A.d_last + (long long)r * A.D : nullptr) : from >= 0 ? A.state + from : nullptr;
      if (p) s = make_float2(p[c], both ? p[c + 1] : 0.f);
    }
    if (publishes && hands_on && !ends) {
      const bool start = order == 0;
      put_word(agg + mine * 2, tagged(start ? 0.f : ta.x, tag));
      put_word(agg + mine * 2 + 1, tagged(start ? fmaf(ta.x, s.x, tb.x) : tb.x, tag));
      put_word(agg + mine * 2 + 2, tagged(start ? 0.f : ta.y, tag));
      put_word(agg + mine * 2 + 3, tagged(start ? fmaf(ta.y, s.y, tb.y) : tb.y, tag));
    }
    // The state that enters the tile is that behind the group before, through the tiles of this group that come first: each
    // warp fetches some of these and joins them.  Always the same products in the same order.
    bool gave_up = false;
    if (ahead > 0) {
      const int share = (ahead + warps - 1) / warps, far = min(ahead, (warp + 1) * share);
      float2 ca = make_float2(1.f, 1.f), cb = make_float2(0.f, 0.f);
      for (int k = far; k > warp * share; --k) {
        float w[4];
        await_words<4>(agg + (mine + back * k) * 2, tag, w, &gave_up);
        cb = make_float2(fmaf(w[0], cb.x, w[1]), fmaf(w[2], cb.y, w[3]));
        ca = make_float2(ca.x * w[0], ca.y * w[2]);
      }
      sm_pa[warp][lane] = ca;
      sm_pb[warp][lane] = cb;
      __syncthreads();
    }
    if (publishes) {
      float2 ca = make_float2(1.f, 1.f), cb = make_float2(0.f, 0.f);
      for (int w = warps - 1; w >= 0 && ahead > 0; --w) {
        const float2 wa = sm_pa[w][lane], wb = sm_pb[w][lane];
        cb = make_float2(fmaf(wa.x, cb.x, wb.x), fmaf(wa.y, cb.y, wb.y));
        ca = make_float2(ca.x * wa.x, ca.y * wa.y);
      }
      if (order != ahead) {
        float w[2];
        await_words<2>(inc + mine + back * (ahead + 1), tag, w, &gave_up);
        s = make_float2(fmaf(ca.x, w[0], cb.x), fmaf(ca.y, w[1], cb.y));
      } else if (ahead > 0) {
        s = cb;                                                  // the first tile's pair holds the state
      }
      if (hands_on && ends) {
        put_word(inc + mine, tagged(fmaf(ta.x, s.x, tb.x), tag));
        put_word(inc + mine + 1, tagged(fmaf(ta.y, s.y, tb.y), tag));
      }
      sm_in[lane] = s;
    }
    if ((gave_up || failed) && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_TIMEOUT);
    __syncthreads();
    const float2 in = sm_in[lane];
    float2 first = make_float2(0.f, 0.f);
    s = make_float2(fmaf(fa.x, in.x, fb.x), fmaf(fa.y, in.y, fb.y));
    if (BWD && t0 == 0 && from >= 0 && live) first = make_float2(A.state[from + c], both ? A.state[from + c + 1] : 0.f);
    auto walk = [&](int n, bool inside) {
      float2 out = both_of(0.f), dg = out;
      if (inside) {
        const float2 a = decay2(lds_pair<BF16>(at_g + n * row_bytes)), x = lds_pair<BF16>(at_x + n * row_bytes);
        if (BWD) {
          float2 before = lds_pair<HBF16>(at_h + n * h_row);
          if (n == 0 && t0 == 0) before = first;
          out = add2(x, s);
          s = mul2(a, out);
          dg = mul2(s, before);
        } else {
          out = s = fma2(a, s, x);
        }
      }
      store_pair<BWD ? BF16 : HBF16, TMA>(out_p + n * out_tok, out, both);
      if (BWD) store_pair<BF16, TMA>(dg_p + n * dg_tok, dg, both);
    };
    if (whole && live) {
#pragma unroll
      for (int i = 0; i < S; ++i) walk(BWD ? S - 1 - i : i, true);
    } else if (live) {
      const int rows = min(S, A.T - t0);
#pragma unroll 1
      for (int i = 0; i < rows; ++i) {
        const int n = BWD ? rows - 1 - i : i;
        walk(n, t0 + n < len);
      }
    }
    const bool ends_row = BWD ? tile == 0 && warp == 0 : tile == used - 1 && warp == warps - 1;
    if (live && ends_row && to >= 0) {
      A.last[to + c] = s.x;
      if (both) A.last[to + c + 1] = s.y;
    }
  }
  if (TMA) mbar_settle(&failed);
  if (tiles > 1 && threadIdx.x == 0 && atomicAdd(&W->done, 1u) == gridDim.x - 1) {
    W->ticket = 0;
    W->done = 0;
    W->epoch = tag;
  }
}

// ---------------------------------------------------------------- launches

// Up to here a thread walks its channels' tokens: 64x12x4096 6.0 us, by tiles 9.8; 8x16x2048 6.2 and 4.1.
constexpr int kStepTokens = 12;

struct ScanShape {
  int warps, tiles;
};

static ScanShape scan_shape(int T, int steps) {
  const int need = (T + steps - 1) / steps;
  const int warps = need < kScanWarps ? need : kScanWarps;
  return {warps, (T + warps * steps - 1) / (warps * steps)};
}

static int scan_blocks(int D) { return (D + kScanCh - 1) / kScanCh; }

// Records of the finer of the two tilings.
static size_t scan_records(int B, int T, int D) {
  if (T <= kStepTokens) return 0;
  return (size_t)scan_shape(T, scan_steps<false>()).tiles * B * scan_blocks(D) * kScanCh;
}

// A tensor map of [B, T, D] with channels dense, boxes of 64 channels by `tokens`; false where TMA cannot read it.
static bool scan_map(CUtensorMap* map, const void* p, bool bf16, const RecurArgs& A, long long tok, long long row, int tokens) {
  const TensorMapEncode encode = tensor_map_encoder();
  const cuuint64_t es = bf16 ? 2 : 4;
  if (A.B == 1) row = tok * A.T;
  if (!encode || (uintptr_t)p % 16 || tok <= 0 || row <= 0 || tok * es % 16 || row * es % 16) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)A.D, (cuuint64_t)A.T, (cuuint64_t)A.B}, strides[2] = {tok * es, row * es};
  const cuuint32_t box[3] = {kScanCh, (cuuint32_t)tokens, 1}, ones[3] = {1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(p), dims, strides,
                box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16, bool HBF16, bool BWD, bool TMA>
static int launch_scan(const RecurArgs& A, const ScanMaps& maps, const ScanShape& S, void* workspace, cudaStream_t st) {
  const int blocks = scan_blocks(A.D), span = S.warps * scan_steps<BF16>();
  const long long grid = (long long)S.tiles * A.B * blocks;
  if (grid > 0x7fffffffLL) return SPEC_E_DIM;
  ScanHeader* W = static_cast<ScanHeader*>(workspace);
  Word* agg = reinterpret_cast<Word*>(W + 1);
  Word* inc = agg + 2LL * S.tiles * A.B * blocks * kScanCh;
  constexpr int token_bytes = kScanCh * ((BF16 ? 4 : 8) + (BWD ? (HBF16 ? 2 : 4) : 0));
  const int smem = span * token_bytes;
  const auto kernel = recur_scan_kernel<BF16, HBF16, BWD, TMA>;
  static std::atomic<unsigned long long> allowed;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), kScanWarps * scan_steps<BF16>() * token_bytes, &allowed)) return SPEC_E_CUDA;
  // Every tile of a small call runs at once and a link of the chain is all it waits for: long groups.  (1x65536x2048
  // takes 7 % longer with groups of 32 than with 16; 4x4096x128 is as fast with either.)  The groups decide
  // the order of the products, so they go by the sizes alone, not by how the rows are aligned.
  const int group = grid <= 4 * 152 ? kScanGroupMost : 16;
  kernel<<<(unsigned)grid, S.warps * 32, smem, st>>>(A, maps, W, agg, inc, S.tiles, blocks, group);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <bool BF16, bool HBF16, bool BWD>
static int launch_long(const RecurArgs& A, void* workspace, cudaStream_t st) {
  const ScanShape S = scan_shape(A.T, scan_steps<BF16>());
  const int span = S.warps * scan_steps<BF16>();
  const long long dense = (long long)A.T * A.D;
  ScanMaps maps;
  const bool tma = A.D % 8 == 0 && paged_aligned(A.h, 8) && paged_aligned(A.dg, 8) && scan_map(&maps.g, A.g, BF16, A, A.g_tok, A.g_row, span) &&
                   scan_map(&maps.x, A.x, BF16, A, BWD ? A.D : A.x_tok, BWD ? dense : A.x_row, span) &&
                   (!BWD || scan_map(&maps.h, A.hin, HBF16, A, A.D, dense, span));
  return tma ? launch_scan<BF16, HBF16, BWD, true>(A, maps, S, workspace, st) : launch_scan<BF16, HBF16, BWD, false>(A, maps, S, workspace, st);
}

template <bool BF16, bool HBF16, int VEC, bool BWD>
static int launch_steps(const RecurArgs& A, cudaStream_t st) {
  const dim3 grid((A.D + kStepThreads * VEC - 1) / (kStepThreads * VEC), A.B);
  recur_step_kernel<BF16, HBF16, VEC, BWD><<<grid, kStepThreads, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

// Whether every access of `vec` channels is aligned to its size.
static bool recur_aligned(const RecurArgs& A, int vec, size_t es, size_t hs) {
  if (A.D % vec || A.g_row % vec || A.g_tok % vec || A.x_row % vec || A.x_tok % vec) return false;
  return paged_aligned(A.g, vec * es) && paged_aligned(A.x, vec * es) && paged_aligned(A.dg, vec * es) &&
         paged_aligned(A.hin, vec * hs) && paged_aligned(A.h, vec * (A.hin ? es : hs));
}

template <bool BF16, bool HBF16, bool BWD>
static int launch_recur(const RecurArgs& A, void* workspace, cudaStream_t st) {
  if (A.T > kStepTokens) return launch_long<BF16, HBF16, BWD>(A, workspace, st);
  // 8 bytes a lane of g where they are aligned
  constexpr int most = BF16 ? 4 : 2;
  if (recur_aligned(A, most, BF16 ? 2 : 4, HBF16 ? 2 : 4)) return launch_steps<BF16, HBF16, most, BWD>(A, st);
  return launch_steps<BF16, HBF16, 1, BWD>(A, st);
}

template <bool BWD>
static int recur_launch(const RecurArgs& A, int dtype, int h_dtype, void* workspace, cudaStream_t st) {
  const bool hb = h_dtype == SPEC_BF16;
  if (dtype == SPEC_BF16)
    return hb ? launch_recur<true, true, BWD>(A, workspace, st) : launch_recur<true, false, BWD>(A, workspace, st);
  return hb ? launch_recur<false, true, BWD>(A, workspace, st) : launch_recur<false, false, BWD>(A, workspace, st);
}

static bool recur_dims(int B, int T, int D) { return B >= 0 && B <= 65535 && T >= 0 && T <= SPEC_MAX_LENGTH && D >= 1 && D <= (1 << 26); }

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
  return sizeof(specv::ScanHeader) + specv::scan_records(B, T, D) * 3 * sizeof(unsigned long long);
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
  return recur_launch<false>(A, dtype, h_dtype, workspace, reinterpret_cast<cudaStream_t>(cuda_stream));
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
  return recur_launch<true>(A, dtype, h_dtype, workspace, reinterpret_cast<cudaStream_t>(cuda_stream));
}
