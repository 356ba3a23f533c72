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

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& x : w) x = 0;
  }
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
  // Forgets what was unpacked, so that it is unpacked again and not kept beside the words.
  __device__ __forceinline__ void again() {
#pragma unroll
    for (uint32_t& x : w) asm volatile("" : "+r"(x));
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
constexpr int kScanGroupMost = 32;
constexpr int kScanSpins = 1 << 20;  // about a second of polling
constexpr int kScanSteps = 8;        // the fewest of scan_steps

// Tokens a warp keeps in registers: a decay in float32 and the rest as loaded,
// about 96 registers forward and 64 backward.
template <bool BF16, int VEC, bool BWD>
constexpr int scan_steps() {
  if (BWD) return VEC == 4 ? 8 : VEC == 2 ? (BF16 ? 16 : 8) : 16;
  return VEC == 4 ? 16 : VEC == 2 ? (BF16 ? 32 : 16) : 32;
}

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

// Where a ticket's tile lies.
struct ScanTile {
  int tile, row, c, len;
  bool live, ok;
  long long from, to;
};

template <int VEC, bool BWD>
__device__ __forceinline__ ScanTile scan_tile(const RecurArgs& A, unsigned ticket, int tiles, int blocks, int lane) {
  ScanTile t;
  const unsigned per = (unsigned)A.B * (unsigned)blocks;
  const unsigned nth = ticket / per, rest = ticket - nth * per, row = rest / (unsigned)blocks;
  t.row = (int)row;
  t.tile = BWD ? tiles - 1 - (int)nth : (int)nth;
  t.c = ((int)(rest - row * (unsigned)blocks) * 32 + lane) * VEC;
  t.live = t.c < A.D;
  t.ok = recur_row<BWD>(A, t.row, &t.len, &t.from, &t.to);
  if (!t.ok) t.len = 0;
  return t;
}

// A CTA takes a tile of (32 VEC channels) x (warps * S tokens) of a row.  Tiles
// go by tickets, all channels of all rows before the next tokens, and a tile
// waits only for tiles of smaller tickets, whose CTAs have begun.
template <bool BF16, bool HBF16, int VEC, bool BWD>
__global__ void __launch_bounds__(kScanWarps * 32, 2) recur_scan_kernel(const RecurArgs A, ScanHeader* W, Word* agg, Word* inc,
                                                                         int tiles, int blocks, int group) {
  using In = Channels<BF16, VEC>;
  using H = Channels<HBF16, VEC>;
  using Out = Channels<BWD ? BF16 : HBF16, VEC>;
  constexpr int S = scan_steps<BF16, VEC, BWD>();
  constexpr int es = BF16 ? 2 : 4, hs = HBF16 ? 2 : 4, os = BWD ? es : hs;
  __shared__ float sm_a[kScanWarps][VEC][32], sm_b[kScanWarps][VEC][32], sm_in[VEC][32];
  __shared__ float sm_pa[kScanWarps][VEC][32], sm_pb[kScanWarps][VEC][32];
  __shared__ unsigned sm_ticket, sm_tag;
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int span = warps * S;
  if (threadIdx.x == 0) {
    sm_ticket = tiles > 1 ? atomicAdd(&W->ticket, 1u) : blockIdx.x;
    sm_tag = *(volatile unsigned*)&W->epoch + 1;
  }
  __syncthreads();
  const unsigned tag = sm_tag;
  const ScanTile C = scan_tile<VEC, BWD>(A, sm_ticket, tiles, blocks, lane);
  if (!C.ok && C.tile == 0 && C.c == 0 && warp == 0 && A.flags) atomicOr(&A.flags[C.row], (uint32_t)SPEC_F_BAD_IDX);
  const int used = (C.len + span - 1) / span;                    // tiles of this row that hold tokens
  const int order = BWD ? used - 1 - C.tile : C.tile;            // this tile's place among them
  const int t0 = C.tile * span + warp * S;
  const bool whole = C.live && t0 + S <= C.len;
  const long long base = ((long long)C.row * A.T + t0) * A.D + C.c;
  unsigned char* const out_p = A.h + base * os;
  unsigned char* const dg_p = BWD ? A.dg + base * es : nullptr;
  const long long out_tok = (long long)A.D * os, dg_tok = (long long)A.D * es;

  if (C.tile >= used) {
    // nothing but zeros here; a row without tokens hands its state on
    if (C.live) {
      float zero[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) zero[v] = 0.f;
      for (int i = 0; i < S && t0 + i < A.T; ++i) {
        Out::store(out_p + i * out_tok, zero);
        if (BWD) In::store(dg_p + i * dg_tok, zero);
      }
      if (C.tile == 0 && warp == 0 && C.to >= 0)
        for (int v = 0; v < VEC; ++v)
          A.last[C.to + C.c + v] = BWD ? (A.d_last && C.ok ? A.d_last[(long long)C.row * A.D + C.c + v] : 0.f)
                                       : (C.from >= 0 ? A.state[C.from + C.c + v] : 0.f);
    }
  } else {
    In g[S], x[S];
    const long long g_tok = A.g_tok * es, x_tok = (BWD ? (long long)A.D : A.x_tok) * es;
    const unsigned char* gp = A.g + (C.row * A.g_row + C.c) * es + t0 * g_tok;
    const unsigned char* xp = A.x + (BWD ? base * es : (C.row * A.x_row + C.c) * es + t0 * x_tok);
    if (whole) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        g[i].load(gp + i * g_tok);
        x[i].load(xp + i * x_tok);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        g[i].zero();
        x[i].zero();
        if (C.live && t0 + i < C.len) {
          g[i].load(gp + i * g_tok);
          x[i].load(xp + i * x_tok);
        }
      }
    }
    // this warp's steps as one: s -> pa s + pb (a token beyond the row has g = x = 0: s -> s)
    float a[S][VEC], pa[VEC], pb[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) pa[v] = 1.f, pb[v] = 0.f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = BWD ? S - 1 - i : i;
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        a[n][v] = decay(g[n].get(v));
        pb[v] = BWD ? a[n][v] * (x[n].get(v) + pb[v]) : fmaf(a[n][v], pb[v], x[n].get(v));
        pa[v] *= a[n][v];
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) sm_a[warp][v][lane] = pa[v], sm_b[warp][v][lane] = pb[v];
    __syncthreads();
    const int ahead = order % group;                             // tiles of this group that come first
    const bool ends = ahead == group - 1, hands_on = order < used - 1;
    const bool publishes = warp == (BWD ? 0 : warps - 1);        // the last in order
    const long long mine = ((long long)C.tile * A.B + C.row) * A.D + C.c;
    const long long back = (BWD ? 1LL : -1LL) * A.B * A.D;       // to the tile before in order
    float ta[VEC], tb[VEC];                                      // the whole tile, in the warp that publishes it
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      // what comes before this warp in the tile
      float fa = 1.f, fb = 0.f;
      for (int w = 0; w < (BWD ? warps - 1 - warp : warp); ++w) {
        const int n = BWD ? warps - 1 - w : w;
        const float wa = sm_a[n][v][lane];
        fb = fmaf(wa, fb, sm_b[n][v][lane]);
        fa *= wa;
      }
      ta[v] = fa * pa[v];
      tb[v] = fmaf(pa[v], fb, pb[v]);
      if (publishes && C.live && hands_on && !ends) {
        put_word(agg + (mine + v) * 2, tagged(ta[v], tag));
        put_word(agg + (mine + v) * 2 + 1, tagged(tb[v], tag));
      }
      pa[v] = fa;
      pb[v] = fb;
    }
    H hb[BWD ? S : 1];
    if (BWD) {
      const unsigned char* hp = A.hin + (base - A.D) * hs;
      const long long h_tok = (long long)A.D * hs;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        hb[BWD ? i : 0].zero();
        if (whole ? i > 0 || t0 > 0 : C.live && t0 + i > 0 && t0 + i < C.len) hb[BWD ? i : 0].load(hp + i * h_tok);
      }
    }
    // The state that enters is that behind the group before, through the tiles of this group that come first: each
    // warp fetches some of these and joins them.  Always the same products in the same order.
    bool gave_up = false;
    if (ahead > 0) {
      const int share = (ahead + warps - 1) / warps, far = min(ahead, (warp + 1) * share);
      float ca[VEC], cb[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) ca[v] = 1.f, cb[v] = 0.f;
      for (int k = far; k > warp * share && C.live; --k) {
        float w[2 * VEC];
        await_words<2 * VEC>(agg + (mine + back * k) * 2, tag, w, &gave_up);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          cb[v] = fmaf(w[2 * v], cb[v], w[2 * v + 1]);
          ca[v] *= w[2 * v];
        }
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) sm_pa[warp][v][lane] = ca[v], sm_pb[warp][v][lane] = cb[v];
      __syncthreads();
    }
    if (publishes) {
      float s[VEC], ca[VEC], cb[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        ca[v] = 1.f, cb[v] = 0.f, s[v] = 0.f;
        for (int w = warps - 1; w >= 0 && ahead > 0; --w) {
          cb[v] = fmaf(sm_pa[w][v][lane], cb[v], sm_pb[w][v][lane]);
          ca[v] *= sm_pa[w][v][lane];
        }
      }
      if (C.live) {
        if (order != ahead) {
          await_words<VEC>(inc + mine + back * (ahead + 1), tag, s, &gave_up);
        } else {
#pragma unroll
          for (int v = 0; v < VEC; ++v)
            s[v] = BWD ? (A.d_last ? A.d_last[(long long)C.row * A.D + C.c + v] : 0.f)
                       : C.from >= 0 ? A.state[C.from + C.c + v] : 0.f;
        }
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        s[v] = fmaf(ca[v], s[v], cb[v]);
        if (C.live && hands_on && ends) put_word(inc + mine + v, tagged(fmaf(ta[v], s[v], tb[v]), tag));
        sm_in[v][lane] = s[v];
      }
    }
    if (gave_up && A.flags) atomicOr(&A.flags[C.row], (uint32_t)SPEC_F_TIMEOUT);
    __syncthreads();
    float s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) s[v] = fmaf(pa[v], sm_in[v][lane], pb[v]);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int n = BWD ? S - 1 - i : i;
      float out[VEC], dg[VEC];
      x[n].again();
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        if (BWD) {
          out[v] = x[n].get(v) + s[v];
          s[v] = a[n][v] * out[v];
          float before = hb[BWD ? n : 0].get(v);
          if (n == 0 && t0 == 0) before = C.from >= 0 && C.live ? A.state[C.from + C.c + v] : 0.f;
          dg[v] = s[v] * before;
        } else {
          s[v] = fmaf(a[n][v], s[v], x[n].get(v));
          out[v] = s[v];
        }
        if (!whole && t0 + n >= C.len) out[v] = dg[v] = 0.f;
      }
      if (whole || (C.live && t0 + n < A.T)) {
        Out::store(out_p + n * out_tok, out);
        if (BWD) In::store(dg_p + n * dg_tok, dg);
      }
    }
    const bool ends_row = BWD ? C.tile == 0 && warp == 0 : C.tile == used - 1 && warp == warps - 1;
    if (C.live && ends_row && C.to >= 0)
#pragma unroll
      for (int v = 0; v < VEC; ++v) A.last[C.to + C.c + v] = s[v];
  }
  if (tiles > 1 && threadIdx.x == 0 && atomicAdd(&W->done, 1u) == gridDim.x - 1) {
    W->ticket = 0;
    W->done = 0;
    W->epoch = tag;
  }
}

// ---------------------------------------------------------------- launches

constexpr int kStepTokens = 32;     // up to here a thread walks its channels' tokens

struct ScanShape {
  int warps, tiles;
};

static ScanShape scan_shape(int T, int steps) {
  const int need = (T + steps - 1) / steps;
  const int warps = need < kScanWarps ? need : kScanWarps;
  return {warps, (T + warps * steps - 1) / (warps * steps)};
}

static size_t scan_records(int B, int T, int D) {
  if (T <= kStepTokens) return 0;
  return (size_t)scan_shape(T, kScanSteps).tiles * B * D;
}

template <bool BF16, bool HBF16, int VEC, bool BWD>
static int launch_recur(const RecurArgs& A, void* workspace, cudaStream_t st) {
  if (A.T <= kStepTokens) {
    const dim3 grid((A.D + kStepThreads * VEC - 1) / (kStepThreads * VEC), A.B);
    recur_step_kernel<BF16, HBF16, VEC, BWD><<<grid, kStepThreads, 0, st>>>(A);
  } else {
    const ScanShape S = scan_shape(A.T, scan_steps<BF16, VEC, BWD>());
    const int blocks = (A.D + 32 * VEC - 1) / (32 * VEC);
    const long long work = (long long)S.tiles * A.B * blocks;
    if (work > 0x7fffffffLL) return SPEC_E_DIM;
    ScanHeader* W = static_cast<ScanHeader*>(workspace);
    Word* agg = reinterpret_cast<Word*>(W + 1);
    Word* inc = agg + 2LL * S.tiles * A.B * A.D;
    const int group = work <= 2 * 152 ? kScanGroupMost : 16;
    recur_scan_kernel<BF16, HBF16, VEC, BWD><<<(unsigned)work, S.warps * 32, 0, st>>>(A, W, agg, inc, S.tiles, blocks, group);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

// Whether every access of `vec` channels is aligned to its size.
static bool recur_aligned(const RecurArgs& A, int vec, size_t es, size_t hs) {
  if (A.D % vec || A.g_row % vec || A.g_tok % vec || A.x_row % vec || A.x_tok % vec) return false;
  return paged_aligned(A.g, vec * es) && paged_aligned(A.x, vec * es) && paged_aligned(A.dg, vec * es) &&
         paged_aligned(A.hin, vec * hs) && paged_aligned(A.h, vec * (A.hin ? es : hs));
}

template <bool BF16, bool HBF16, bool BWD>
static int launch_vec(const RecurArgs& A, void* workspace, cudaStream_t st) {
  // 8 bytes a lane of g, less where a warp's width would leave half of its lanes idle
  constexpr int most = BF16 ? 4 : 2;
  if (A.D > 16 * most && recur_aligned(A, most, BF16 ? 2 : 4, HBF16 ? 2 : 4))
    return launch_recur<BF16, HBF16, most, BWD>(A, workspace, st);
  if (BF16 && A.D > 32 && recur_aligned(A, 2, 2, HBF16 ? 2 : 4))
    return launch_recur<BF16, HBF16, 2, BWD>(A, workspace, st);
  return launch_recur<BF16, HBF16, 1, BWD>(A, workspace, st);
}

template <bool BWD>
static int recur_launch(const RecurArgs& A, int dtype, int h_dtype, void* workspace, cudaStream_t st) {
  const bool hb = h_dtype == SPEC_BF16;
  if (dtype == SPEC_BF16)
    return hb ? launch_vec<true, true, BWD>(A, workspace, st) : launch_vec<true, false, BWD>(A, workspace, st);
  return hb ? launch_vec<false, true, BWD>(A, workspace, st) : launch_vec<false, false, BWD>(A, workspace, st);
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
