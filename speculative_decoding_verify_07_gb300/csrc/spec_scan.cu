// spec_scan: h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t, y_t = c_t . h_t, for N
// states of each channel.
//
// A channel's states lie with N / 4 neighbouring lanes, four each, so that a warp
// reads and writes 512 bytes of states side by side; the sum over the states goes
// through the lanes.
//
// A few tokens: bound by the states' bytes (one in, one out a token for the commit).
#include <algorithm>

#include "spec_mixer.cuh"
#include "spec_tma.cuh"

#ifndef SPEC_SCAN_CTAS
#define SPEC_SCAN_CTAS 2
#endif

namespace specv {

struct ScanArgs {
  const void *x, *dt, *z, *b, *c;
  const float *a, *skip, *dt_bias, *state;
  const int32_t *slot, *lens;
  void* y;
  float *states, *last;
  const int32_t* last_slot;
  uint32_t* flags;
  long long x_row, x_tok, dt_row, dt_tok, z_row, z_tok, b_row, b_tok, b_group, c_row, c_tok, c_group;
  int B, T, D, each, slots, last_slots;      // each: channels of a group
  bool softplus;
};

// ln(1 + exp(v)) within 12 half steps (2^-24) of itself: max(v, 0) + 2 atanh(e / (2 + e)), e = exp(-|v|), by
// the series of atanh up to s^15, s = e / (2 + e) at most 1/3 (what is left out is 2^-26 of it).
__device__ __forceinline__ float2 softplus(float2 v) {
  const float2 pos = make_float2(v.x < 0.f ? 0.f : v.x, v.y < 0.f ? 0.f : v.y);
  const float2 m = make_float2(-fminf(fabsf(v.x), 87.f), -fminf(fabsf(v.y), 87.f));
  // exp(m) with the rounding of m log2(e) made up for
  const float2 p = mul2(m, both_of(kLog2e)), low = fma2(m, both_of(1.92596299e-8f), fma2(m, both_of(kLog2e), make_float2(-p.x, -p.y)));
  const float2 e0 = make_float2(exp2_fast(p.x), exp2_fast(p.y)), e = fma2(e0, mul2(low, both_of(0.6931471805599453f)), e0);
  const float2 s = make_float2(__fdividef(e.x, 2.f + e.x), __fdividef(e.y, 2.f + e.y)), q = mul2(s, s);
  float2 t = both_of(1.f / 15.f);
  t = fma2(t, q, both_of(1.f / 13.f));
  t = fma2(t, q, both_of(1.f / 11.f));
  t = fma2(t, q, both_of(1.f / 9.f));
  t = fma2(t, q, both_of(1.f / 7.f));
  t = fma2(t, q, both_of(1.f / 5.f));
  t = fma2(t, q, both_of(1.f / 3.f));
  t = fma2(t, q, both_of(1.f));
  return fma2(add2(s, s), t, pos);
}

// exp(g) of two states, y = g log2(e).  An error of the decay adds up over the tokens that
// the state remembers, 1 / (1 - exp(g)) of them, and that of ex2.approx leans to one side
// (by 1e-8 to 3e-8 in the mean below |g| = 1/2, measured), so below |g| = 1/32 the series to
// g^3 is taken instead.
__device__ __forceinline__ float2 scan_decay(float2 y) {
  constexpr float ln2 = 0.6931471805599453f;
  const float2 near = fma2(fma2(fma2(y, both_of(ln2 * ln2 * ln2 / 6.f), both_of(ln2 * ln2 / 2.f)), y, both_of(ln2)), y, both_of(1.f));
  const float2 a = make_float2(exp2_fast(y.x), exp2_fast(y.y));
  constexpr float border = 0.03125f / ln2;
  return make_float2(fabsf(y.x) < border ? near.x : a.x, fabsf(y.y) < border ? near.y : a.y);
}

// Four neighbouring states' b or c, as they are in memory.
template <bool BF16>
struct ScanFour {
  uint32_t w[BF16 ? 2 : 4];
  __device__ __forceinline__ void load(const void* p, long long i, bool wide) {
    if (BF16) {
      const uint16_t* q = static_cast<const uint16_t*>(p) + i;
      if (wide) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = __ldg(q) | (uint32_t)__ldg(q + 1) << 16;
        w[1] = __ldg(q + 2) | (uint32_t)__ldg(q + 3) << 16;
      }
    } else {
      const uint32_t* q = static_cast<const uint32_t*>(p) + i;
      if (wide) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
        w[0] = v.x, w[1] = v.y, w[BF16 ? 0 : 2] = v.z, w[BF16 ? 0 : 3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < (BF16 ? 2 : 4); ++j) w[j] = __ldg(q + j);
      }
    }
  }
  __device__ __forceinline__ float2 get(int j) const {
    if (BF16) return make_float2(bf16_lo(w[j]), bf16_hi(w[j]));
    return make_float2(__uint_as_float(w[BF16 ? 0 : 2 * j]), __uint_as_float(w[BF16 ? 0 : 2 * j + 1]));
  }
};

// The sums over a channel's L lanes of four tokens' parts: two of four tokens for two lanes, one for four and more.
// Which tokens: scan_token.
template <int L>
__device__ __forceinline__ int scan_token(int lane) { return (lane & 1) * 2 + (L > 2 ? lane >> 1 & 1 : 0); }
template <int L>
__device__ __forceinline__ void scan_sum(float* y, int lane) {
  const bool odd = lane & 1;
  float k0 = odd ? y[2] : y[0], k1 = odd ? y[3] : y[1];
  k0 += __shfl_xor_sync(0xffffffffu, odd ? y[0] : y[2], 1);
  k1 += __shfl_xor_sync(0xffffffffu, odd ? y[1] : y[3], 1);
  y[0] = k0;
  y[1] = k1;
  if (L == 2) return;
  const bool two = lane & 2;
  float k = two ? k1 : k0;
  k += __shfl_xor_sync(0xffffffffu, two ? k0 : k1, 2);
#pragma unroll
  for (int w = 4; w < L; w *= 2) k += __shfl_xor_sync(0xffffffffu, k, w);
  y[0] = k;
}

// ---------------------------------------------------------------- few tokens

constexpr int kScanStepThreads = 128;

// Four tokens at a time: each of a channel's lanes fetches one token's inputs (two where there are two lanes), and
// the lanes hand them to one another.
template <bool BF16, int N>
__global__ void __launch_bounds__(kScanStepThreads) scan_step_kernel(const ScanArgs A, bool wide) {
  constexpr int L = N / 4, own = L == 2 ? 2 : 1;
  const int r = blockIdx.y;
  const long long i = (long long)blockIdx.x * kScanStepThreads + threadIdx.x;
  const bool mine = i < (long long)A.D * L;      // (lanes beyond the last channel follow its sums)
  const int d = mine ? (int)(i / L) : A.D - 1, lane = (int)(i % L), q = lane * 4, j0 = scan_token<L>(lane);
  const MixerRow R = mixer_row(A, r, i == 0);
  const int g = d / A.each;
  const long long xb = r * A.x_row + d, db = r * A.dt_row + d, zb = r * A.z_row + d;
  const long long bb = r * A.b_row + g * A.b_group + q, cb = r * A.c_row + g * A.c_group + q;
  const long long out = (long long)r * A.T * A.D + d;
  const float4 av = __ldg(reinterpret_cast<const float4*>(A.a + (long long)d * N + q));
  const float2 a[2] = {mul2(make_float2(av.x, av.y), both_of(kLog2e)), mul2(make_float2(av.z, av.w), both_of(kLog2e))};
  const float skip = A.skip ? __ldg(A.skip + d) : 0.f, bias = A.dt_bias ? __ldg(A.dt_bias + d) : 0.f;
  float2 h[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  if (R.from >= 0) {
    const float4 s = *reinterpret_cast<const float4*>(A.state + ((long long)R.from * A.D + d) * N + q);
    h[0] = make_float2(s.x, s.y);
    h[1] = make_float2(s.z, s.w);
  }
#pragma unroll 1
  for (int t0 = 0; t0 < R.len; t0 += 4) {
    float x[own], z[own], delta[2] = {0.f, 0.f}, put[own];
    ScanFour<BF16> b[4], c[4];
#pragma unroll
    for (int k = 0; k < own; ++k) {
      const int t = min(t0 + j0 + k, R.len - 1);
      x[k] = load_one<BF16>(A.x, xb + t * A.x_tok);
      delta[k] = load_one<BF16>(A.dt, db + t * A.dt_tok) + bias;
      z[k] = A.z ? load_one<BF16>(A.z, zb + t * A.z_tok) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = min(t0 + k, R.len - 1);
      b[k].load(A.b, bb + t * A.b_tok, wide);
      c[k].load(A.c, cb + t * A.c_tok, wide);
    }
    if (A.softplus) {
      const float2 s = softplus(make_float2(delta[0], delta[1]));
      delta[0] = s.x, delta[1] = s.y;
    }
#pragma unroll
    for (int k = 0; k < own; ++k) put[k] = delta[k] * x[k];
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t0 + k >= R.len) break;
      // the lane of the channel that has token k: scan_token's inverse
      const int from = L == 2 ? k >> 1 : (k >> 1) + (k & 1) * 2, at = L == 2 ? k & 1 : 0;
      const float2 step = both_of(__shfl_sync(0xffffffffu, at ? delta[1] : delta[0], from, L));
      const float2 in = both_of(__shfl_sync(0xffffffffu, put[own > 1 ? at : 0], from, L));
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        h[j] = fma2(scan_decay(mul2(step, a[j])), h[j], mul2(in, b[k].get(j)));
        sum = fma2(c[k].get(j), h[j], sum);
      }
      y[k] = sum.x + sum.y;
      if (A.states && mine)
        __stcs(reinterpret_cast<float4*>(A.states + (out + (long long)(t0 + k) * A.D) * N + q), make_float4(h[0].x, h[0].y, h[1].x, h[1].y));
    }
    scan_sum<L>(y, lane);
#pragma unroll
    for (int k = 0; k < own; ++k) {
      const int t = t0 + j0 + k;
      if (mine && t < R.len && lane < 4) {
        float v = fmaf(skip, x[k], y[k]);
        if (A.z) v *= silu(z[k]);
        store_one<BF16>(A.y, out + (long long)t * A.D, v);
      }
    }
  }
  if (!mine) return;
  for (int t = R.len; t < A.T; ++t) {
    if (lane == 0) store_one<BF16>(A.y, out + (long long)t * A.D, 0.f);
    if (A.states) __stcs(reinterpret_cast<float4*>(A.states + (out + (long long)t * A.D) * N + q), make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (R.to >= 0) *reinterpret_cast<float4*>(A.last + ((long long)R.to * A.D + d) * N + q) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}

// --------------------------------------------------------------- many tokens
//
// A CTA walks tiles of tokens of its channels: delta, delta x, b and c of a tile are made
// in shared memory by all threads, each lane then takes two channels by four states through
// the tile's tokens and leaves its part of each sum there, and what goes through a token's
// elements again (the sum, skip, gate, output) is done by the thread that fetched them.  Two
// channels a lane share the loads of b and c.
//
// Decays are ex2.approx alone here, whose lean to one side (see scan_decay) would add up over
// the tokens that a state remembers.  So the tile's decays are also multiplied, and at its end
// the state that entered gets the difference to the exact decay of the tile's sum of delta.

#ifndef SPEC_SCAN_THREADS
#define SPEC_SCAN_THREADS 256
#endif
constexpr int kScanThreads = SPEC_SCAN_THREADS;
constexpr int kScanPair = 2;           // channels of a lane
constexpr int kScanTile = 16;          // tokens of a tile

template <bool BF16, int N, int VEC>
struct ScanShape {
  static constexpr int L = N / 4;                              // lanes of a channel
  static constexpr int CH = kScanThreads / L * kScanPair;      // channels of a CTA
  static constexpr int vecs = CH / VEC;                        // a token's channels, VEC at a time
  static constexpr int rows = kScanThreads / vecs;             // tokens fetched at a time
  static constexpr int per = rows > kScanTile ? 1 : kScanTile / rows;
  static constexpr int bc = kScanTile * N / 2 < kScanThreads ? 1 : kScanTile * N / 2 / kScanThreads;    // pairs of states of b and c a thread
};

// VEC neighbouring elements as they are in memory.
template <bool BF16, int VEC>
struct ScanVec {
  static constexpr int kWords = BF16 ? (VEC + 1) / 2 : VEC;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const void* p) {
    if (VEC == 1 && BF16) {
      w[0] = __ldg(static_cast<const uint16_t*>(p));
    } else if (kWords == 1) {
      w[0] = __ldg(static_cast<const uint32_t*>(p));
    } else if (kWords == 2) {
      const uint2 v = __ldg(static_cast<const uint2*>(p));
      w[0] = v.x, w[kWords - 1] = v.y;
    } else {
      const uint4 v = __ldg(static_cast<const uint4*>(p));
      w[0] = v.x, w[kWords / 4] = v.y, w[kWords / 2] = v.z, w[kWords / 4 * 3] = v.w;
    }
  }
  // Elements 2 i and 2 i + 1 (zero where there is none).
  __device__ __forceinline__ float2 get(int i) const {
    if (BF16) return make_float2(bf16_lo(w[i]), VEC > 1 ? bf16_hi(w[i]) : 0.f);
    return make_float2(__uint_as_float(w[VEC > 1 ? 2 * i : 0]), VEC > 1 ? __uint_as_float(w[VEC > 1 ? 2 * i + 1 : 0]) : 0.f);
  }
};

// Where the CTA's channels lie: those of one group.
struct ScanPlace {
  int r, seg, g, d0, left;       // left: channels from d0 to the group's end
};
__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& A, int ch) {
  const int blocks = (A.each + ch - 1) / ch, groups = A.D / A.each;
  ScanPlace P;
  P.r = blockIdx.y;
  P.seg = blockIdx.x / (blocks * groups);
  const int b = blockIdx.x - P.seg * blocks * groups;
  P.g = b / blocks;
  const int c = (b - P.g * blocks) * ch;
  P.d0 = P.g * A.each + c;
  P.left = min(A.each - c, ch);
  return P;
}

template <int N, int CH, bool Y>
struct ScanShared {
  float2 step[kScanTile][CH];                    // (delta, delta x)
  float b[kScanTile][N], c[Y ? kScanTile : 1][N];
  float part[Y ? kScanTile : 1][kScanPair][kScanThreads];     // each thread's part of the sums of its channels
};

// A tile's elements on their way, and where this thread's lie.
template <bool BF16, int N, int VEC, bool Y, bool GATE>
struct ScanFetch {
  using S = ScanShape<BF16, N, VEC>;
  static constexpr int es = BF16 ? 2 : 4;
  ScanVec<BF16, VEC> x[S::per], dt[S::per], z[GATE ? S::per : 1];
  ScanVec<BF16, 2> b[S::bc], c[Y ? S::bc : 1];
  const unsigned char *px, *pdt, *pz;              // of the row's token 0
  const unsigned char *pb, *pc;
  bool whole;                                      // all channels of the CTA are there

  // The i-th fetch's token of the tile, and the first channel.
  static __device__ __forceinline__ int token(int i) { return threadIdx.x / S::vecs + i * S::rows; }
  static __device__ __forceinline__ int channel() { return threadIdx.x % S::vecs * VEC; }
  static __device__ __forceinline__ bool real(int i) { return S::rows <= kScanTile || token(i) < kScanTile; }

  __device__ __forceinline__ ScanFetch(const ScanArgs& A, const ScanPlace& P) {
    px = static_cast<const unsigned char*>(A.x) + (P.r * A.x_row + P.d0) * es;
    pdt = static_cast<const unsigned char*>(A.dt) + (P.r * A.dt_row + P.d0) * es;
    if (GATE) pz = static_cast<const unsigned char*>(A.z) + (P.r * A.z_row + P.d0) * es;
    pb = static_cast<const unsigned char*>(A.b) + (P.r * A.b_row + P.g * A.b_group) * es;
    if (Y) pc = static_cast<const unsigned char*>(A.c) + (P.r * A.c_row + P.g * A.c_group) * es;
    whole = P.left == S::CH;
  }
  __device__ __forceinline__ void load(const ScanArgs& A, const ScanPlace& P, int t0, int end, bool pairs) {
    const bool all = whole && t0 + kScanTile <= end;
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      const int t = t0 + token(i), c = channel();
      if (real(i) && (all || (t < end && c < P.left))) {
        x[i].load(px + (t * A.x_tok + c) * es);
        dt[i].load(pdt + (t * A.dt_tok + c) * es);
        if (GATE) z[GATE ? i : 0].load(pz + (t * A.z_tok + c) * es);
      } else {
        x[i].zero(), dt[i].zero();
        if (GATE) z[GATE ? i : 0].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < S::bc; ++i) {
      const int at = i * kScanThreads + threadIdx.x, t = t0 + at / (N / 2), n = at % (N / 2) * 2;
      b[i].zero();
      if (Y) c[Y ? i : 0].zero();
      if (at < kScanTile * N / 2 && t < end) {
        get(b[i], pb + (t * A.b_tok + n) * es, pairs);
        if (Y) get(c[Y ? i : 0], pc + (t * A.c_tok + n) * es, pairs);
      }
    }
  }
  static __device__ __forceinline__ void get(ScanVec<BF16, 2>& v, const unsigned char* p, bool pairs) {
    if (pairs) {
      v.load(p);
    } else {
      ScanVec<BF16, 1> lo, hi;
      lo.load(p);
      hi.load(p + es);
      if (BF16) v.w[0] = lo.w[0] | hi.w[0] << 16;
      else v.w[0] = lo.w[0], v.w[BF16 ? 0 : 1] = hi.w[0];
    }
  }
  // The tile in shared memory.  Tokens behind `end` leave the state.
  __device__ __forceinline__ void put(const ScanArgs& A, const ScanPlace& P, int t0, int end, ScanShared<N, S::CH, Y>& sm) const {
    const bool all = whole && t0 + kScanTile <= end;
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      const int t = token(i), c = channel();
      if (!real(i)) continue;
      const bool there = all || (t0 + t < end && c < P.left);
#pragma unroll
      for (int v = 0; v < (VEC + 1) / 2; ++v) {
        float2 bias = make_float2(0.f, 0.f);
        if (A.dt_bias && there) {
          if (VEC > 1) bias = __ldg(reinterpret_cast<const float2*>(A.dt_bias + P.d0 + c) + v);
          else bias.x = __ldg(A.dt_bias + P.d0 + c);
        }
        float2 delta = add2(dt[i].get(v), bias);
        if (A.softplus) delta = softplus(delta);
        if (!there) delta = make_float2(0.f, 0.f);
        const float2 in = mul2(delta, x[i].get(v));
        if (VEC > 1) *reinterpret_cast<float4*>(&sm.step[t][c + 2 * v]) = make_float4(delta.x, in.x, delta.y, in.y);
        else sm.step[t][c] = make_float2(delta.x, in.x);
      }
    }
#pragma unroll
    for (int i = 0; i < S::bc; ++i) {
      const int at = i * kScanThreads + threadIdx.x, t = at / (N / 2), n = at % (N / 2) * 2;
      if (at < kScanTile * N / 2) {
        *reinterpret_cast<float2*>(&sm.b[t][n]) = b[i].get(0);
        if (Y) *reinterpret_cast<float2*>(&sm.c[Y ? t : 0][n]) = c[Y ? i : 0].get(0);
      }
    }
  }
};

// A lane's four states of two channels.
struct ScanStates {
  float2 v[kScanPair][2];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int c = 0; c < kScanPair; ++c) v[c][0] = v[c][1] = both_of(x);
  }
  // channel d of `p`, [channel][N], and the next one where there is one
  __device__ __forceinline__ void load(const float* p, long long d, int N, int q, bool both) {
#pragma unroll
    for (int c = 0; c < kScanPair; ++c) {
      const float4 s = *reinterpret_cast<const float4*>(p + (d + (both ? c : 0)) * N + q);
      v[c][0] = make_float2(s.x, s.y);
      v[c][1] = make_float2(s.z, s.w);
    }
  }
  __device__ __forceinline__ void store(float* p, long long d, int N, int q, bool both) const {
#pragma unroll
    for (int c = 0; c < kScanPair; ++c)
      if (c == 0 || both) *reinterpret_cast<float4*>(p + (d + c) * N + q) = make_float4(v[c][0].x, v[c][0].y, v[c][1].x, v[c][1].y);
  }
  __device__ __forceinline__ void times(float by) {
#pragma unroll
    for (int c = 0; c < kScanPair; ++c) v[c][0] = mul2(v[c][0], both_of(by)), v[c][1] = mul2(v[c][1], both_of(by));
  }
};

// Workspace of a call whose tokens are split: each segment's sum of delta by (row, segment, channel), then by (row,
// segment, channel, state) the state behind the segment if it began with zeros, which scan_join_kernel turns into
// the state that enters it.
struct ScanSplit {
  int segments, span;                  // tokens of a segment
  float* sums;
  float* states;
};

template <bool BF16, int N, int VEC, bool GATE>
__global__ void __launch_bounds__(kScanThreads, SPEC_SCAN_CTAS) scan_tile_kernel(const ScanArgs A, const ScanSplit W, bool pairs) {
  using S = ScanShape<BF16, N, VEC>;
  using F = ScanFetch<BF16, N, VEC, true, GATE>;
  constexpr int L = S::L, CH = S::CH;
  extern __shared__ __align__(16) unsigned char raw[];
  ScanShared<N, CH, true>& sm = *reinterpret_cast<ScanShared<N, CH, true>*>(raw);
  const ScanPlace P = scan_place(A, CH);
  const MixerRow R = mixer_row(A, P.r, P.seg == 0 && P.d0 == 0 && threadIdx.x == 0);
  const int first = P.seg * W.span, stop = (int)min((long long)first + W.span, (long long)A.T), end = min(stop, R.len);
  const int ch = threadIdx.x / L * kScanPair, lane = threadIdx.x % L, q = lane * 4, d = P.d0 + min(ch, P.left - 1);
  const bool mine = ch < P.left, both = ch + 1 < P.left;
  F in(A, P);
  if (first < end) in.load(A, P, first, end, pairs);
  ScanStates a, h;
  a.load(A.a, d, N, q, both);
  a.times(kLog2e);
  h.fill(0.f);
  if (W.segments > 1) h.load(W.states, (long long)(P.r * W.segments + P.seg) * A.D + d, N, q, both);
  else if (R.from >= 0) h.load(A.state, (long long)R.from * A.D + d, N, q, both);
  const long long out = (long long)P.r * A.T * A.D + P.d0;
  for (int t0 = first; t0 < end; t0 += kScanTile) {
    in.put(A, P, t0, end, sm);
    ScanVec<BF16, VEC> x[S::per], z[GATE ? S::per : 1];
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      x[i] = in.x[i];
      if (GATE) z[GATE ? i : 0] = in.z[GATE ? i : 0];
    }
    __syncthreads();
    if (t0 + kScanTile < end) in.load(A, P, t0 + kScanTile, end, pairs);
    const ScanStates was = h;
    ScanStates all;
    all.fill(1.f);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int t = 0; t < kScanTile; t += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 s = *reinterpret_cast<const float4*>(&sm.step[t + j][ch]);
        const float4 b = *reinterpret_cast<const float4*>(&sm.b[t + j][q]), c = *reinterpret_cast<const float4*>(&sm.c[t + j][q]);
        sum = add2(sum, make_float2(s.x, s.z));
#pragma unroll
        for (int k = 0; k < kScanPair; ++k) {
          const float step = k ? s.z : s.x, in = k ? s.w : s.y;
          const float2 w0 = make_float2(exp2_fast(step * a.v[k][0].x), exp2_fast(step * a.v[k][0].y));
          const float2 w1 = make_float2(exp2_fast(step * a.v[k][1].x), exp2_fast(step * a.v[k][1].y));
          all.v[k][0] = mul2(all.v[k][0], w0);
          all.v[k][1] = mul2(all.v[k][1], w1);
          h.v[k][0] = fma2(w0, h.v[k][0], make_float2(in * b.x, in * b.y));
          h.v[k][1] = fma2(w1, h.v[k][1], make_float2(in * b.z, in * b.w));
          const float2 y = fma2(make_float2(c.z, c.w), h.v[k][1], mul2(make_float2(c.x, c.y), h.v[k][0]));
          sm.part[t + j][k][threadIdx.x] = y.x + y.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kScanPair; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 w = scan_decay(mul2(both_of(k ? sum.y : sum.x), a.v[k][j]));
        // (a state that is not finite stays what it has become)
        const float2 s = make_float2(fabsf(was.v[k][j].x) < INFINITY ? was.v[k][j].x : 0.f, fabsf(was.v[k][j].y) < INFINITY ? was.v[k][j].y : 0.f);
        h.v[k][j] = fma2(add2(w, make_float2(-all.v[k][j].x, -all.v[k][j].y)), s, h.v[k][j]);
      }
    __syncthreads();
    const bool every = in.whole && t0 + kScanTile <= end;
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      const int t = F::token(i), c = F::channel();
      if (!F::real(i) || !(every || (t0 + t < end && c < P.left))) continue;
      float2 y[(VEC + 1) / 2];
#pragma unroll
      for (int v = 0; v < (VEC + 1) / 2; ++v) {
        float2 skip = make_float2(0.f, 0.f);
        y[v] = make_float2(0.f, 0.f);
        // the parts of a channel's lanes
        const float* p = &sm.part[t][VEC > 1 ? 0 : c & 1][(c / 2 + v) * L];
        if (L == 2) {
          const float2 e = *reinterpret_cast<const float2*>(p);
          y[v].x = e.x + e.y;
          if (VEC > 1) {
            const float2 o = *reinterpret_cast<const float2*>(p + kScanThreads);
            y[v].y = o.x + o.y;
          }
        } else {
#pragma unroll
          for (int m = 0; m < L / 4; ++m) {
            const float4 e = *reinterpret_cast<const float4*>(p + 4 * m);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (VEC > 1) o = *reinterpret_cast<const float4*>(p + kScanThreads + 4 * m);
            y[v] = add2(y[v], add2(add2(make_float2(e.x, o.x), make_float2(e.y, o.y)), add2(make_float2(e.z, o.z), make_float2(e.w, o.w))));
          }
        }
        if (A.skip) {
          if (VEC > 1) skip = __ldg(reinterpret_cast<const float2*>(A.skip + P.d0 + c) + v);
          else skip.x = __ldg(A.skip + P.d0 + c);
        }
        y[v] = fma2(skip, x[i].get(v), y[v]);
        if (GATE) {
          const float2 g = z[GATE ? i : 0].get(v);
          y[v] = mul2(y[v], make_float2(silu(g.x), VEC > 1 ? silu(g.y) : 0.f));
        }
      }
      const long long to = out + (long long)(t0 + t) * A.D + c;
      constexpr int last = (VEC + 1) / 2 - 1;
      if (VEC == 1) store_one<BF16>(A.y, to, y[0].x);
      else if (BF16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + to) = make_uint2(pack_bf16(y[0].x, y[0].y), pack_bf16(y[last].x, y[last].y));
      else *reinterpret_cast<float4*>(static_cast<float*>(A.y) + to) = make_float4(y[0].x, y[0].y, y[last].x, y[last].y);
    }
  }
  for (long long i = (long long)max(first, R.len) * P.left + threadIdx.x; i < (long long)stop * P.left; i += kScanThreads)
    store_one<BF16>(A.y, out + i / P.left * A.D + i % P.left, 0.f);
  // the segment of the last token has the last state
  if (mine && R.to >= 0 && (W.segments == 1 || (R.len > 0 ? first < R.len && R.len <= stop : P.seg == 0)))
    h.store(A.last, (long long)R.to * A.D + d, N, q, both);
}

// The state behind a segment that begins with zeros, from its last token to the first:
// sum_t exp(a (delta of the tokens after t)) delta_t x_t b_t.  Each weight is taken by
// itself, so nothing adds up.
template <bool BF16, int N, int VEC>
__global__ void __launch_bounds__(kScanThreads) scan_segment_kernel(const ScanArgs A, const ScanSplit W, bool pairs) {
  using S = ScanShape<BF16, N, VEC>;
  constexpr int L = S::L, CH = S::CH;
  extern __shared__ __align__(16) unsigned char raw[];
  ScanShared<N, CH, false>& sm = *reinterpret_cast<ScanShared<N, CH, false>*>(raw);
  const ScanPlace P = scan_place(A, CH);
  const MixerRow R = mixer_row(A, P.r, false);
  const int first = P.seg * W.span, end = min((int)min((long long)first + W.span, (long long)A.T), R.len);
  const int ch = threadIdx.x / L * kScanPair, lane = threadIdx.x % L, q = lane * 4, d = P.d0 + min(ch, P.left - 1);
  const bool both = ch + 1 < P.left;
  ScanFetch<BF16, N, VEC, false, false> in(A, P);
  const int tiles = first < end ? (end - first + kScanTile - 1) / kScanTile : 0;
  if (tiles) in.load(A, P, first + (tiles - 1) * kScanTile, end, pairs);
  ScanStates a, h;
  a.load(A.a, d, N, q, both);
  a.times(kLog2e);
  h.fill(0.f);
  float2 behind = make_float2(0.f, 0.f);                  // the delta of the tiles behind this one
  for (int k = tiles - 1; k >= 0; --k) {
    const int t0 = first + k * kScanTile;
    if (k < tiles - 1) __syncthreads();
    in.put(A, P, t0, end, sm);
    __syncthreads();
    if (k) in.load(A, P, t0 - kScanTile, end, pairs);
    float2 here = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int t = kScanTile - 1; t >= 0; --t) {
      const float4 s = *reinterpret_cast<const float4*>(&sm.step[t][ch]);
      const float4 b = *reinterpret_cast<const float4*>(&sm.b[t][q]);
      const float2 after = add2(behind, here);
#pragma unroll
      for (int c = 0; c < kScanPair; ++c) {
        const float far = c ? after.y : after.x, in = c ? s.w : s.y;
        h.v[c][0] = fma2(make_float2(exp2_fast(far * a.v[c][0].x), exp2_fast(far * a.v[c][0].y)), make_float2(in * b.x, in * b.y), h.v[c][0]);
        h.v[c][1] = fma2(make_float2(exp2_fast(far * a.v[c][1].x), exp2_fast(far * a.v[c][1].y)), make_float2(in * b.z, in * b.w), h.v[c][1]);
      }
      here = add2(here, make_float2(s.x, s.z));
    }
    behind = add2(behind, here);
  }
  if (ch < P.left) {
    const long long at = (long long)(P.r * W.segments + P.seg) * A.D + d;
    h.store(W.states, at, N, q, both);
    if (lane == 0) {
      W.sums[at] = behind.x;
      if (both) W.sums[at + 1] = behind.y;
    }
  }
}

// Walks the segments of four states: what is behind one enters the next.
template <int N>
__global__ void __launch_bounds__(kScanThreads) scan_join_kernel(const ScanArgs A, const ScanSplit W) {
  constexpr int L = N / 4;
  const long long i = (long long)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= (long long)A.D * L) return;
  const int d = (int)(i / L), q = (int)(i % L) * 4, r = blockIdx.y;
  const MixerRow R = mixer_row(A, r, false);
  const float4 av = *reinterpret_cast<const float4*>(A.a + (long long)d * N + q);
  const float2 a[2] = {mul2(make_float2(av.x, av.y), both_of(kLog2e)), mul2(make_float2(av.z, av.w), both_of(kLog2e))};
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
  if (R.from >= 0) h = *reinterpret_cast<const float4*>(A.state + ((long long)R.from * A.D + d) * N + q);
#pragma unroll 4
  for (int s = 0; s < W.segments; ++s) {
    const long long at = (long long)(r * W.segments + s) * A.D + d;
    float4* const p = reinterpret_cast<float4*>(W.states + at * N + q);
    const float4 put = *p;
    const float sum = W.sums[at];
    *p = h;
    const float2 k0 = scan_decay(mul2(both_of(sum), a[0])), k1 = scan_decay(mul2(both_of(sum), a[1]));
    h = make_float4(fmaf(k0.x, h.x, put.x), fmaf(k0.y, h.y, put.y), fmaf(k1.x, h.z, put.z), fmaf(k1.y, h.w, put.w));
  }
}

constexpr int kScanStepTokens = 16;    // up to so many are walked by scan_step_kernel
#ifndef SPEC_SCAN_FILL
#define SPEC_SCAN_FILL 600
#endif

static int scan_blocks(int D, int each, int N) {
  const int ch = kScanThreads / (N / 4) * kScanPair;
  return (each + ch - 1) / ch * (D / each);
}

// Into how many segments a row's tokens are split, so that there are CTAs for all SMs.
static int scan_segments(int B, int T, int D, int each, int N) {
  const long long ctas = (long long)scan_blocks(D, each, N) * B;
  const long long want = ctas >= SPEC_SCAN_FILL / 2 ? 1 : (SPEC_SCAN_FILL + ctas - 1) / ctas;
  return (int)std::max(1ll, std::min(want, (long long)T / 128));
}

// (the most segments that a call of these sizes may have, whatever its groups: one group has the fewest CTAs)
static size_t scan_split_bytes(int B, int T, int D, int N) {
  const size_t n = scan_segments(B, T, D, D, N);
  return n > 1 ? (n * B * D * 4 + 255) / 256 * 256 + n * B * D * N * 4 : 0;
}

template <bool BF16, int N, int VEC>
static int launch_tiles(const ScanArgs& A, bool pairs, char* workspace, cudaStream_t st) {
  using S = ScanShape<BF16, N, VEC>;
  const int blocks = scan_blocks(A.D, A.each, N);
  ScanSplit W;
  W.segments = scan_segments(A.B, A.T, A.D, A.each, N);
  W.span = ((A.T + W.segments - 1) / W.segments + kScanTile - 1) / kScanTile * kScanTile;
  W.segments = (A.T + W.span - 1) / W.span;
  W.sums = reinterpret_cast<float*>(workspace);
  W.states = reinterpret_cast<float*>(workspace + ((size_t)W.segments * A.B * A.D * 4 + 255) / 256 * 256);
  constexpr int smem = sizeof(ScanShared<N, S::CH, true>), less = sizeof(ScanShared<N, S::CH, false>);
  const dim3 grid((unsigned)blocks * W.segments, A.B);
  if (W.segments > 1) {
    scan_segment_kernel<BF16, N, VEC><<<grid, kScanThreads, less, st>>>(A, W, pairs);
    const dim3 joins((unsigned)(((long long)A.D * S::L + kScanThreads - 1) / kScanThreads), A.B);
    scan_join_kernel<N><<<joins, kScanThreads, 0, st>>>(A, W);
  }
  static std::atomic<unsigned long long> allowed[2];
  const auto gated = scan_tile_kernel<BF16, N, VEC, true>, plain = scan_tile_kernel<BF16, N, VEC, false>;
  if (!allow_shared(reinterpret_cast<const void*>(A.z ? gated : plain), smem, &allowed[A.z != nullptr])) return SPEC_E_CUDA;
  (A.z ? gated : plain)<<<grid, kScanThreads, smem, st>>>(A, W, pairs);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <bool BF16, int N>
static int launch_scan(const ScanArgs& A, bool wide, void* workspace, cudaStream_t st) {
  if (A.T > kScanStepTokens && !A.states) {
    constexpr int es = BF16 ? 2 : 4;
    // four channels, and pairs of states, by one access where they are aligned
    const bool four = A.each % 4 == 0 && (A.x_row | A.x_tok | A.dt_row | A.dt_tok | A.z_row | A.z_tok) % 4 == 0 &&
                      paged_aligned(A.x, 4 * es) && paged_aligned(A.dt, 4 * es) && paged_aligned(A.z, 4 * es) &&
                      paged_aligned(A.y, 4 * es) && paged_aligned(A.skip, 8) && paged_aligned(A.dt_bias, 8);
    const bool pairs = (A.b_row | A.b_tok | A.b_group | A.c_row | A.c_tok | A.c_group) % 2 == 0 && paged_aligned(A.b, 2 * es) &&
                       paged_aligned(A.c, 2 * es);
    char* const ws = static_cast<char*>(workspace);
    return four ? launch_tiles<BF16, N, 4>(A, pairs, ws, st) : launch_tiles<BF16, N, 1>(A, pairs, ws, st);
  }
  const dim3 grid((unsigned)(((long long)A.D * (N / 4) + kScanStepThreads - 1) / kScanStepThreads), A.B);
  scan_step_kernel<BF16, N><<<grid, kScanStepThreads, 0, st>>>(A, wide);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <bool BF16>
static int launch_scan_of(const ScanArgs& A, int N, bool wide, void* workspace, cudaStream_t st) {
  switch (N) {
    case 8: return launch_scan<BF16, 8>(A, wide, workspace, st);
    case 16: return launch_scan<BF16, 16>(A, wide, workspace, st);
    case 32: return launch_scan<BF16, 32>(A, wide, workspace, st);
    case 64: return launch_scan<BF16, 64>(A, wide, workspace, st);
    default: return launch_scan<BF16, 128>(A, wide, workspace, st);
  }
}

static bool scan_dims(int B, int T, int D, int N) {
  return B >= 0 && B <= 65535 && T >= 0 && T <= SPEC_MAX_LENGTH && D >= 1 && D <= (1 << 24) &&
         (N == 8 || N == 16 || N == 32 || N == 64 || N == 128);
}

}  // namespace specv

extern "C" size_t spec_scan_workspace_size(int B, int T, int D, int N) {
  if (!specv::scan_dims(B, T, D, N)) return 0;
  return std::max<size_t>(256, specv::scan_split_bytes(B, T, D, N));
}

extern "C" int spec_scan(const spec_scan_t* s, void* workspace, size_t workspace_bytes, void* cuda_stream) {
  using namespace specv;
  if (!s) return SPEC_E_NULL;
  const int rc = mixer_check(*s);
  if (rc != SPEC_OK) return rc;
  if (!scan_dims(s->B, s->T, s->D, s->N) || s->groups < 1 || s->D % s->groups) return SPEC_E_DIM;
  if (s->B == 0 || (s->T == 0 && !s->last)) return SPEC_OK;
  if (!s->a || !workspace || (s->T > 0 && (!s->x || !s->dt || !s->b || !s->c || !s->y))) return SPEC_E_NULL;
  const size_t es = s->dtype == SPEC_BF16 ? 2 : 4;
  for (const void* p : {s->x, s->dt, s->z, s->b, s->c, (const void*)s->y})
    if (!paged_aligned(p, es)) return SPEC_E_ALIGN;
  for (const float* p : {s->a, s->state, (const float*)s->states, (const float*)s->last})
    if (!paged_aligned(p, 16)) return SPEC_E_ALIGN;
  if (!paged_aligned(s->skip, 4) || !paged_aligned(s->dt_bias, 4) || !paged_aligned(workspace, 256)) return SPEC_E_ALIGN;
  if (workspace_bytes < spec_scan_workspace_size(s->B, s->T, s->D, s->N)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  ScanArgs A;
  A.x = s->x, A.dt = s->dt, A.z = s->z, A.b = s->b, A.c = s->c;
  A.a = s->a, A.skip = s->skip, A.dt_bias = s->dt_bias, A.state = s->state;
  A.slot = s->slot, A.lens = s->lens, A.y = s->y, A.states = s->states, A.last = s->last, A.last_slot = s->last_slot;
  A.flags = s->flags;
  A.x_row = s->x_row, A.x_tok = s->x_tok, A.dt_row = s->dt_row, A.dt_tok = s->dt_tok, A.z_row = s->z_row, A.z_tok = s->z_tok;
  A.b_row = s->b_row, A.b_tok = s->b_tok, A.b_group = s->b_group, A.c_row = s->c_row, A.c_tok = s->c_tok, A.c_group = s->c_group;
  A.B = s->B, A.T = s->T, A.D = s->D, A.each = s->D / s->groups, A.slots = s->slots, A.last_slots = s->last_slots;
  A.softplus = s->softplus != 0;
  // four states of b and c by one load where they are aligned
  const bool wide = paged_aligned(s->b, 4 * es) && paged_aligned(s->c, 4 * es) &&
                    (A.b_row | A.b_tok | A.b_group | A.c_row | A.c_tok | A.c_group) % 4 == 0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  return s->dtype == SPEC_BF16 ? launch_scan_of<true>(A, s->N, wide, workspace, st)
                              : launch_scan_of<false>(A, s->N, wide, workspace, st);
}
