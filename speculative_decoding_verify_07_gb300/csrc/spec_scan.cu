// spec_scan: h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t, y_t = c_t . h_t, for N
// states of each channel.
//
// A channel's states lie with neighbouring lanes, four or eight each, so that a warp reads
// and writes states side by side; the sum over the states goes through the lanes.
//
// A few tokens: one kernel, bound by the instructions of a warp's 16 channels (the
// states' bytes, one in and one out a token for the commit, would allow half the time:
// 64x3 tokens of 4096 channels by 16 states 26 us, 3300 GB/s).  Many tokens: tiles of
// tokens, see below; a long row is split where there are few channels.
//
// Measured, 16 states, bf16, gate and softplus: 4x2048 tokens x 4096 channels 213 us (537 M
// states, 2.5 T states a second), 16x1024x4096 360 us, 1x4096x4096 181 us (four
// segments), 1x32768x2048 631 us.
#include <algorithm>

#include "spec_mixer.cuh"
#include "spec_scan_split.h"
#include "spec_tma.cuh"

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

// ln(1 + exp(v)) within 12 half steps (2^-24) of itself where exp(v) is a normal number, and 0 below (v < -87.3): max(v, 0)
// + ln(1 + e), e = exp(-|v|), with the polynomial of degree 8 that is nearest to ln(1 + e) / e over [0, 1] (by Remez's
// method; 1.3e-7 of it off as evaluated here).
__device__ __forceinline__ float softplus(float v) {
  float pos;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(pos) : "f"(v));
  // exp(-m) with the roundings of log2(e) and of the product made up for (of 88 it is below 2^-126 and flushed to zero)
  const float m = fminf(fabsf(v), 88.f), p = m * -kLog2e, low = fmaf(m, -1.92596299e-8f, fmaf(m, -kLog2e, -p));
  const float e0 = exp2_fast(p), e = fmaf(e0, low * 0.6931471805599453f, e0);
  float t = 0x1.56ee0ap-8f;
  t = fmaf(t, e, -0x1.e369f2p-6f);
  t = fmaf(t, e, 0x1.4069dcp-4f);
  t = fmaf(t, e, -0x1.17d2c2p-3f);
  t = fmaf(t, e, 0x1.874a80p-3f);
  t = fmaf(t, e, -0x1.fcc8c6p-3f);
  t = fmaf(t, e, 0x1.553004p-2f);
  t = fmaf(t, e, -0x1.fffeacp-2f);
  t = fmaf(t, e, 0x1.fffffep-1f);
  return fmaf(t, e, pos);
}

// a in powers of two.  What is below every number is the lowest, so that a step of zero, of a tile's last tokens or of a part
// without any, leaves the state of a = -inf too.
__device__ __forceinline__ float scan_rate(float a) {
  float r;
  asm("max.NaN.f32 %0, %1, 0fFF7FFFFF;" : "=f"(r) : "f"(a * kLog2e));
  return r;
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

constexpr int kScanStepThreads = 128, kScanStepCtas = 5;      // an SM: with 4 and 8 the verify step took 5 and 20 % longer

template <int N>
struct Count {
  static constexpr int value = N;
};

// Each of a channel's lanes has four states, or twice four, so far apart that the lanes' lie side by side.
template <int N>
struct ScanStep {
  static constexpr int chunks = N == 8 ? 1 : 2, L = N / 4 / chunks;
};

// Four tokens at a time: each of a channel's lanes fetches one token's inputs (two where there are two lanes), and
// the lanes hand them to one another.
template <bool BF16, int N>
__global__ void __launch_bounds__(kScanStepThreads, kScanStepCtas) scan_step_kernel(const ScanArgs A, bool wide) {
  constexpr int L = ScanStep<N>::L, CK = ScanStep<N>::chunks, own = L == 2 ? 2 : 1;
  const long long i = (long long)blockIdx.x * kScanStepThreads + threadIdx.x;
  const bool mine = i < (long long)A.D * L;      // (lanes beyond the last channel follow its sums)
  const int d = mine ? (int)(i / L) : A.D - 1, lane = (int)(i % L), q = lane * 4, j0 = scan_token<L>(lane), r = blockIdx.y;
  const MixerRow R = mixer_row(A, r, i == 0);
  const int g = A.each == A.D ? 0 : d / A.each, at = d * N + q;      // (D N is below 2^31)
  const long long xb = r * A.x_row + d, db = r * A.dt_row + d, zb = r * A.z_row + d;
  const long long bb = r * A.b_row + g * A.b_group + q, cb = r * A.c_row + g * A.c_group + q;
  const long long out = (long long)r * A.T * A.D, states = out * N + at;
  const float skip = A.skip ? __ldg(A.skip + d) : 0.f, bias = A.dt_bias ? __ldg(A.dt_bias + d) : 0.f;
  float2 a[CK][2], h[CK][2];
#pragma unroll
  for (int m = 0; m < CK; ++m) {
    const float4 av = __ldg(reinterpret_cast<const float4*>(A.a + at + m * 4 * L));
    a[m][0] = make_float2(scan_rate(av.x), scan_rate(av.y));
    a[m][1] = make_float2(scan_rate(av.z), scan_rate(av.w));
    h[m][0] = h[m][1] = make_float2(0.f, 0.f);
    if (R.from >= 0) {
      const float4 s = *reinterpret_cast<const float4*>(A.state + (long long)R.from * A.D * N + at + m * 4 * L);
      h[m][0] = make_float2(s.x, s.y);
      h[m][1] = make_float2(s.z, s.w);
    }
  }
  // (a run of tokens has no branch inside, so that their chains of latencies lie side by side)
  auto run = [&](int t0, auto tokens) {
    constexpr int left = decltype(tokens)::value;
    float x[own], z[own], delta[2] = {0.f, 0.f}, put[own];
    ScanFour<BF16> b[left][CK], c[left][CK];
#pragma unroll
    for (int k = 0; k < own; ++k) {
      const int t = t0 + min(j0 + k, left - 1);
      x[k] = load_one<BF16>(A.x, xb + t * A.x_tok);
      delta[k] = load_one<BF16>(A.dt, db + t * A.dt_tok) + bias;
      z[k] = A.z ? load_one<BF16>(A.z, zb + t * A.z_tok) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < left; ++k) {
#pragma unroll
      for (int m = 0; m < CK; ++m) {
        b[k][m].load(A.b, bb + (t0 + k) * A.b_tok + m * 4 * L, wide);
        c[k][m].load(A.c, cb + (t0 + k) * A.c_tok + m * 4 * L, wide);
      }
    }
#pragma unroll
    for (int k = 0; k < own; ++k) {
      if (A.softplus) delta[k] = softplus(delta[k]);
      put[k] = delta[k] * x[k];
    }
    float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < left; ++k) {
      // the lane of the channel that has token k: scan_token's inverse
      const int from = L == 2 ? k >> 1 : (k >> 1) + (k & 1) * 2, which = L == 2 ? k & 1 : 0;
      const float2 step = both_of(__shfl_sync(0xffffffffu, which ? delta[1] : delta[0], from, L));
      const float2 in = both_of(__shfl_sync(0xffffffffu, put[own > 1 ? which : 0], from, L));
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int m = 0; m < CK; ++m) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          h[m][j] = fma2(scan_decay(mul2(step, a[m][j])), h[m][j], mul2(in, b[k][m].get(j)));
          sum = fma2(c[k][m].get(j), h[m][j], sum);
        }
        if (A.states && mine)
          __stcs(reinterpret_cast<float4*>(A.states + states + (long long)(t0 + k) * A.D * N + m * 4 * L),
                 make_float4(h[m][0].x, h[m][0].y, h[m][1].x, h[m][1].y));
      }
      y[k] = sum.x + sum.y;
    }
    scan_sum<L>(y, lane);
#pragma unroll
    for (int k = 0; k < own; ++k) {
      if (mine && j0 + k < left && lane < 4) {
        float v = fmaf(skip, x[k], y[k]);
        if (A.z) v *= silu(z[k]);
        store_one<BF16>(A.y, out + (long long)(t0 + j0 + k) * A.D + d, v);
      }
    }
  };
  int t0 = 0;
#pragma unroll 1
  for (; t0 + 4 <= R.len; t0 += 4) run(t0, Count<4>());
  if (R.len - t0 == 3) run(t0, Count<3>());
  if (R.len - t0 == 2) run(t0, Count<2>());
  if (R.len - t0 == 1) run(t0, Count<1>());
  if (!mine) return;
  for (int t = R.len; t < A.T; ++t) {
    if (lane == 0) store_one<BF16>(A.y, out + (long long)t * A.D + d, 0.f);
    if (A.states)
#pragma unroll
      for (int m = 0; m < CK; ++m)
        __stcs(reinterpret_cast<float4*>(A.states + states + (long long)t * A.D * N + m * 4 * L), make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (R.to >= 0)
#pragma unroll
    for (int m = 0; m < CK; ++m)
      *reinterpret_cast<float4*>(A.last + (long long)R.to * A.D * N + at + m * 4 * L) = make_float4(h[m][0].x, h[m][0].y, h[m][1].x, h[m][1].y);
}

// --------------------------------------------------------------- many tokens
//
// A CTA walks tiles of tokens of its channels, with two halves of its warps one behind the
// other.  One half makes delta, delta x, b and c of a tile in shared memory.  The other takes
// it from there, a lane two channels by four states, through the tile's tokens and leaves each
// lane's part of the sums.  The first then goes through the tile's elements again (the sum,
// skip, gate, output).
//
// Bound by issue slots (busy in 54 % of the cycles, 63 % where an SM has work), the multiply-add
// pipe (57 %) and the walk's loads from shared memory (64 %), which take turns: the walk alone,
// without the elements, took 160 of 215 us, and with neither loads nor exponentials still 124.
// Both halves by the same warps 252 us; four channels a lane 300 (half the warps); 16-bit b and c
// unpacked by the walk 222.
//
// Decays are ex2.approx alone here, whose lean to one side (see scan_decay) would add up over
// the tokens that a state remembers.  So the tile's decays are also multiplied, and at its end
// the state that entered gets the difference to the exact decay of the tile's sum of delta.

constexpr int kScanGroup = 8;          // tokens that a lane takes together

template <bool BF16, int N, int VEC>
struct ScanShape {
  static constexpr int L = N / 4;                              // lanes of a channel
  static constexpr int CH = kScanThreads / L * kScanLane;      // channels of a CTA
  static constexpr int vecs = CH / VEC;                        // a token's channels, VEC at a time
  static constexpr int rows = kScanThreads / vecs;             // tokens of a fetch
  static constexpr int per = rows > kScanTile ? 1 : kScanTile / rows;
  static constexpr int bc_rows = kScanThreads / (N / 2);       // the same of pairs of states of b and c
  static constexpr int bc = bc_rows > kScanTile ? 1 : kScanTile / bc_rows;
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
  __device__ __forceinline__ float get(int i) const {
    if (BF16) return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    return __uint_as_float(w[BF16 ? 0 : i]);
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
  struct Tile {
    float4 step[kScanTile][CH / 2];              // (delta, delta, delta x, delta x) of two channels
    float b[kScanTile][N], c[Y ? kScanTile : 1][N];
    // each lane's parts of the sums of its two channels; rows are so far apart that a warp's 256 bytes meet no bank more
    // than twice
    float2 part[Y ? kScanTile : 1][N / 4][CH / 2 + (N < 128 ? 128 / N : 2)];
  } tile[2];
  float bias[CH], skip[Y ? CH : 1];

  __device__ __forceinline__ static void fill(float* to, const float* p, const ScanPlace& P) {
    for (int c = threadIdx.x; c < CH; c += 2 * kScanThreads) to[c] = p && c < P.left ? __ldg(p + P.d0 + c) : 0.f;
  }
};

// The halves' barriers, one of each for either buffer: a tile is made, a tile has been walked.
constexpr int kScanMade = 1, kScanWalked = 3;
template <int ID>
__device__ __forceinline__ void scan_wait(bool second) {
  if (second) asm volatile("bar.sync %0, 256;" ::"n"(ID + 1) : "memory");
  else asm volatile("bar.sync %0, 256;" ::"n"(ID) : "memory");
}
template <int ID>
__device__ __forceinline__ void scan_tell(bool second) {
  if (second) asm volatile("bar.arrive %0, 256;" ::"n"(ID + 1) : "memory");
  else asm volatile("bar.arrive %0, 256;" ::"n"(ID) : "memory");
}

// A tile's elements on their way, and where this thread's lie.
template <bool BF16, int N, int VEC, bool Y, bool GATE>
struct ScanFetch {
  using S = ScanShape<BF16, N, VEC>;
  using Shared = ScanShared<N, S::CH, Y>;
  using Tile = typename Shared::Tile;
  static constexpr int es = BF16 ? 2 : 4;
  ScanVec<BF16, VEC> x[S::per], dt[S::per], z[GATE ? S::per : 1];
  ScanVec<BF16, 2> b[S::bc], c[Y ? S::bc : 1];
  const unsigned char *px, *pdt, *pz, *pb, *pc;    // of this thread's first element in the row's first tile

  // The i-th fetch's token of the tile, and its first channel.
  static __device__ __forceinline__ int token(int i) { return threadIdx.x % kScanThreads / S::vecs + i * S::rows; }
  static __device__ __forceinline__ int channel() { return threadIdx.x % S::vecs * VEC; }
  static __device__ __forceinline__ bool real(int i) { return S::rows <= kScanTile || token(i) < kScanTile; }
  // The same of b and c: a pair of states.
  static __device__ __forceinline__ int bc_token(int i) { return threadIdx.x % kScanThreads / (N / 2) + i * S::bc_rows; }
  static __device__ __forceinline__ int bc_state() { return threadIdx.x % (N / 2) * 2; }
  static __device__ __forceinline__ bool bc_real(int i) { return S::bc_rows <= kScanTile || bc_token(i) < kScanTile; }

  __device__ __forceinline__ ScanFetch(const ScanArgs& A, const ScanPlace& P) {
    const int c = P.d0 + channel(), t = token(0);
    px = static_cast<const unsigned char*>(A.x) + (P.r * A.x_row + t * A.x_tok + c) * es;
    pdt = static_cast<const unsigned char*>(A.dt) + (P.r * A.dt_row + t * A.dt_tok + c) * es;
    if (GATE) pz = static_cast<const unsigned char*>(A.z) + (P.r * A.z_row + t * A.z_tok + c) * es;
    pb = static_cast<const unsigned char*>(A.b) + (P.r * A.b_row + P.g * A.b_group + bc_token(0) * A.b_tok + bc_state()) * es;
    if (Y) pc = static_cast<const unsigned char*>(A.c) + (P.r * A.c_row + P.g * A.c_group + bc_token(0) * A.c_tok + bc_state()) * es;
  }
  __device__ __forceinline__ void load(const ScanArgs& A, const ScanPlace& P, int t0, int end, bool pairs) {
    const int rows = end - t0;
    const unsigned char *qx = px + t0 * A.x_tok * es, *qdt = pdt + t0 * A.dt_tok * es, *qz = pz;
    if (GATE) qz += t0 * A.z_tok * es;
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      x[i].zero(), dt[i].zero();
      if (GATE) z[GATE ? i : 0].zero();
      if (real(i) && token(i) < rows && channel() < P.left) {
        x[i].load(qx + i * (S::rows * es) * A.x_tok);
        dt[i].load(qdt + i * (S::rows * es) * A.dt_tok);
        if (GATE) z[GATE ? i : 0].load(qz + i * (S::rows * es) * A.z_tok);
      }
    }
    const unsigned char *qb = pb + t0 * A.b_tok * es, *qc = pc;
    if (Y) qc += t0 * A.c_tok * es;
#pragma unroll
    for (int i = 0; i < S::bc; ++i) {
      b[i].zero();
      if (Y) c[Y ? i : 0].zero();
      if (bc_real(i) && bc_token(i) < rows) {
        get(b[i], qb + i * (S::bc_rows * es) * A.b_tok, pairs);
        if (Y) get(c[Y ? i : 0], qc + i * (S::bc_rows * es) * A.c_tok, pairs);
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
  __device__ __forceinline__ void put(const ScanArgs& A, const ScanPlace& P, int t0, int end, const float* bias, Tile& sm) const {
#pragma unroll
    for (int i = 0; i < S::per; ++i) {
      if (!real(i)) continue;
      const int at = channel();
      const bool there = token(i) < end - t0 && at < P.left;
      float delta[VEC], in[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        delta[v] = dt[i].get(v) + bias[at + v];
        if (A.softplus) delta[v] = softplus(delta[v]);
        if (!there) delta[v] = 0.f;
        in[v] = delta[v] * x[i].get(v);
      }
      float4* const to = &sm.step[token(i)][at / 2];
      if (VEC == 1) {
        float* const one = reinterpret_cast<float*>(to) + at % 2;
        one[0] = delta[0];
        one[2] = in[0];
      }
#pragma unroll
      for (int v = 0; v + 1 < VEC; v += 2) to[v / 2] = make_float4(delta[v], delta[VEC > 1 ? v + 1 : 0], in[v], in[VEC > 1 ? v + 1 : 0]);
    }
#pragma unroll
    for (int i = 0; i < S::bc; ++i) {
      if (!bc_real(i)) continue;
      *reinterpret_cast<float2*>(&sm.b[bc_token(i)][bc_state()]) = make_float2(b[i].get(0), b[i].get(1));
      if (Y) *reinterpret_cast<float2*>(&sm.c[Y ? bc_token(i) : 0][bc_state()]) = make_float2(c[Y ? i : 0].get(0), c[Y ? i : 0].get(1));
    }
  }
};

// A lane's four states of two channels, side by side.
struct ScanStates {
  float2 v[4];
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = both_of(x);
  }
  // channel d of `p`, [channel][N], from state q on, and the next one where there is one
  __device__ __forceinline__ void load(const float* p, long long d, int N, int q, bool both) {
    const float4 x = *reinterpret_cast<const float4*>(p + d * N + q), y = *reinterpret_cast<const float4*>(p + (d + (both ? 1 : 0)) * N + q);
    v[0] = make_float2(x.x, y.x);
    v[1] = make_float2(x.y, y.y);
    v[2] = make_float2(x.z, y.z);
    v[3] = make_float2(x.w, y.w);
  }
  __device__ __forceinline__ void store(float* p, long long d, int N, int q, bool both) const {
    *reinterpret_cast<float4*>(p + d * N + q) = make_float4(v[0].x, v[1].x, v[2].x, v[3].x);
    if (both) *reinterpret_cast<float4*>(p + (d + 1) * N + q) = make_float4(v[0].y, v[1].y, v[2].y, v[3].y);
  }
  __device__ __forceinline__ void rates() {
#pragma unroll
    for (int n = 0; n < 4; ++n) v[n] = make_float2(scan_rate(v[n].x), scan_rate(v[n].y));
  }
};

template <bool BF16, int N, int VEC, bool GATE>
__global__ void __launch_bounds__(2 * kScanThreads, kScanCtas) scan_tile_kernel(const ScanArgs A, const ScanSplit W, bool pairs) {
  using S = ScanShape<BF16, N, VEC>;
  using F = ScanFetch<BF16, N, VEC, true, GATE>;
  using Shared = ScanShared<N, S::CH, true>;
  constexpr int L = S::L, CH = S::CH;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const ScanPlace P = scan_place(A, CH);
  const MixerRow R = mixer_row(A, P.r, P.seg == 0 && P.d0 == 0 && threadIdx.x == 0);
  const int first = P.seg * W.span, stop = (int)min((long long)first + W.span, (long long)A.T), end = min(stop, R.len);
  const int tiles = first < end ? (end - first + kScanTile - 1) / kScanTile : 0;
  const long long out = (long long)P.r * A.T * A.D + P.d0;
  sm.fill(sm.bias, A.dt_bias, P);
  sm.fill(sm.skip, A.skip, P);
  if (threadIdx.x >= kScanThreads) {
    // ------------------------------------------------------ the elements
    F in(A, P);
    if (tiles) in.load(A, P, first, end, pairs);
    // of the tiles that are being walked (single elements would be too many, and are fetched again)
    constexpr bool hold = VEC > 1;
    ScanVec<BF16, VEC> x[2][hold ? S::per : 1], z[2][hold && GATE ? S::per : 1];
    __syncthreads();
    for (int k0 = 0; k0 < tiles + 2; k0 += 2)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int k = k0 + u;
        if (k >= 2 && k - 2 < tiles) {
          scan_wait<kScanWalked>(u);
          const int t0 = first + (k - 2) * kScanTile;
#pragma unroll
          for (int i = 0; i < S::per; ++i) {
            const int t = F::token(i), at = F::channel();
            if (!F::real(i) || t >= end - t0 || at >= P.left) continue;
            // the lanes' parts, of VEC channels at a time
            float y[VEC], two[VEC];
#pragma unroll
            for (int m = 0; m < L; ++m) {
              float e[VEC];
              const float* const p = reinterpret_cast<const float*>(&sm.tile[u].part[t][m][0]) + at;
              if (VEC > 1) *reinterpret_cast<float4*>(e) = *reinterpret_cast<const float4*>(p);
              else e[0] = p[0];
#pragma unroll
              for (int v = 0; v < VEC; ++v) {
                if (m % 2 == 0) two[v] = e[v];
                else y[v] = m > 1 ? y[v] + (two[v] + e[v]) : two[v] + e[v];
              }
            }
            if (!hold) {
              x[u][0].load(in.px + (t0 + (long long)i * S::rows) * A.x_tok * F::es);
              if (GATE) z[u][0].load(in.pz + (t0 + (long long)i * S::rows) * A.z_tok * F::es);
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
              y[v] = fmaf(sm.skip[at + v], x[u][hold ? i : 0].get(v), y[v]);
              if (GATE) y[v] *= silu(z[u][hold && GATE ? i : 0].get(v));
            }
            const long long to = out + (long long)(t0 + t) * A.D + at;
            constexpr int n1 = VEC > 1 ? 1 : 0, n2 = VEC > 1 ? 2 : 0, n3 = VEC > 1 ? 3 : 0;
            if (VEC == 1) store_one<BF16>(A.y, to, y[0]);
            else if (BF16) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(A.y) + to) = make_uint2(pack_bf16(y[0], y[n1]), pack_bf16(y[n2], y[n3]));
            else *reinterpret_cast<float4*>(static_cast<float*>(A.y) + to) = make_float4(y[0], y[n1], y[n2], y[n3]);
          }
        }
        if (k < tiles) {
          const int t0 = first + k * kScanTile;
          in.put(A, P, t0, end, sm.bias, sm.tile[u]);
#pragma unroll
          for (int i = 0; i < (hold ? S::per : 0); ++i) {
            x[u][i] = in.x[i];
            if (GATE) z[u][GATE ? i : 0] = in.z[GATE ? i : 0];
          }
          scan_tell<kScanMade>(u);
          if (k + 1 < tiles) in.load(A, P, t0 + kScanTile, end, pairs);
        }
      }
    for (long long i = (long long)max(first, R.len) * P.left + threadIdx.x % kScanThreads; i < (long long)stop * P.left; i += kScanThreads)
      store_one<BF16>(A.y, out + i / P.left * A.D + i % P.left, 0.f);
  } else {
    // -------------------------------------------------------- the states
    const int ch = threadIdx.x / L * kScanLane, lane = threadIdx.x % L, q = lane * 4, d = P.d0 + min(ch, P.left - 1);
    const bool both = ch + 1 < P.left;      // (lanes without channels follow the last one)
    ScanStates a, h;
    a.load(A.a, d, N, q, both);
    a.rates();
    h.fill(0.f);
    if (W.segments > 1) h.load(W.states, ((long long)P.r * W.segments + P.seg) * W.fine * A.D + d, N, q, both);
    else if (R.from >= 0) h.load(A.state, (long long)R.from * A.D + d, N, q, both);
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      typename Shared::Tile& tile = sm.tile[k & 1];
      scan_wait<kScanMade>(k & 1);
      const ScanStates was = h;
      ScanStates all;
      all.fill(1.f);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int t = 0; t < kScanTile; t += kScanGroup) {
        // (loads first, then the arithmetic of all tokens, then stores, which the compiler moves no load across)
        float4 s[kScanGroup], b[kScanGroup], c[kScanGroup];
        float2 y[kScanGroup];
#pragma unroll
        for (int j = 0; j < kScanGroup; ++j) {
          s[j] = tile.step[t + j][ch / 2];
          b[j] = *reinterpret_cast<const float4*>(&tile.b[t + j][q]);
          c[j] = *reinterpret_cast<const float4*>(&tile.c[t + j][q]);
        }
#pragma unroll
        for (int j = 0; j < kScanGroup; ++j) {
          const float bb[4] = {b[j].x, b[j].y, b[j].z, b[j].w}, cc[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
          const float2 step = make_float2(s[j].x, s[j].y), put = make_float2(s[j].z, s[j].w);
          sum = add2(sum, step);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float2 e = mul2(step, a.v[n]), w = make_float2(exp2_fast(e.x), exp2_fast(e.y));
            all.v[n] = mul2(all.v[n], w);
            h.v[n] = fma2(w, h.v[n], mul2(put, both_of(bb[n])));
            y[j] = n ? fma2(both_of(cc[n]), h.v[n], y[j]) : mul2(both_of(cc[n]), h.v[n]);
          }
        }
#pragma unroll
        for (int j = 0; j < kScanGroup; ++j) tile.part[t + j][lane][ch / 2] = y[j];
      }
      scan_tell<kScanWalked>(k & 1);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const float2 w = scan_decay(mul2(sum, a.v[n])), u = was.v[n];
        // (a state that is not finite stays what it has become)
        const float2 s = make_float2(fabsf(u.x) < INFINITY ? u.x : 0.f, fabsf(u.y) < INFINITY ? u.y : 0.f);
        h.v[n] = fma2(add2(w, make_float2(-all.v[n].x, -all.v[n].y)), s, h.v[n]);
      }
    }
    // the segment of the last token has the last state
    if (ch < P.left && R.to >= 0 && (W.segments == 1 || (R.len > 0 ? first < R.len && R.len <= stop : P.seg == 0)))
      h.store(A.last, (long long)R.to * A.D + d, N, q, both);
  }
}

// The state behind a segment that begins with zeros, from its last token to the first:
// sum_t exp(a (delta of the tokens after t)) delta_t x_t b_t.  Each weight is taken by
// itself, so nothing adds up.
template <bool BF16, int N, int VEC>
__global__ void __launch_bounds__(2 * kScanThreads) scan_segment_kernel(const ScanArgs A, const ScanSplit W, bool pairs) {
  using S = ScanShape<BF16, N, VEC>;
  using Shared = ScanShared<N, S::CH, false>;
  constexpr int L = S::L, CH = S::CH;
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const ScanPlace P = scan_place(A, CH);
  const MixerRow R = mixer_row(A, P.r, false);
  const int span = W.span / W.fine, first = P.seg * span, end = min((int)min((long long)first + span, (long long)A.T), R.len);
  const int tiles = first < end ? (end - first + kScanTile - 1) / kScanTile : 0;
  sm.fill(sm.bias, A.dt_bias, P);
  if (threadIdx.x >= kScanThreads) {
    ScanFetch<BF16, N, VEC, false, false> in(A, P);
    if (tiles) in.load(A, P, first + (tiles - 1) * kScanTile, end, pairs);
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      const int t0 = first + (tiles - 1 - k) * kScanTile;
      if (k >= 2) scan_wait<kScanWalked>(k & 1);
      in.put(A, P, t0, end, sm.bias, sm.tile[k & 1]);
      scan_tell<kScanMade>(k & 1);
      if (k + 1 < tiles) in.load(A, P, t0 - kScanTile, end, pairs);
    }
    // (what is told is also waited for)
    if (tiles >= 2) scan_wait<kScanWalked>(tiles & 1);
    if (tiles >= 1) scan_wait<kScanWalked>((tiles - 1) & 1);
  } else {
    const int ch = threadIdx.x / L * kScanLane, lane = threadIdx.x % L, q = lane * 4, d = P.d0 + min(ch, P.left - 1);
    const bool both = ch + 1 < P.left;
    ScanStates a, h;
    a.load(A.a, d, N, q, both);
    a.rates();
    h.fill(0.f);
    float2 behind = make_float2(0.f, 0.f);           // the delta of the tiles behind this one
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < tiles; ++k) {
      const typename Shared::Tile& tile = sm.tile[k & 1];
      scan_wait<kScanMade>(k & 1);
      float2 here = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int t = kScanTile - 1; t >= 0; --t) {
        const float4 b = *reinterpret_cast<const float4*>(&tile.b[t][q]), s = tile.step[t][ch / 2];
        const float bb[4] = {b.x, b.y, b.z, b.w};
        const float2 far = add2(behind, here), put = make_float2(s.z, s.w);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float2 e = mul2(far, a.v[n]);
          h.v[n] = fma2(make_float2(exp2_fast(e.x), exp2_fast(e.y)), mul2(put, both_of(bb[n])), h.v[n]);
        }
        here = add2(here, make_float2(s.x, s.y));
      }
      scan_tell<kScanWalked>(k & 1);
      behind = add2(behind, here);
    }
    if (ch < P.left) {
      const long long at = ((long long)P.r * W.segments * W.fine + P.seg) * A.D + d;
      h.store(W.states, at, N, q, both);
      if (lane == 0) {
        W.sums[at] = behind.x;
        if (both) W.sums[at + 1] = behind.y;
      }
    }
  }
}

// k h + put, k = exp2(y) of many tokens: an infinite h stays what it is, as it does token by token, where no decay is rounded
// to zero though all of them together are.
__device__ __forceinline__ float scan_enter(float k, float y, float h, float put) {
  return fmaf(k == 0.f && y > -INFINITY && fabsf(h) == INFINITY ? 1.f : k, h, put);
}

// What scan_segment_kernel left of a part's four states, anew, for a part where that is not finite: an infinite term stays in
// the sum although its weight is rounded to zero.  (From memory and by the join: a look at each tile in the first pass cost it
// a CTA an SM, 1x32768x2048 658 us.)
template <bool BF16>
__device__ __noinline__ float4 scan_again(const ScanArgs& A, int r, int d, long long b, float4 a, int first, int end) {
  const float bias = A.dt_bias ? __ldg(A.dt_bias + d) : 0.f;
  float behind = 0.f, here = 0.f;
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int t = end - 1; t >= first; --t) {
    float delta = load_one<BF16>(A.dt, r * A.dt_row + t * A.dt_tok + d) + bias;
    if (A.softplus) delta = softplus(delta);
    const float far = behind + here, in = delta * load_one<BF16>(A.x, r * A.x_row + t * A.x_tok + d);
    auto add = [&](float& to, float rate, int n) {
      const float e = far * rate;
      to = scan_enter(exp2_fast(e), e, in * load_one<BF16>(A.b, b + t * A.b_tok + n), to);
    };
    add(h.x, a.x, 0), add(h.y, a.y, 1), add(h.z, a.z, 2), add(h.w, a.w, 3);
    here += delta;
    // (summed up tile by tile, as there)
    if ((t - first) % kScanTile == 0) behind += here, here = 0.f;
    if (h.x != h.x && h.y != h.y && h.z != h.z && h.w != h.w) break;
  }
  return h;
}

// Walks the parts of four states, eight parts' loads at a time: what is behind one enters the next.  (1x32768x2048 631 us in
// all, 646 with a part's loads behind the last one's store.)
template <bool BF16, int N>
__global__ void __launch_bounds__(kScanThreads) scan_join_kernel(const ScanArgs A, const ScanSplit W) {
  constexpr int L = N / 4, ahead = 8;
  const long long i = (long long)blockIdx.x * kScanThreads + threadIdx.x;
  if (i >= (long long)A.D * L) return;
  const int d = (int)(i / L), q = (int)(i % L) * 4, r = blockIdx.y, parts = W.segments * W.fine, span = W.span / W.fine;
  const MixerRow R = mixer_row(A, r, false);
  const float4 av = *reinterpret_cast<const float4*>(A.a + (long long)d * N + q);
  const float4 a = make_float4(scan_rate(av.x), scan_rate(av.y), scan_rate(av.z), scan_rate(av.w));
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
  if (R.from >= 0) h = *reinterpret_cast<const float4*>(A.state + ((long long)R.from * A.D + d) * N + q);
  auto finite = [](float4 v) { return fabsf((v.x + v.y) + (v.z + v.w)) < INFINITY; };
#pragma unroll 1
  for (int s0 = 0; s0 < parts; s0 += ahead) {
    float4 put[ahead];
    float sum[ahead];
    bool odd = false;
#pragma unroll
    for (int j = 0; j < ahead; ++j) {
      const long long at = ((long long)r * parts + min(s0 + j, parts - 1)) * A.D + d;
      put[j] = *reinterpret_cast<const float4*>(W.states + at * N + q);
      sum[j] = W.sums[at];
    }
#pragma unroll
    for (int j = 0; j < ahead; ++j) odd = odd || !finite(put[j]);
#pragma unroll
    for (int j = 0; j < ahead; ++j) {
      if (s0 + j >= parts) break;
      if (odd && !finite(put[j])) {
        const int first = (s0 + j) * span, end = min((int)min((long long)first + span, (long long)A.T), R.len);
        put[j] = scan_again<BF16>(A, r, d, r * A.b_row + d / A.each * A.b_group + q, a, first, end);
      }
      *reinterpret_cast<float4*>(W.states + (((long long)r * parts + s0 + j) * A.D + d) * N + q) = h;
      const float2 y0 = mul2(both_of(sum[j]), make_float2(a.x, a.y)), y1 = mul2(both_of(sum[j]), make_float2(a.z, a.w));
      const float2 k0 = scan_decay(y0), k1 = scan_decay(y1);
      h = make_float4(scan_enter(k0.x, y0.x, h.x, put[j].x), scan_enter(k0.y, y0.y, h.y, put[j].y),
                      scan_enter(k1.x, y1.x, h.z, put[j].z), scan_enter(k1.y, y1.y, h.w, put[j].w));
    }
  }
}

constexpr int kScanStepTokens = 16;    // up to so many are walked by scan_step_kernel

template <bool BF16, int N, int VEC>
static int launch_tiles(const ScanArgs& A, bool pairs, char* workspace, cudaStream_t st) {
  using S = ScanShape<BF16, N, VEC>;
  const int blocks = scan_blocks(A.D, A.each, N);
  ScanSplit W = scan_split(A.B, A.T, A.D, A.each, N);
  W.sums = reinterpret_cast<float*>(workspace);
  W.states = reinterpret_cast<float*>(workspace + scan_states_at(scan_parts(W, A.B), A.D));
  constexpr int smem = sizeof(ScanShared<N, S::CH, true>), less = sizeof(ScanShared<N, S::CH, false>);
  const dim3 grid((unsigned)blocks * W.segments, A.B);
  if (W.segments > 1) {
    static std::atomic<unsigned long long> allowed;
    if (!allow_shared(reinterpret_cast<const void*>(scan_segment_kernel<BF16, N, VEC>), less, &allowed)) return SPEC_E_CUDA;
    scan_segment_kernel<BF16, N, VEC><<<dim3(grid.x * W.fine, A.B), 2 * kScanThreads, less, st>>>(A, W, pairs);
    const dim3 joins((unsigned)(((long long)A.D * S::L + kScanThreads - 1) / kScanThreads), A.B);
    scan_join_kernel<BF16, N><<<joins, kScanThreads, 0, st>>>(A, W);
  }
  static std::atomic<unsigned long long> allowed[2];
  const auto gated = scan_tile_kernel<BF16, N, VEC, true>, plain = scan_tile_kernel<BF16, N, VEC, false>;
  if (!allow_shared(reinterpret_cast<const void*>(A.z ? gated : plain), smem, &allowed[A.z != nullptr])) return SPEC_E_CUDA;
  (A.z ? gated : plain)<<<grid, 2 * kScanThreads, smem, st>>>(A, W, pairs);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <bool BF16, int N>
static int launch_scan(const ScanArgs& A, bool wide, void* workspace, cudaStream_t st) {
  if (A.T > kScanStepTokens && !A.states) {
    constexpr int es = BF16 ? 2 : 4;
    // four channels, and pairs of states, by one access where they are aligned
    const bool four = A.each % 4 == 0 && (A.x_row | A.x_tok | A.dt_row | A.dt_tok | A.z_row | A.z_tok) % 4 == 0 &&
                      paged_aligned(A.x, 4 * es) && paged_aligned(A.dt, 4 * es) && paged_aligned(A.z, 4 * es) &&
                      paged_aligned(A.y, 4 * es);
    const bool pairs = (A.b_row | A.b_tok | A.b_group | A.c_row | A.c_tok | A.c_group) % 2 == 0 && paged_aligned(A.b, 2 * es) &&
                       paged_aligned(A.c, 2 * es);
    char* const ws = static_cast<char*>(workspace);
    return four ? launch_tiles<BF16, N, 4>(A, pairs, ws, st) : launch_tiles<BF16, N, 1>(A, pairs, ws, st);
  }
  const dim3 grid((unsigned)(((long long)A.D * ScanStep<N>::L + kScanStepThreads - 1) / kScanStepThreads), A.B);
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
  return std::max<size_t>(256, specv::scan_bytes(specv::scan_parts_most(B, T, D, N), D, N));
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
