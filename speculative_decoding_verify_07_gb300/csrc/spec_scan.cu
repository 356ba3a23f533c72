// spec_scan: h_t = exp(delta_t a) h_{t-1} + delta_t x_t b_t, y_t = c_t . h_t, for N
// states of each channel.
//
// A channel's states lie with N / 4 neighbouring lanes, four each, so that a warp
// reads and writes 512 bytes of states side by side; the sum over the states goes
// through the lanes.
//
// A few tokens: bound by the states' bytes (one in, one out a token for the commit).
#include "spec_mixer.cuh"

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
__device__ __forceinline__ float softplus(float v) {
  const float pos = v < 0.f ? 0.f : v, m = fminf(fabsf(v), 87.f);
  // exp(-m) with the rounding of m log2(e) made up for
  const float p = -m * kLog2e, low = fmaf(-m, kLog2e, -p) - m * 1.92596299e-8f;
  const float e0 = exp2_fast(p), e = fmaf(e0, low * 0.6931471805599453f, e0);
  const float s = __fdividef(e, 2.f + e), q = s * s;
  float t = 1.f / 15.f;
  t = fmaf(t, q, 1.f / 13.f);
  t = fmaf(t, q, 1.f / 11.f);
  t = fmaf(t, q, 1.f / 9.f);
  t = fmaf(t, q, 1.f / 7.f);
  t = fmaf(t, q, 1.f / 5.f);
  t = fmaf(t, q, 1.f / 3.f);
  t = fmaf(t, q, 1.f);
  return fmaf(2.f * s, t, pos);
}

// exp(g) of two states, y = g log2(e).  An error of the decay adds up over the tokens that
// the state remembers, 1 / (1 - exp(g)) of them, and that of ex2.approx leans to one side
// (by 1e-8 to 3e-8 in the mean from 2^-1 down, measured), so below |g| = 1/32 the series to
// g^3 is taken instead.
__device__ __forceinline__ float2 scan_decay(float2 y) {
  constexpr float ln2 = 0.6931471805599453f;
  const float2 near = fma2(fma2(fma2(y, both_of(ln2 * ln2 * ln2 / 6.f), both_of(ln2 * ln2 / 2.f)), y, both_of(ln2)), y, both_of(1.f));
  const float2 a = make_float2(exp2_fast(y.x), exp2_fast(y.y));
  constexpr float border = 0.03125f / ln2;
  return make_float2(fabsf(y.x) < border ? near.x : a.x, fabsf(y.y) < border ? near.y : a.y);
}

// Four neighbouring states' b or c.
template <bool BF16>
__device__ __forceinline__ void load_four(const void* p, long long i, bool wide, float2* out) {
  if (BF16) {
    const uint16_t* q = static_cast<const uint16_t*>(p) + i;
    if (wide) {
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(q));
      out[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
      out[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
      return;
    }
  } else if (wide) {
    const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    out[0] = make_float2(w.x, w.y);
    out[1] = make_float2(w.z, w.w);
    return;
  }
  out[0] = make_float2(load_one<BF16>(p, i), load_one<BF16>(p, i + 1));
  out[1] = make_float2(load_one<BF16>(p, i + 2), load_one<BF16>(p, i + 3));
}

// ---------------------------------------------------------------- few tokens

constexpr int kScanStepThreads = 128;

template <bool BF16, int N, bool WIDE>
__global__ void __launch_bounds__(kScanStepThreads) scan_step_kernel(const ScanArgs A) {
  constexpr int L = N / 4;                       // lanes of a channel
  const int r = blockIdx.y;
  const long long i = (long long)blockIdx.x * kScanStepThreads + threadIdx.x;
  const bool mine = i < (long long)A.D * L;      // (lanes beyond the last channel follow its sums)
  const int d = mine ? (int)(i / L) : A.D - 1, q = (int)(i % L) * 4;
  const MixerRow R = mixer_row(A, r, i == 0);
  const int g = d / A.each;
  const float4 av = *reinterpret_cast<const float4*>(A.a + (long long)d * N + q);
  const float2 a[2] = {mul2(make_float2(av.x, av.y), both_of(kLog2e)), mul2(make_float2(av.z, av.w), both_of(kLog2e))};
  float2 h[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  if (R.from >= 0) {
    const float4 s = *reinterpret_cast<const float4*>(A.state + ((long long)R.from * A.D + d) * N + q);
    h[0] = make_float2(s.x, s.y);
    h[1] = make_float2(s.z, s.w);
  }
  const float skip = A.skip ? __ldg(A.skip + d) : 0.f, bias = A.dt_bias ? __ldg(A.dt_bias + d) : 0.f;
  const long long xb = r * A.x_row + d, db = r * A.dt_row + d, zb = r * A.z_row + d;
  const long long bb = r * A.b_row + g * A.b_group + q, cb = r * A.c_row + g * A.c_group + q;
  const long long out = (long long)r * A.T * A.D + d;
#pragma unroll 2
  for (int t = 0; t < R.len; ++t) {
    const float x = load_one<BF16>(A.x, xb + t * A.x_tok);
    float delta = load_one<BF16>(A.dt, db + t * A.dt_tok) + bias;
    float2 b[2], c[2];
    load_four<BF16>(A.b, bb + t * A.b_tok, WIDE, b);
    load_four<BF16>(A.c, cb + t * A.c_tok, WIDE, c);
    if (A.softplus) delta = softplus(delta);
    const float2 put = both_of(delta * x);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      h[j] = fma2(scan_decay(mul2(both_of(delta), a[j])), h[j], mul2(put, b[j]));
      sum = fma2(c[j], h[j], sum);
    }
    float y = sum.x + sum.y;
#pragma unroll
    for (int w = 1; w < L; w *= 2) y += __shfl_xor_sync(0xffffffffu, y, w);
    if (mine) {
      if (q == 0) {
        y = fmaf(skip, x, y);
        if (A.z) y *= silu(load_one<BF16>(A.z, zb + t * A.z_tok));
        store_one<BF16>(A.y, out + (long long)t * A.D, y);
      }
      if (A.states) __stcs(reinterpret_cast<float4*>(A.states + (out + (long long)t * A.D) * N + q), make_float4(h[0].x, h[0].y, h[1].x, h[1].y));
    }
  }
  if (!mine) return;
  for (int t = R.len; t < A.T; ++t) {
    if (q == 0) store_one<BF16>(A.y, out + (long long)t * A.D, 0.f);
    if (A.states) __stcs(reinterpret_cast<float4*>(A.states + (out + (long long)t * A.D) * N + q), make_float4(0.f, 0.f, 0.f, 0.f));
  }
  if (R.to >= 0) *reinterpret_cast<float4*>(A.last + ((long long)R.to * A.D + d) * N + q) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
}

template <bool BF16, int N>
static int launch_scan(const ScanArgs& A, bool wide, cudaStream_t st) {
  const dim3 grid((unsigned)(((long long)A.D * (N / 4) + kScanStepThreads - 1) / kScanStepThreads), A.B);
  if (wide) scan_step_kernel<BF16, N, true><<<grid, kScanStepThreads, 0, st>>>(A);
  else scan_step_kernel<BF16, N, false><<<grid, kScanStepThreads, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <bool BF16>
static int launch_scan_of(const ScanArgs& A, int N, bool wide, cudaStream_t st) {
  switch (N) {
    case 8: return launch_scan<BF16, 8>(A, wide, st);
    case 16: return launch_scan<BF16, 16>(A, wide, st);
    case 32: return launch_scan<BF16, 32>(A, wide, st);
    case 64: return launch_scan<BF16, 64>(A, wide, st);
    default: return launch_scan<BF16, 128>(A, wide, st);
  }
}

static bool scan_dims(int B, int T, int D, int N) {
  return B >= 0 && B <= 65535 && T >= 0 && T <= SPEC_MAX_LENGTH && D >= 1 && D <= (1 << 24) &&
         (N == 8 || N == 16 || N == 32 || N == 64 || N == 128);
}

}  // namespace specv

extern "C" size_t spec_scan_workspace_size(int B, int T, int D, int N) {
  if (!specv::scan_dims(B, T, D, N)) return 0;
  return 256;
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
  return s->dtype == SPEC_BF16 ? launch_scan_of<true>(A, s->N, wide, st) : launch_scan_of<false>(A, s->N, wide, st);
}
