// spec_conv: y_t = act(bias + sum_i w_i x_{t - W + 1 + i}), channel by channel.
//
// Bound by memory: each input is read once and each output written once for 2 W
// operations.  A thread has 16 bytes of neighbouring channels and walks a tile of
// tokens with the last W - 1 inputs in registers, so a tile reads W - 1 tokens
// before its own again (from L2).
//
// Measured, width 4, SiLU: 4x8192 tokens x 4096 channels bf16 114 us, 4700 GB/s (70 % of the
// copy bandwidth; with rows of uneven lengths 76 us, 80 %), 4x4096x4096 float32 88 us, 6100 GB/s
// (91 %): a 16-bit token has twice the arithmetic a byte.  Tiles of 64 tokens take as long with
// large batches and 20 % longer with 3x1021 tokens; four tokens ahead and not eight 4 % longer.
#include "spec_mixer.cuh"

namespace specv {

struct ConvArgs {
  const unsigned char* x;
  const float* weight;
  const float* bias;
  const unsigned char* state;
  const int32_t* slot;
  const int32_t* lens;
  unsigned char* y;
  unsigned char* states;
  unsigned char* last;
  const int32_t* last_slot;
  uint32_t* flags;
  long long x_row, x_tok;      // elements
  int dtype, B, T, C, slots, last_slots, blocks;
};

constexpr int kConvThreads = 128;
constexpr int kConvTile = 32;      // tokens of a tile
constexpr int kConvAhead = 8;      // tokens loaded before they are used

// VEC neighbouring channels of one token, as they are in memory.
template <bool BF16, int VEC>
struct ConvVec {
  static constexpr int kBytes = VEC * (BF16 ? 2 : 4), kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const unsigned char* p) {
    if (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[kWords / 4] = v.y, w[kWords / 2] = v.z, w[kWords / 4 * 3] = v.w;
    } else if (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(unsigned char* p) const {
    if (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[kWords / 4], w[kWords / 2], w[kWords / 4 * 3]);
    else if (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  __device__ __forceinline__ float get(int v) const {
    if (!BF16) return __uint_as_float(w[v]);
    return v % 2 ? bf16_hi(w[v / 2]) : bf16_lo(w[v / 2]);
  }
  __device__ __forceinline__ void set(const float* x) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      if (!BF16) w[v] = __float_as_uint(x[v]);
      else if (v % 2 == 0) w[v / 2] = pack_bf16(x[v], v + 1 < VEC ? x[v + 1 < VEC ? v + 1 : v] : 0.f);
    }
  }
};

template <bool BF16, int VEC, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(const ConvArgs A) {
  using V = ConvVec<BF16, VEC>;
  constexpr int es = BF16 ? 2 : 4, K = W - 1;
  const int r = blockIdx.y, tile = blockIdx.x / A.blocks;
  const int c = ((blockIdx.x - tile * A.blocks) * kConvThreads + threadIdx.x) * VEC;
  if (c >= A.C) return;
  const MixerRow R = mixer_row(A, r, tile == 0 && c == 0);
  const long long t0 = (long long)tile * kConvTile, t1 = min(t0 + kConvTile, (long long)A.T);
  const unsigned char* const x = A.x + (r * A.x_row + c) * es;
  const long long x_tok = A.x_tok * es, tok = (long long)A.C * es;
  unsigned char* const y = A.y + ((long long)r * A.T * A.C + c) * es;
  unsigned char* const states = A.states ? A.states + ((long long)r * A.T * K * A.C + c) * es : nullptr;
  // the first tile has to do with the row's states: no other thread reads or writes these channels of them
  const unsigned char* const first = R.from >= 0 ? A.state + ((long long)R.from * K * A.C + c) * es : nullptr;

  V before[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const long long t = t0 - K + i;
    before[i].zero();
    if (t >= 0) {
      if (t < R.len) before[i].load(x + t * x_tok);
    } else if (first) {
      before[i].load(first + i * tok);      // (t0 is 0)
    }
  }
  if (t0 < R.len) {
    float w[W][VEC], b[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      b[v] = A.bias ? __ldg(A.bias + c + v) : 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) w[i][v] = __ldg(A.weight + (long long)i * A.C + c + v);
    }
    const long long end = min(t1, (long long)R.len);
    for (long long t = t0; t < end; t += kConvAhead) {
      V in[kConvAhead];
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) in[j].load(x + min(t + j, end - 1) * x_tok);
#pragma unroll
      for (int j = 0; j < kConvAhead; ++j) {
        if (t + j >= end) break;
        float out[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          float s = b[v];
#pragma unroll
          for (int i = 0; i < K; ++i) s = fmaf(w[i][v], before[i].get(v), s);
          s = fmaf(w[K][v], in[j].get(v), s);
          out[v] = SILU ? silu(s) : s;
        }
#pragma unroll
        for (int i = 0; i + 1 < K; ++i) before[i] = before[i + 1];
        before[K - 1] = in[j];
        V o;
        o.set(out);
        o.store(y + (t + j) * tok);
        if (states)
#pragma unroll
          for (int i = 0; i < K; ++i) before[i].store(states + ((t + j) * K + i) * tok);
      }
    }
  }
  V none;
  none.zero();
  for (long long t = max(t0, (long long)R.len); t < t1; ++t) {
    none.store(y + t * tok);
    if (states)
      for (int i = 0; i < K; ++i) none.store(states + (t * K + i) * tok);
  }
  if (tile == 0 && R.to >= 0) {
    // The state behind the last token, entry by entry: what an entry takes from the first state lies at the same place
    // of it or further on, so a state may be written over itself.
    unsigned char* const last = A.last + ((long long)R.to * K * A.C + c) * es;
#pragma unroll 1
    for (int i = 0; i < K; ++i) {
      const long long at = (long long)R.len - K + i;
      V v;
      v.zero();
      if (at >= 0) v.load(x + at * x_tok);
      else if (first) v.load(first + (K + at) * tok);
      v.store(last + i * tok);
    }
  }
}

template <bool BF16, int VEC, int W>
static int launch_conv(ConvArgs& A, bool silu, cudaStream_t st) {
  A.blocks = (A.C + kConvThreads * VEC - 1) / (kConvThreads * VEC);
  const long long tiles = A.T > 0 ? ((long long)A.T + kConvTile - 1) / kConvTile : 1;
  if (tiles * A.blocks > 0x7fffffff) return SPEC_E_DIM;
  const dim3 grid((unsigned)(tiles * A.blocks), A.B);
  if (silu) conv_kernel<BF16, VEC, W, true><<<grid, kConvThreads, 0, st>>>(A);
  else conv_kernel<BF16, VEC, W, false><<<grid, kConvThreads, 0, st>>>(A);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

// 16 bytes of channels a thread where every array allows it.
template <bool BF16, int W>
static int launch_conv_of(ConvArgs& A, bool silu, cudaStream_t st) {
  constexpr int vec = BF16 ? 8 : 4;
  const bool wide = A.C % vec == 0 && A.x_row % vec == 0 && A.x_tok % vec == 0 && paged_aligned(A.x, 16) && paged_aligned(A.y, 16) &&
                    paged_aligned(A.state, 16) && paged_aligned(A.states, 16) && paged_aligned(A.last, 16);
  return wide ? launch_conv<BF16, vec, W>(A, silu, st) : launch_conv<BF16, 1, W>(A, silu, st);
}

template <bool BF16>
static int launch_conv_width(ConvArgs& A, int width, bool silu, cudaStream_t st) {
  switch (width) {
    case 2: return launch_conv_of<BF16, 2>(A, silu, st);
    case 3: return launch_conv_of<BF16, 3>(A, silu, st);
    case 4: return launch_conv_of<BF16, 4>(A, silu, st);
    case 5: return launch_conv_of<BF16, 5>(A, silu, st);
    case 6: return launch_conv_of<BF16, 6>(A, silu, st);
    case 7: return launch_conv_of<BF16, 7>(A, silu, st);
    default: return launch_conv_of<BF16, 8>(A, silu, st);
  }
}

}  // namespace specv

extern "C" int spec_conv(const spec_conv_t* conv, void* cuda_stream) {
  using namespace specv;
  if (!conv) return SPEC_E_NULL;
  const int rc = mixer_check(*conv);
  if (rc != SPEC_OK) return rc;
  if (conv->C < 1 || conv->C > (1 << 26) || conv->width < 2 || conv->width > SPEC_MAX_CONV) return SPEC_E_DIM;
  if (conv->B == 0 || (conv->T == 0 && !conv->last)) return SPEC_OK;
  if (conv->T > 0 && (!conv->x || !conv->weight || !conv->y)) return SPEC_E_NULL;
  const size_t es = conv->dtype == SPEC_BF16 ? 2 : 4;
  if (!paged_aligned(conv->x, es) || !paged_aligned(conv->y, es) || !paged_aligned(conv->state, es) ||
      !paged_aligned(conv->states, es) || !paged_aligned(conv->last, es) || !paged_aligned(conv->weight, 4) ||
      !paged_aligned(conv->bias, 4))
    return SPEC_E_ALIGN;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  ConvArgs A;
  A.x = static_cast<const unsigned char*>(conv->x);
  A.weight = conv->weight;
  A.bias = conv->bias;
  A.state = static_cast<const unsigned char*>(conv->state);
  A.slot = conv->slot;
  A.lens = conv->lens;
  A.y = static_cast<unsigned char*>(conv->y);
  A.states = static_cast<unsigned char*>(conv->states);
  A.last = static_cast<unsigned char*>(conv->last);
  A.last_slot = conv->last_slot;
  A.flags = conv->flags;
  A.x_row = conv->x_row;
  A.x_tok = conv->x_tok;
  A.dtype = conv->dtype;
  A.B = conv->B;
  A.T = conv->T;
  A.C = conv->C;
  A.slots = conv->slots;
  A.last_slots = conv->last_slots;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  return conv->dtype == SPEC_BF16 ? launch_conv_width<true>(A, conv->width, conv->silu != 0, st)
                                  : launch_conv_width<false>(A, conv->width, conv->silu != 0, st);
}
