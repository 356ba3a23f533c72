// Attention of a few query rows (16, 32 or 64: tokens times the group) over a
// long cache: verify and decode steps.
//
// Bound by the cache's bytes: for M rows a position of one head costs
// 4 * M * D operations for 4 D bytes (2 D in 8 bits), 16 to 128 a byte, which
// the warp-level matrix instructions deliver beside the loads; the wide
// tcgen05 tile of 128 rows would spend its time on padding.
//
// One producer warp brings tiles of 64 positions by TMA, a box a run of
// positions within a page, through a ring of stages.  Four consumer warps
// divide the positions (16 each, or 32 where 64 rows need two warps in the other
// direction) and keep their own running maximum, sum and weighted values in
// registers, so no warp waits for another within an item; they are joined in
// shared memory at its end.  The maximum only moves when a score passes it by
// 2^8, which keeps weights below 2^8 and rescales the sums a few times a row
// instead of at every tile.  8-bit codes become bf16 in registers: the code's
// bits, shifted, are a bf16 number 2^-120 too small, and one packed product
// corrects that exactly; the scales go to the scores (keys) and the weights
// (values) in float32.
#include "spec_attend.cuh"

namespace specv {

constexpr int kRowsKT = 64;
constexpr int kRowsThreads = 160;
constexpr float kRowsSlack = 8.f;

template <int D, bool E4M3, int MT>
struct RowsShape {
  static constexpr int M = 16 * MT;
  static constexpr int row_bytes = D * (E4M3 ? 1 : 2);
  static constexpr int halves = row_bytes > 128 ? 2 : 1;         // 128-byte columns of a row
  static constexpr int half_bytes = row_bytes / halves;
  static constexpr int half_tile = kRowsKT * half_bytes;
  static constexpr int kv_tile = kRowsKT * row_bytes;
  static constexpr int stage = 2 * kv_tile;
  static constexpr int q_bytes = M * D * 2;
  static constexpr int pitch = D + 8;                            // floats a row of the joined values
  static constexpr int o_bytes = M * pitch * 4;
  static constexpr int ctas = MT == 4 ? 1 : 2;                   // an SM
  static constexpr int most = (224 * 1024 / ctas - q_bytes - o_bytes - 4096) / (stage + 2 * kRowsKT);
  static constexpr int stages = most > 6 ? 6 : most;
  static constexpr int smem = 1024 + stages * (stage + 2 * kRowsKT) + q_bytes + o_bytes;
  static constexpr int wm = MT == 4 ? 2 : 1;                     // warps across the query rows
  static constexpr int wk = 4 / wm;                              // and across the positions
  static constexpr int mt = MT / wm;                             // 16-row tiles a warp
  static constexpr int keys = kRowsKT / wk;                      // positions a warp
  static constexpr int part_floats = M * (D + 2);
};

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}

// Codes in the upper bytes of two halves as bf16: sign, then the seven bits of
// magnitude at the top of bf16's mantissa and below its exponent, times 2^120.
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t high) {
  uint32_t w = ((high >> 4) & 0x07f007f0u) | (high & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0x7b807b80u));
  return w;
}

__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, bool E4M3, int MT>
__global__ void __launch_bounds__(kRowsThreads, (MT == 4 ? 1 : 2)) attend_rows_kernel(const AttendArgs A, const __grid_constant__ CUtensorMap kmap,
                                                                      const __grid_constant__ CUtensorMap vmap) {
  using S = RowsShape<D, E4M3, MT>;
  constexpr int M = S::M, KT = kRowsKT, MTW = S::mt;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long full[S::stages], empty[S::stages];
  __shared__ unsigned long long there[S::stages];     // which positions of the stage are there
  __shared__ AttendShare share;
  __shared__ long long sums[kRowsThreads];
  __shared__ float sm_m[S::wk][M], sm_l[S::wk][M];
  __shared__ int sees[M];
  __shared__ int failed, odd, last_part;
  unsigned char* const base = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  unsigned char* const q_sm = base + S::stages * S::stage;
  float* const o_sm = reinterpret_cast<float*>(q_sm + S::q_bytes);
  unsigned char* const e_sm = q_sm + S::q_bytes + S::o_bytes;      // [stage][k, v][KT] exponents
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < S::stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  attend_share<M, KT, kRowsThreads>(A, &share, sums);
  AttendWalk<M, KT> W(A, share);

  if (warp == 4) {
    // ------------------------------------------------------------- producer
    int stage = 0;
    uint32_t phase = 0;
    const int boxes = KT / A.box;
    // a box of one 64-byte row would not begin at a multiple of 128 bytes: its lane copies it
    const bool by_hand = S::half_bytes == 64 && A.box == 1;
    while (W.next()) {
      const int limit = attend_sees(A, W.R, (min((W.qt + 1) * M, W.R.n * A.group) - 1) / A.group);
      for (int t = W.a; t < W.b; ++t) {
        const int key0 = t * KT;
        // the pages of this lane's boxes, and of its positions where these have exponents
        int page[2], slot[2];
        uint8_t ke[2], ve[2];
        bool ok[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int pos = key0 + lane + 32 * j;
          page[j] = pos < limit ? paged_lookup(A.C, W.row, pos, &slot[j]) : -1;
          ok[j] = page[j] >= 0;
          ke[j] = ve[j] = 0;
          if (E4M3 && ok[j]) {
            const long long e = page[j] * A.C.exp_bytes + (long long)W.head * A.C.page_size + slot[j];
            ke[j] = __ldg(A.C.k_exp + e);
            ve[j] = __ldg(A.C.v_exp + e);
          }
          if (!ok[j] && pos < limit && A.flags) atomicOr(&A.flags[W.row], (uint32_t)SPEC_F_BAD_IDX);
        }
        const unsigned long long mask = (unsigned long long)__ballot_sync(0xffffffffu, ok[1]) << 32 | __ballot_sync(0xffffffffu, ok[0]);
        mbar_await(&empty[stage], phase ^ 1, &failed);
        if (E4M3) {
          unsigned char* e = e_sm + stage * 2 * KT;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            e[lane + 32 * j] = ke[j];
            e[KT + lane + 32 * j] = ve[j];
          }
        }
        if (by_hand) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (!ok[j]) continue;
            const int k = lane + 32 * j;
            const long long vec = ((long long)W.head * A.C.page_size + slot[j]) * D + page[j] * A.C.page_bytes;
#pragma unroll
            for (int c = 0; c < S::half_bytes / 16; ++c) {
              unsigned char* to = base + stage * S::stage + k * S::half_bytes + (c ^ (k >> 1 & 3)) * 16;
              *reinterpret_cast<uint4*>(to) = __ldg(reinterpret_cast<const uint4*>(A.C.k + vec) + c);
              *reinterpret_cast<uint4*>(to + S::kv_tile) = __ldg(reinterpret_cast<const uint4*>(A.C.v + vec) + c);
            }
          }
          __syncwarp();
        }
        int copies = 0;
        if (!failed && !by_hand)
          for (int b = lane; b < boxes; b += 32) copies += (int)(mask >> (b * A.box)) & 1;
        copies = __reduce_add_sync(0xffffffffu, copies);
        if (lane == 0) {
          there[stage] = mask;
          mbar_arrive_expect_tx(&full[stage], copies * 2 * A.box * S::row_bytes);
        }
        __syncwarp();
        if (copies) {
          const uint32_t dst = smem_u32(base + stage * S::stage);
          for (int b0 = 0; b0 < boxes; b0 += 32) {
            // a box begins at position b * box, which another lane looked up
            const int b = b0 + lane, at = (b * A.box) & 63;
            const int p0 = __shfl_sync(0xffffffffu, page[0], at & 31), p1 = __shfl_sync(0xffffffffu, page[1], at & 31);
            const int s0 = __shfl_sync(0xffffffffu, slot[0], at & 31), s1 = __shfl_sync(0xffffffffu, slot[1], at & 31);
            const int p = at < 32 ? p0 : p1, s = at < 32 ? s0 : s1;
            if (b < boxes && (mask >> at & 1)) {
#pragma unroll
              for (int h = 0; h < S::halves; ++h) {
                const uint32_t to = dst + h * S::half_tile + at * S::half_bytes;
                tma_load_4d(to, &kmap, h * 64, s, W.head, p, &full[stage]);
                tma_load_4d(to + S::kv_tile, &vmap, h * 64, s, W.head, p, &full[stage]);
              }
            }
          }
        }
        if (++stage == S::stages) stage = 0, phase ^= 1;
      }
    }
    // the copies in flight land before the CTA may end
    for (int i = 0; i < S::stages; ++i) {
      mbar_await(&empty[stage], phase ^ 1, &failed);
      if (++stage == S::stages) stage = 0, phase ^= 1;
    }
    return;
  }

  // --------------------------------------------------------------- consumers
  int stage = 0;
  uint32_t phase = 0;
  const int mw = warp % S::wm, kw = warp / S::wm;         // this warp's place across rows and positions
  const int q4 = lane % 4, r8 = lane / 4;
  while (W.next()) {
    const int rows = min(M, W.R.n * A.group - W.qt * M);  // query rows of this tile
    // Q as the matrix instruction's A fragments, 16 bytes a lane, and what each row sees.
    for (int i = threadIdx.x; i < M * D / 8; i += 128) {
      const int fl = i % 32, ks = i / 32 % (D / 16), m0 = i / 32 / (D / 16) * 16 + fl / 4, q = fl % 4;
      uint2 w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + 8 * h;
        w[h] = make_uint2(0, 0);
        if (m < rows) {
          const int g = W.qt * M + m, token = g / A.group, head = W.head * A.group + g - token * A.group;
          const uint16_t* p = A.q + (W.R.first + token) * A.q_token + (long long)head * D;
          if (E4M3) {
            // a lane's four of k-step ks: those that its 16-byte load of codes brings (see below)
            const int d = D == 128 ? 32 * q + 16 * (ks / 4) + 4 * (ks % 4) : 16 * q + 4 * ks;
            w[h] = *reinterpret_cast<const uint2*>(p + d);
          } else {
            w[h].x = *reinterpret_cast<const uint32_t*>(p + ks * 16 + 2 * q);
            w[h].y = *reinterpret_cast<const uint32_t*>(p + ks * 16 + 2 * q + 8);
          }
        }
      }
      *reinterpret_cast<uint4*>(q_sm + i * 16) = make_uint4(w[0].x, w[1].x, w[0].y, w[1].y);
    }
    if (threadIdx.x < M) {
      const int g = min(W.qt * M + (int)threadIdx.x, W.R.n * A.group - 1);
      sees[threadIdx.x] = attend_sees(A, W.R, g / A.group);
    }
    if (threadIdx.x == 0) odd = 0;
    rows_sync();
    const int fewest = sees[0];                           // the first row's token comes first
    int lim[MTW][2];
#pragma unroll
    for (int i = 0; i < MTW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) lim[i][h] = sees[(mw * MTW + i) * 16 + 8 * h + r8];

    float o[MTW][D / 8][4], m[MTW][2], l[MTW][2];
#pragma unroll
    for (int i = 0; i < MTW; ++i) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][d][e] = 0.f;
      m[i][0] = m[i][1] = -INFINITY;
      l[i][0] = l[i][1] = 0.f;
    }

    for (int t = W.a; t < W.b; ++t) {
      mbar_await(&full[stage], phase, &failed);
      const uint32_t ks_base = smem_u32(base + stage * S::stage), vs_base = ks_base + S::kv_tile;
      const unsigned long long mask = there[stage];
      const bool edge = (t + 1) * KT > fewest || mask != ~0ull;
#pragma unroll
      for (int step = 0; step < S::keys / 16; ++step) {
        const int k0 = kw * S::keys + step * 16;          // this warp's 16 positions of the tile
        if (edge) {
          // A value of weight zero must be finite: positions that are not there are cleared, and what is not
          // finite of those that only some rows see is cleared and remembered.
          bool found = false;
#pragma unroll
          for (int i = lane; i < 16 * (S::row_bytes / 16); i += 32) {
            const int k = k0 + i / (S::row_bytes / 16), c = i % (S::row_bytes / 16);
            unsigned char* p = base + stage * S::stage + S::kv_tile + (c * 16 / S::half_bytes) * S::half_tile + k * S::half_bytes;
            const int cc = c % (S::half_bytes / 16);
            p += (S::half_bytes == 128 ? cc ^ (k & 7) : cc ^ (k >> 1 & 3)) * 16;
            uint4 w = *reinterpret_cast<uint4*>(p);
            if (!(mask >> k & 1)) {
              *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
            } else if (!E4M3 && t * KT + k >= fewest) {
              uint32_t* x = reinterpret_cast<uint32_t*>(&w);
              bool bad = false;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if ((x[j] & 0x7f80u) == 0x7f80u) x[j] &= 0xffff0000u, bad = true;
                if ((x[j] & 0x7f800000u) == 0x7f800000u) x[j] &= 0xffffu, bad = true;
              }
              if (bad) *reinterpret_cast<uint4*>(p) = w;
              found = found || bad;
            }
          }
          if (found) odd = 1;
          __syncwarp();
        }
        float s[MTW][2][4];
#pragma unroll
        for (int i = 0; i < MTW; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][n][e] = 0.f;
        const uint32_t qa = smem_u32(q_sm) + (mw * MTW) * D * 32 + lane * 16;
        if (!E4M3) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t kb[4];
            const int k = k0 + (lane / 16) * 8 + lane % 8, c = (ks % 4) * 2 + (lane / 8 & 1);
            ldsm4(kb, ks_base + (ks / 4) * S::half_tile + k * 128 + ((c ^ (k & 7)) << 4));
#pragma unroll
            for (int i = 0; i < MTW; ++i) {
              const uint4 f = lds128(qa + (i * (D / 16) + ks) * 512);
              const uint32_t a[4] = {f.x, f.y, f.z, f.w};
              mma_bf16(s[i][0], a, kb[0], kb[1]);
              mma_bf16(s[i][1], a, kb[2], kb[3]);
            }
          }
        } else {
          // A lane loads 16 codes of its position (16-byte column 2 q + j of 8, or q of 4); which dimension stands
          // at which place of the sum does not matter, so its bytes 4 i .. 4 i + 3 are its four of k-step 4 j + i.
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint4 kc[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int k = k0 + 8 * n + r8;
              const int c = D == 128 ? (2 * q4 + j) ^ (k & 7) : q4 ^ (k >> 1 & 3);
              kc[n] = lds128(ks_base + k * S::row_bytes + c * 16);
            }
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              uint32_t kb[2][2];
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const uint32_t w = i4 == 0 ? kc[n].x : i4 == 1 ? kc[n].y : i4 == 2 ? kc[n].z : kc[n].w;
                kb[n][0] = e4m3_bf16(__byte_perm(w, 0, 0x1404));
                kb[n][1] = e4m3_bf16(__byte_perm(w, 0, 0x3424));
              }
#pragma unroll
              for (int i = 0; i < MTW; ++i) {
                const uint4 f = lds128(qa + (i * (D / 16) + 4 * j + i4) * 512);
                const uint32_t a[4] = {f.x, f.y, f.z, f.w};
                mma_bf16(s[i][0], a, kb[0][0], kb[0][1]);
                mma_bf16(s[i][1], a, kb[1][0], kb[1][1]);
              }
            }
          }
        }
        // scores in powers of two, masked; the scales of this lane's columns
        float vs[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int k = k0 + 8 * n + 2 * q4;
          float ksc[2] = {A.scale_log2, A.scale_log2};
          if (E4M3) {
            const unsigned char* e = e_sm + stage * 2 * KT + k;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              ksc[j] *= exp_value(e[j]);
              vs[n][j] = exp_value(e[KT + j]);
            }
          }
#pragma unroll
          for (int i = 0; i < MTW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[i][n][e] *= ksc[e & 1];
              if (edge && (t * KT + k + (e & 1) >= lim[i][e >> 1] || !(mask >> (k + (e & 1)) & 1))) s[i][n][e] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < MTW; ++i) {
          float top[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(fmaxf(s[i][0][2 * h], s[i][0][2 * h + 1]), fmaxf(s[i][1][2 * h], s[i][1][2 * h + 1]));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          }
          if (__any_sync(0xffffffffu, top[0] > m[i][0] + kRowsSlack || top[1] > m[i][1] + kRowsSlack)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float to = fmaxf(m[i][h], top[h]);
              const float keep = to == -INFINITY ? 1.f : exp2_fast(m[i][h] - to);
              m[i][h] = to;
              l[i][h] *= keep;
#pragma unroll
              for (int d = 0; d < D / 8; ++d) o[i][d][2 * h] *= keep, o[i][d][2 * h + 1] *= keep;
            }
          }
          uint32_t p[2][2];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float from = m[i][h] == -INFINITY ? 0.f : m[i][h];
              float a = exp2_fast(s[i][n][2 * h] - from), b = exp2_fast(s[i][n][2 * h + 1] - from);
              l[i][h] += a + b;
              if (E4M3) {
                // a scale that is not seen may be NaN
                a = edge && a == 0.f ? 0.f : a * vs[n][0];
                b = edge && b == 0.f ? 0.f : b * vs[n][1];
              }
              p[n][h] = pack_bf16(a, b);
            }
          const uint32_t pa[4] = {p[0][0], p[0][1], p[1][0], p[1][1]};
          // the values' fragments are loaded again for a second 16-row tile: registers are short
          if (!E4M3) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              uint32_t vb[4];
              const int k = k0 + (lane / 8 & 1) * 8 + lane % 8, c = (d % 4) * 2 + lane / 16;
              ldsm4_t(vb, vs_base + (d / 4) * S::half_tile + k * 128 + ((c ^ (k & 7)) << 4));
              mma_bf16(o[i][2 * d], pa, vb[0], vb[1]);
              mma_bf16(o[i][2 * d + 1], pa, vb[2], vb[3]);
            }
          } else {
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
              // pairs of dimensions move as one 16-bit element; even and odd ones are tiles of their own
              uint32_t vb[4];
              const int k = k0 + (lane / 8 & 1) * 8 + lane % 8, c = 2 * d + lane / 16;
              ldsm4_t(vb, vs_base + k * S::row_bytes + ((D == 128 ? c ^ (k & 7) : c ^ (k >> 1 & 3)) << 4));
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                mma_bf16(o[i][4 * d + 2 * j], pa, e4m3_bf16(vb[2 * j] << 8 & 0xff00ff00u), e4m3_bf16(vb[2 * j + 1] << 8 & 0xff00ff00u));
                mma_bf16(o[i][4 * d + 2 * j + 1], pa, e4m3_bf16(vb[2 * j] & 0xff00ff00u), e4m3_bf16(vb[2 * j + 1] & 0xff00ff00u));
              }
            }
          }
        }
      }
      if (edge) fence_proxy_async();     // what was cleared is written before the next copy lands here
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == S::stages) stage = 0, phase ^= 1;
    }

    // ------------------------------------------------ join the warps' positions
#pragma unroll
    for (int i = 0; i < MTW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
        if (q4 == 0) {
          const int row = (mw * MTW + i) * 16 + 8 * h + r8;
          sm_m[kw][row] = m[i][h];
          sm_l[kw][row] = l[i][h];
        }
      }
    rows_sync();
    float mine[MTW][2];
#pragma unroll
    for (int i = 0; i < MTW; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = (mw * MTW + i) * 16 + 8 * h + r8;
        float top = sm_m[0][row];
#pragma unroll
        for (int w = 1; w < S::wk; ++w) top = fmaxf(top, sm_m[w][row]);
        mine[i][h] = top == -INFINITY ? 1.f : exp2_fast(m[i][h] - top);
      }
    for (int w = 0; w < S::wk; ++w) {
      if (kw == w) {
#pragma unroll
        for (int i = 0; i < MTW; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* row = o_sm + ((mw * MTW + i) * 16 + 8 * h + r8) * S::pitch;
#pragma unroll
            for (int d = 0; d < D / 8; d += 2) {
              // in 16 bits columns 8 d + 2 q of two tiles; in 8 bits 8 d + 4 q .. + 3 of an even and an odd tile
              float x[4] = {o[i][d][2 * h] * mine[i][h], o[i][d][2 * h + 1] * mine[i][h], o[i][d + 1][2 * h] * mine[i][h],
                            o[i][d + 1][2 * h + 1] * mine[i][h]};
              float* p0 = row + 8 * d + (E4M3 ? 4 : 2) * q4;
              float* p1 = E4M3 ? p0 + 2 : p0 + 8;
              if (E4M3) {
                const float y = x[1];
                x[1] = x[2];
                x[2] = y;
              }
              float2 a = make_float2(x[0], x[1]), b = make_float2(x[2], x[3]);
              if (w) {
                const float2 c = *reinterpret_cast<float2*>(p0), e = *reinterpret_cast<float2*>(p1);
                a.x += c.x, a.y += c.y, b.x += e.x, b.y += e.y;
              }
              *reinterpret_cast<float2*>(p0) = a;
              *reinterpret_cast<float2*>(p1) = b;
            }
          }
      }
      rows_sync();
    }
    if (odd) {
      // values that are not finite at positions that only some rows see
      for (int k = max(fewest, W.a * KT); k < min(sees[M - 1], W.b * KT); ++k) {
        int slot;
        const int page = paged_lookup(A.C, W.row, k, &slot);
        if (page < 0) continue;
        const uint16_t* v = reinterpret_cast<const uint16_t*>(A.C.v + page * A.C.page_bytes) + ((long long)W.head * A.C.page_size + slot) * D;
        for (int d = threadIdx.x; d < D; d += 128) {
          const float x = __uint_as_float((uint32_t)v[d] << 16);
          if (isfinite(x)) continue;
          for (int row = 0; row < M; ++row)
            if (k < sees[row]) o_sm[row * S::pitch + d] += x;
        }
      }
      rows_sync();
    }
    // each thread keeps its place of the joined result: row, and columns of 8
    const bool whole = W.whole();
    const long long item = W.item_begin();
    const int c0 = whole ? 0 : share_of(share.total, item, share.ctas);
    const int c1 = whole ? 0 : share_of(share.total, item + W.tiles - 1, share.ctas);
    if (!whole) {
      float* part = A.parts + ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0)) * S::part_floats;
      for (int i = threadIdx.x; i < M * D / 4; i += 128) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        __stcg(reinterpret_cast<float4*>(part + row * D + d), *reinterpret_cast<float4*>(o_sm + row * S::pitch + d));
      }
      if (threadIdx.x < M) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < S::wk; ++w) top = fmaxf(top, sm_m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < S::wk; ++w) sum += sm_l[w][threadIdx.x] * (top == -INFINITY ? 1.f : exp2_fast(sm_m[w][threadIdx.x] - top));
        __stcg(part + M * D + threadIdx.x, top);
        __stcg(part + M * D + M + threadIdx.x, sum);
      }
      __threadfence();
      rows_sync();
      if (threadIdx.x == 0) {
        const unsigned had = atomicAdd(&A.joined[c0], 1u);
        last_part = had == (unsigned)(c1 - c0);
        if (last_part) A.joined[c0] = 0;
        __threadfence();
      }
      rows_sync();
    }
    if (whole || last_part) {
      for (int i = threadIdx.x; i < rows * (D / 8); i += 128) {
        const int row = i / (D / 8), d = i % (D / 8) * 8;
        float x[8], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (whole) {
#pragma unroll
          for (int w = 0; w < S::wk; ++w) top = fmaxf(top, sm_m[w][row]);
#pragma unroll
          for (int w = 0; w < S::wk; ++w) sum += sm_l[w][row] * (top == -INFINITY ? 1.f : exp2_fast(sm_m[w][row] - top));
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = o_sm[row * S::pitch + d + e];
        } else {
          for (int c = c0; c <= c1; ++c) {
            const float* part = A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats;
            const float pm = __ldcg(part + M * D + row), pl = __ldcg(part + M * D + M + row);
            const float4 a = __ldcg(reinterpret_cast<const float4*>(part + row * D + d));
            const float4 b = __ldcg(reinterpret_cast<const float4*>(part + row * D + d + 4));
            const float to = fmaxf(top, pm);
            const float keep = to == -INFINITY ? 1.f : exp2_fast(top - to), add = to == -INFINITY ? 1.f : exp2_fast(pm - to);
            top = to;
            sum = sum * keep + pl * add;
            const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * keep + y[e] * add;
          }
        }
        const int g = W.qt * M + row, token = g / A.group;
        const long long at = (long long)(W.R.first + token) * A.hq + W.head * A.group + g - token * A.group;
        const float inv = sum == 0.f ? 1.f : 1.f / sum;
        *reinterpret_cast<uint4*>(A.out + at * D + d) =
            make_uint4(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv), pack_bf16(x[4] * inv, x[5] * inv),
                       pack_bf16(x[6] * inv, x[7] * inv));
        if (d == 0 && A.lse) A.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      }
    }
    if (threadIdx.x == 0 && failed && A.flags) atomicOr(&A.flags[W.row], (uint32_t)SPEC_F_TIMEOUT);
    rows_sync();
  }
}

template <int D, bool E4M3, int MT>
static int launch_rows(const AttendArgs& A, const CUtensorMap* maps, cudaStream_t st) {
  using S = RowsShape<D, E4M3, MT>;
  static_assert(S::stages >= 2, "a ring needs two stages");
  const auto kernel = attend_rows_kernel<D, E4M3, MT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_E_CUDA;
  }
  kernel<<<S::ctas * 152, kRowsThreads, S::smem, st>>>(A, maps[0], maps[1]);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

int launch_attend_rows(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st) {
  if (A.C.D == 128) {
    if (e4m3) return rows <= 16 ? launch_rows<128, true, 1>(A, maps, st) : rows <= 32 ? launch_rows<128, true, 2>(A, maps, st) : launch_rows<128, true, 4>(A, maps, st);
    return rows <= 16 ? launch_rows<128, false, 1>(A, maps, st) : rows <= 32 ? launch_rows<128, false, 2>(A, maps, st) : launch_rows<128, false, 4>(A, maps, st);
  }
  if (e4m3) return rows <= 16 ? launch_rows<64, true, 1>(A, maps, st) : rows <= 32 ? launch_rows<64, true, 2>(A, maps, st) : launch_rows<64, true, 4>(A, maps, st);
  return rows <= 16 ? launch_rows<64, false, 1>(A, maps, st) : rows <= 32 ? launch_rows<64, false, 2>(A, maps, st) : launch_rows<64, false, 4>(A, maps, st);
}

}  // namespace specv
