// Attention of a few query rows (tokens times the group, in tiles of 16 or 32) over
// a long cache: verify and decode steps.
//
// Bound by the cache's bytes: for M rows a position of one head costs
// 4 * M * D operations for 4 D bytes (2 D in 8 bits), 16 to 64 a byte, which
// the warp-level matrix instructions deliver beside the loads; the wide
// tcgen05 tile of 128 rows would spend its time on padding.
//
// The four warps of a CTA divide each tile of positions, 16 each (32 of an 8-bit
// cache: as many bytes), and share nothing until an item ends: every warp brings
// its own positions by TMA (a box a run of positions within a page) through a ring
// of its own, several tiles ahead and across the ends of items, and keeps its own
// running maximum, sum and weighted values in registers.  The maximum only moves when a score
// passes it by 2^8, which keeps weights below 2^8 and rescales the sums a few
// times a row instead of at every tile.
//
// 8-bit codes become fp16 in registers by the conversion instruction (exact),
// so the products are fp16: each query is brought into its range by a power
// of two of its own, and the values' scales 2^e go into the exponent,
//   t_j = log2(weight_j) + e_j,   p_j = 2^(t_j - max t),   sum += p_j 2^-e_j,
// so that the weights of large terms keep all 11 bits whatever the scales.  A
// position whose scale lies far below another's (a value of zero has the smallest
// of all) would lose its weight that way, p_j being no number any more: where a
// tile has exponent bytes out of the ordinary range, its weights are summed by
// 2^((t_j - e_j - max t) / 2) squared instead, which is in range for all scales.
//
// Measured, 8 heads of 128, group 4, 64 rows of 3 tokens: over 8000 positions in
// bf16 191 us, 5600 GB/s (84 % of the copy bandwidth), over up to 12000 in e4m3
// 206 us, 4270 GB/s (64 %: issue slots are busy in 37 % of the cycles and the matrix
// pipe in 22, with two warps a scheduler, each a chain of loads, conversions,
// products and softmax, waiting for itself); one token over 333 positions 11.5 us,
// a chain of latencies (share, page table, copy, products, join).
#include "spec_attend.cuh"

namespace specv {

constexpr int kRowsWarps = 4;
constexpr int kRowsThreads = kRowsWarps * 32;
constexpr float kRowsSlack = 8.f;
constexpr int kRowsShift = 32;       // sums of an 8-bit cache are kept 2^-32 times their size: 2^-e is up to 2^126
static_assert(254 - (int)kAttendTop - kRowsShift >= 1, "so 2^-e of the largest scale is a normal number");
constexpr unsigned kRowsLow = 64, kRowsHigh = 144;   // the ordinary range: within 2^80 a weight of 2^-46 stays a normal number

template <int D, bool E4M3, int MT>
struct RowsShape {
  static constexpr int M = 16 * MT;
  static constexpr int NK = E4M3 ? 32 : 16;                      // positions that a warp takes at a time
  static constexpr int KT = NK * kRowsWarps;
  static constexpr int row_bytes = D * (E4M3 ? 1 : 2);
  static constexpr int halves = row_bytes > 128 ? 2 : 1;         // 128-byte columns of a row
  static constexpr int half_bytes = row_bytes / halves;
  static constexpr int half_tile = NK * half_bytes;
  static constexpr int kv_tile = NK * row_bytes;
  static constexpr int stage = 2 * kv_tile;                      // of one warp
  static constexpr int q_bytes = M * D * 2;
  static constexpr int pitch = D + 8;                            // floats a row of the joined values
  static constexpr int o_bytes = M * pitch * 4;
  static constexpr int ctas = 2;          // an SM
  static constexpr int small = E4M3 ? 14336 : 6144;              // at least what the small arrays take, the scales among them
  static constexpr int most = (225 * 1024 / ctas - 1024 - q_bytes - o_bytes - small) / (kRowsWarps * stage);
  static constexpr int stages = most > 6 ? 6 : most;
  static constexpr int smem = 1024 + stages * kRowsWarps * stage + q_bytes + o_bytes;
  static constexpr int part_floats = M * (D + 2);
};

template <bool F16>
__device__ __forceinline__ void mma_16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
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
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}

// x 2^y where 2^y may be out of range, x being far from 1.
__device__ __forceinline__ float times_exp2(float x, float y) {
  const float half = exp2_fast(0.5f * y);
  return x * half * half;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What a warp brings next: its positions of a tile, looked up a tile before
// their copies begin.
template <int M, int NK, bool E4M3>
struct RowsFetch {
  AttendWalk<M, NK * kRowsWarps, false> I;
  int t, limit;          // the tile, and the positions that its item sees
  bool more;
  int page, slot;        // of position `lane` (NK of them)
  uint32_t ke, ve;       // its exponents

  __device__ __forceinline__ RowsFetch(const AttendArgs& A, const AttendShare& S) : I(A, S) { segment(); }
  __device__ __forceinline__ void segment() {
    more = I.next();
    t = I.a;
    if (more) limit = attend_sees(I.A, I.R, attend_token(I.A, min((I.qt + 1) * M, I.R.n * I.A.group) - 1));
  }
  __device__ __forceinline__ void look(int warp, int lane) {
    page = -1;
    ke = ve = 0;
    if (!more) return;
    const AttendArgs& A = I.A;
    const int pos = (t * kRowsWarps + warp) * NK + lane;
    if ((NK == 32 || lane < NK) && pos < limit) {
      page = paged_lookup(A.C, I.row, pos, &slot);
      if (page < 0 && A.flags) atomicOr(&A.flags[I.row], (uint32_t)SPEC_F_BAD_IDX);
      if (E4M3 && page >= 0) {
        const long long e = page * A.C.exp_bytes + (unsigned)(I.head * A.C.page_size + slot);
        ke = __ldg(A.C.k_exp + e);
        ve = __ldg(A.C.v_exp + e);
      }
    }
  }
  __device__ __forceinline__ void step() {
    if (++t >= I.b) segment();
  }
};

template <int D, bool E4M3, int MT>
__global__ void __launch_bounds__(kRowsThreads, (RowsShape<D, E4M3, MT>::ctas))
    attend_rows_kernel(const AttendArgs A, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = RowsShape<D, E4M3, MT>;
  constexpr int M = S::M, KT = S::KT, NK = S::NK, NS = NK / 16;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) unsigned long long full[kRowsWarps][S::stages];
  // bits: positions of the stage that are there; whether values are NaN (1), scales above (2) or below (4) the ordinary
  __shared__ unsigned there[kRowsWarps][S::stages][2];
  __shared__ __align__(8) float scales[kRowsWarps][S::stages][E4M3 ? 3 : 1][E4M3 ? NK : 1];   // keys' 2^e, values' e and 2^-e
  __shared__ AttendShare share;
  __shared__ long long sums[kRowsThreads];
  __shared__ float sm_m[kRowsWarps][M], sm_l[kRowsWarps][M], tops[kRowsThreads / M][M];
  __shared__ int sees[M];
  __shared__ long long q_at[M], out_at[M];        // where a query row is read and written
  __shared__ int failed, odd, last_part, first_nan;
  // 8-bit cache: a query row's largest magnitude
  __shared__ unsigned q_top[E4M3 ? M : 1];
  unsigned char* const base = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  unsigned char* const q_sm = base + S::stages * kRowsWarps * S::stage;
  float* const o_sm = reinterpret_cast<float*>(q_sm + S::q_bytes);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  unsigned char* const ring = base + warp * S::stages * S::stage;

  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < kRowsWarps * S::stages; ++i) mbar_init(&full[0][0] + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  attend_share<M, KT, kRowsThreads, 0>(A, &share, sums);

  RowsFetch<M, NK, E4M3> F(A, share);
  F.look(warp, lane);
  // a box of one 64-byte row would not begin at a multiple of 128 bytes: its lane copies it
  const bool by_hand = S::half_bytes == 64 && A.box == 1;
  const int box = min(A.box, NK), copies_of = by_hand ? 0 : NK / box * 2 * S::halves;
  const unsigned starts = by_hand ? 0u : attend_starts(box, 0);
  constexpr unsigned all = NK == 32 ? ~0u : 0xffffu;
  auto bring = [&](int stage) {
    if (!F.more) return;
    const bool go = !mbar_given_up(&failed);       // (lanes may differ on it: they meet again whatever it is)
    const unsigned mask = __ballot_sync(0xffffffffu, F.page >= 0);
    unsigned found = 0;
    if (E4M3 && __any_sync(0xffffffffu, F.page >= 0 && F.ve - kRowsLow > kRowsHigh - kRowsLow))
      found = __reduce_or_sync(0xffffffffu, F.ve > kAttendTop ? 1u : F.ve > kRowsHigh ? 2u : F.page >= 0 && F.ve < kRowsLow ? 4u : 0u);
    unsigned char* const to = ring + stage * S::stage;
    const unsigned bytes = __popc(mask & starts & all) * (box * 2 * S::row_bytes);
    if (E4M3) {
      float* s = &scales[warp][stage][0][0] + lane;
      s[0] = exp_value(F.ke);
      const int e = F.ve > kAttendTop ? 127 : max((int)F.ve, 1);
      s[NK * (E4M3 ? 1 : 0)] = (float)(e - 127);
      s[2 * NK * (E4M3 ? 1 : 0)] = __uint_as_float((uint32_t)(254 - e - kRowsShift) << 23);
    }
    if (by_hand) {
      if (F.page >= 0) {
        const long long at = ((long long)F.I.head * A.C.page_size + F.slot) * D + F.page * A.C.page_bytes;
#pragma unroll
        for (int c = 0; c < S::half_bytes / 16; ++c) {
          unsigned char* p = to + lane * S::half_bytes + (c ^ (lane >> 1 & 3)) * 16;
          *reinterpret_cast<uint4*>(p) = __ldg(reinterpret_cast<const uint4*>(A.C.k + at) + c);
          *reinterpret_cast<uint4*>(p + S::kv_tile) = __ldg(reinterpret_cast<const uint4*>(A.C.v + at) + c);
        }
      }
    }
    if (lane == 0) {
      there[warp][stage][0] = mask;
      there[warp][stage][1] = found;
      if (go) mbar_arrive_expect_tx(&full[warp][stage], bytes);
    }
    __syncwarp();
    if (bytes) {
      for (int i0 = 0; i0 < copies_of; i0 += 32) {
        const int i = i0 + lane, part = i % (2 * S::halves), at = i / (2 * S::halves) * box;
        const int page = __shfl_sync(0xffffffffu, F.page, at % NK), slot = __shfl_sync(0xffffffffu, F.slot, at % NK);
        if (i < copies_of && page >= 0 && go) {
          const int half = part % S::halves;
          const bool v = part >= S::halves;
          tma_load_4d(smem_u32(to + (v ? S::kv_tile : 0) + half * S::half_tile + at * S::half_bytes), v ? &vmap : &kmap, half * 64,
                      slot, F.I.head, page, &full[warp][stage]);
        }
      }
    }
    F.step();
    F.look(warp, lane);
  };
  for (int i = 0; i < S::stages; ++i) bring(i);

  int stage = 0;
  uint32_t phase = 0;
  const int q4 = lane % 4, r8 = lane / 4;
  AttendWalk<M, KT, false> W(A, share);
  while (W.next()) {
    const int rows = min(M, W.R.n * A.group - W.qt * M);  // query rows of this tile
    if (threadIdx.x == 0) odd = 0, first_nan = 0x7fffffff;
    if (threadIdx.x < M) {
      if (E4M3) q_top[threadIdx.x] = 0;
      const int g = min(W.qt * M + (int)threadIdx.x, W.R.n * A.group - 1), token = attend_token(A, g);
      const int head = W.head * A.group + g - token * A.group;
      sees[threadIdx.x] = attend_sees(A, W.R, token);
      q_at[threadIdx.x] = (W.R.first + token) * A.q_token + (long long)head * D;
      out_at[threadIdx.x] = (long long)(W.R.first + token) * A.hq + head;
    }
    __syncthreads();
    // Q as the matrix instruction's A fragments, 16 bytes a lane.
    constexpr int each = M * D / 8 / kRowsThreads;
    uint2 qw[each][2];
    uint32_t top[MT][2] = {};                             // (load u is of rows 16 i + r8 and those 8 on, with i = u / (D / 64))
#pragma unroll
    for (int u = 0; u < each; ++u) {
      const int i = u * kRowsThreads + threadIdx.x;
      const int fl = i % 32, ks = i / 32 % (D / 16), m0 = i / 32 / (D / 16) * 16 + fl / 4, q = fl % 4;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + 8 * h;
        qw[u][h] = make_uint2(0, 0);
        if (m < rows) {
          const uint16_t* p = A.q + q_at[m];
          if (E4M3) {
            // a lane's four of k-step ks: those that its 16-byte load of codes brings (see below)
            const int d = D == 128 ? 32 * q + 16 * (ks / 4) + 4 * (ks % 4) : 16 * q + 4 * ks;
            qw[u][h] = *reinterpret_cast<const uint2*>(p + d);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t x = (e < 2 ? qw[u][h].x : qw[u][h].y) >> (e % 2 * 16) & 0x7fffu;
              top[u / (D / 64)][h] = max(top[u / (D / 64)][h], x < 0x7f80u ? x : 0u);
            }
          } else {
            qw[u][h].x = *reinterpret_cast<const uint32_t*>(p + ks * 16 + 2 * q);
            qw[u][h].y = *reinterpret_cast<const uint32_t*>(p + ks * 16 + 2 * q + 8);
          }
        }
      }
    }
    float q_scale[MT][2], by_row[MT][2];                  // (what turns a row's products into powers of two)
    if (E4M3) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[i][h] = max(top[i][h], __shfl_xor_sync(0xffffffffu, top[i][h], 1));
          top[i][h] = max(top[i][h], __shfl_xor_sync(0xffffffffu, top[i][h], 2));
          if (q4 == 0) atomicMax(&q_top[E4M3 ? i * 16 + 8 * h + r8 : 0], top[i][h]);
        }
      __syncthreads();
      // a row's largest magnitude to 2^13 .. 2^14 (what is 2^-27 of it is still a normal number), whatever the other rows'
      auto up = [&](int row) { return min(13 - ((int)(q_top[E4M3 ? row : 0] >> 7) - 127), 126); };
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int to = up(i * 16 + 8 * h + r8);
          q_scale[i][h] = __uint_as_float((uint32_t)(127 + to) << 23);
          by_row[i][h] = A.scale_log2 * __uint_as_float((uint32_t)(127 - to) << 23);
        }
    }
#pragma unroll
    for (int u = 0; u < each; ++u) {
      uint32_t w[4] = {qw[u][0].x, qw[u][1].x, qw[u][0].y, qw[u][1].y};
      if (E4M3)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float by = q_scale[u / (D / 64)][e & 1];
          w[e] = pack_f16(bf16_lo(w[e]) * by, bf16_hi(w[e]) * by);
        }
      *reinterpret_cast<uint4*>(q_sm + (u * kRowsThreads + threadIdx.x) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    const int fewest = sees[0];                           // the first row's token comes first
    int lim[MT][2];
    float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][d][e] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lim[i][h] = sees[i * 16 + 8 * h + r8];
        m[i][h] = -INFINITY;
        l[i][h] = 0.f;
      }
    }

    bool high_scales = false;                             // among this warp's positions so far
    for (int t = W.a; t < W.b; ++t) {
      mbar_await(&full[warp][stage], phase, &failed);
      unsigned char* const k_sm = ring + stage * S::stage;
      const uint32_t ks_base = smem_u32(k_sm), vs_base = ks_base + S::kv_tile;
      const unsigned mask = there[warp][stage][0];
      bool far_scales = false;
      if (E4M3) {
        const unsigned found = there[warp][stage][1];
        if (found & 1) odd = 1;
        high_scales = high_scales || (found & 2);
        far_scales = high_scales || (found & 4);
      }
      const int key0 = t * KT + warp * NK;                // this warp's first position
      const bool edge = key0 + NK > fewest || mask != all;
      if (edge) {
        // A value of weight zero must be finite: positions that are not there are cleared, and what is not finite of
        // those that only some rows see is cleared and remembered.
        bool found = false;
#pragma unroll
        for (int i = lane; i < NK * (S::row_bytes / 16); i += 32) {
          const int k = i / (S::row_bytes / 16), c = i % (S::row_bytes / 16), cc = c % (S::half_bytes / 16);
          unsigned char* p = k_sm + S::kv_tile + c / (S::half_bytes / 16) * S::half_tile + k * S::half_bytes +
                             (S::half_bytes == 128 ? cc ^ (k & 7) : cc ^ (k >> 1 & 3)) * 16;
          if (!(mask >> k & 1)) {
            *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
          } else if (!E4M3 && key0 + k >= fewest) {
            uint4 w = *reinterpret_cast<uint4*>(p);
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
      float s[NS][MT][2][4];
#pragma unroll
      for (int z = 0; z < NS; ++z)
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[z][i][n][e] = 0.f;
      const uint32_t qa = smem_u32(q_sm) + lane * 16;
      if (!E4M3) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kb[4];
          const int k = (lane / 16) * 8 + lane % 8, c = (ks % 4) * 2 + (lane / 8 & 1);
          ldsm4(kb, ks_base + (ks / 4) * S::half_tile + k * 128 + ((c ^ (k & 7)) << 4));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const uint4 f = lds128(qa + (i * (D / 16) + ks) * 512);
            const uint32_t a[4] = {f.x, f.y, f.z, f.w};
            mma_16<false>(s[0][i][0], a, kb[0], kb[1]);
            mma_16<false>(s[0][i][1], a, kb[2], kb[3]);
          }
        }
      } else {
        // A lane loads 16 codes of its position (16-byte column 2 q + j of 8, or q of 4); which dimension stands at
        // which place of the sum does not matter, so its bytes 4 i .. 4 i + 3 are its four of k-step 4 j + i.
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 kc[NS][2];
#pragma unroll
          for (int z = 0; z < NS; ++z)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int k = 16 * z + 8 * n + r8;
              const int c = D == 128 ? (2 * q4 + j) ^ (k & 7) : q4 ^ (k >> 1 & 3);
              kc[z][n] = lds128(ks_base + k * S::row_bytes + c * 16);
            }
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            uint32_t kb[NS][2][2];
#pragma unroll
            for (int z = 0; z < NS; ++z)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                e4m3_f16(i4 == 0 ? kc[z][n].x : i4 == 1 ? kc[z][n].y : i4 == 2 ? kc[z][n].z : kc[z][n].w, &kb[z][n][0], &kb[z][n][1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              const uint4 f = lds128(qa + (i * (D / 16) + 4 * j + i4) * 512);
              const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
              for (int z = 0; z < NS; ++z) {
                mma_16<true>(s[z][i][0], a, kb[z][0][0], kb[z][0][1]);
                mma_16<true>(s[z][i][1], a, kb[z][1][0], kb[z][1][1]);
              }
            }
          }
        }
      }
      // scores in powers of two (of 8-bit values: with the exponent), masked
      float inv[NS][2][2];
#pragma unroll
      for (int z = 0; z < NS; ++z)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int k = 16 * z + 8 * n + 2 * q4;
          float2 by, plus;
          if (E4M3) {
            const float* f = &scales[warp][stage][0][0] + k;
            const float2 c = *reinterpret_cast<const float2*>(f + 2 * NK);
            by = *reinterpret_cast<const float2*>(f);
            plus = *reinterpret_cast<const float2*>(f + NK);
            inv[z][n][0] = c.x, inv[z][n][1] = c.y;
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& x = s[z][i][n][e];
              x = E4M3 ? fmaf(x, (e & 1 ? by.y : by.x) * by_row[i][e >> 1], e & 1 ? plus.y : plus.x) : x * A.scale_log2;
              if (edge && (key0 + k + (e & 1) >= lim[i][e >> 1] || !(mask >> (k + (e & 1)) & 1))) x = -INFINITY;
            }
        }
      uint32_t pa[NS][MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        float high[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          high[h] = fmaxf(fmaxf(s[0][i][0][2 * h], s[0][i][0][2 * h + 1]), fmaxf(s[0][i][1][2 * h], s[0][i][1][2 * h + 1]));
#pragma unroll
          for (int z = 1; z < NS; ++z)
            high[h] = fmaxf(high[h], fmaxf(fmaxf(s[z][i][0][2 * h], s[z][i][0][2 * h + 1]), fmaxf(s[z][i][1][2 * h], s[z][i][1][2 * h + 1])));
        }
        // a lane's own maximum tells whether the row's has passed; the lanes of a row agree on it only then
        if (__any_sync(0xffffffffu, high[0] > m[i][0] + kRowsSlack || high[1] > m[i][1] + kRowsSlack)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            high[h] = fmaxf(high[h], __shfl_xor_sync(0xffffffffu, high[h], 1));
            high[h] = fmaxf(high[h], __shfl_xor_sync(0xffffffffu, high[h], 2));
            const float was = m[i][h], to = fmaxf(was, high[h]);
            const float keep = to == -INFINITY ? 1.f : exp2_fast(was - to);
            m[i][h] = to;
            l[i][h] = E4M3 ? times_exp2(l[i][h], to == -INFINITY ? 0.f : was - to) : l[i][h] * keep;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) o[i][d][2 * h] *= keep, o[i][d][2 * h + 1] *= keep;
          }
        }
        const float from[2] = {m[i][0] == -INFINITY ? 0.f : m[i][0], m[i][1] == -INFINITY ? 0.f : m[i][1]};
        if (E4M3 && __builtin_expect(far_scales, 0)) {
#pragma unroll
          for (int z = 0; z < NS; ++z)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const float2 e = *reinterpret_cast<const float2*>(&scales[warp][stage][E4M3 ? 1 : 0][E4M3 ? 16 * z + 8 * n + 2 * q4 : 0]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float a = exp2_fast(0.5f * (s[z][i][n][2 * h] - e.x - from[h]) - kRowsShift / 2);
                const float b = exp2_fast(0.5f * (s[z][i][n][2 * h + 1] - e.y - from[h]) - kRowsShift / 2);
                l[i][h] = fmaf(b, b, fmaf(a, a, l[i][h]));
              }
              if (i == 0) inv[z][n][0] = inv[z][n][1] = 0.f;
            }
        }
#pragma unroll
        for (int z = 0; z < NS; ++z)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float a = exp2_fast(s[z][i][n][2 * h] - from[h]), b = exp2_fast(s[z][i][n][2 * h + 1] - from[h]);
              if (E4M3) {
                l[i][h] = fmaf(b, inv[z][n][1], fmaf(a, inv[z][n][0], l[i][h]));
                pa[z][i][2 * n + h] = pack_f16(a, b);
              } else {
                l[i][h] += a + b;
                pa[z][i][2 * n + h] = pack_bf16(a, b);
              }
            }
      }
      if (!E4M3) {
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t vb[4];
          const int k = (lane / 8 & 1) * 8 + lane % 8, c = (d % 4) * 2 + lane / 16;
          ldsm4_t(vb, vs_base + (d / 4) * S::half_tile + k * 128 + ((c ^ (k & 7)) << 4));
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            mma_16<false>(o[i][2 * d], pa[0][i], vb[0], vb[1]);
            mma_16<false>(o[i][2 * d + 1], pa[0][i], vb[2], vb[3]);
          }
        }
      } else {
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int z = 0; z < NS; ++z) {
            // pairs of dimensions move as one 16-bit element; even and odd ones are tiles of their own
            uint32_t vb[4];
            const int k = 16 * z + (lane / 8 & 1) * 8 + lane % 8, c = 2 * d + lane / 16;
            ldsm4_t(vb, vs_base + k * S::row_bytes + ((D == 128 ? c ^ (k & 7) : c ^ (k >> 1 & 3)) << 4));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t e0, o0, e1, o1;
              e4m3_f16(__byte_perm(vb[2 * j], 0, 0x3120), &e0, &o0);
              e4m3_f16(__byte_perm(vb[2 * j + 1], 0, 0x3120), &e1, &o1);
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                mma_16<true>(o[i][4 * d + 2 * j], pa[z][i], e0, e1);
                mma_16<true>(o[i][4 * d + 2 * j + 1], pa[z][i], o0, o1);
              }
            }
          }
      }
      if (edge || by_hand) fence_proxy_async();     // what was written here comes before the next copy
      __syncwarp();
      bring(stage);
      if (++stage == S::stages) stage = 0, phase ^= 1;
    }

    // ------------------------------------------------ join the warps' positions
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
        l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
        if (q4 == 0) {
          const int row = i * 16 + 8 * h + r8;
          sm_m[warp][row] = m[i][h];
          sm_l[warp][row] = l[i][h];
        }
      }
    __syncthreads();
    float mine[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = i * 16 + 8 * h + r8;
        float top = sm_m[0][row];
#pragma unroll
        for (int w = 1; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w][row]);
        mine[i][h] = top == -INFINITY ? 1.f : exp2_fast(m[i][h] - top);
      }
    for (int w = 0; w < kRowsWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* row = o_sm + (i * 16 + 8 * h + r8) * S::pitch;
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
      __syncthreads();
    }
    if (odd) {
      const int k1 = min(sees[M - 1], W.b * KT);
      if (E4M3) {
        // values of NaN: rows that see the first of them
        for (int k = W.a * KT + threadIdx.x; k < k1; k += kRowsThreads) {
          int slot;
          const int page = paged_lookup(A.C, W.row, k, &slot);
          if (page >= 0 && A.C.v_exp[page * A.C.exp_bytes + (long long)W.head * A.C.page_size + slot] > kAttendTop) atomicMin(&first_nan, k);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < M * D; i += kRowsThreads)
          if (first_nan < sees[i / D]) o_sm[i / D * S::pitch + i % D] = __uint_as_float(0x7fc00000u);
      } else {
        // values that are not finite at positions that only some rows see
        for (int k = max(fewest, W.a * KT); k < k1; ++k) {
          int slot;
          const int page = paged_lookup(A.C, W.row, k, &slot);
          if (page < 0) continue;
          const uint16_t* v = reinterpret_cast<const uint16_t*>(A.C.v + page * A.C.page_bytes) + ((long long)W.head * A.C.page_size + slot) * D;
          for (int d = threadIdx.x; d < D; d += kRowsThreads) {
            const float x = __uint_as_float((uint32_t)v[d] << 16);
            if (isfinite(x)) continue;
            for (int row = 0; row < M; ++row)
              if (k < sees[row]) o_sm[row * S::pitch + d] += x;
          }
        }
      }
      __syncthreads();
    }
    const bool whole = W.whole();
    const int item = W.item_begin();
    int c0 = 0, c1 = 0;
    if (!whole) share_parts(share, item, W.tiles, &c0, &c1);
    if (!whole) {
      float* part = A.parts + ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0)) * S::part_floats;
      for (int i = threadIdx.x; i < M * D / 4; i += kRowsThreads) {
        const int row = i / (D / 4), d = i % (D / 4) * 4;
        __stcg(reinterpret_cast<float4*>(part + row * D + d), *reinterpret_cast<float4*>(o_sm + row * S::pitch + d));
      }
      if (threadIdx.x < M) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w][threadIdx.x]);
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w)
          sum += times_exp2(sm_l[w][threadIdx.x], top == -INFINITY ? 0.f : sm_m[w][threadIdx.x] - top);
        __stcg(part + M * D + threadIdx.x, top);
        __stcg(part + M * D + M + threadIdx.x, sum);
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const unsigned had = atomicAdd(&A.joined[c0], 1u);
        last_part = had == (unsigned)(c1 - c0);
        if (last_part) A.joined[c0] = 0;
        __threadfence();
      }
      __syncthreads();
    }
    // The parts' maxima first, then what they add up to: no part's loads wait for the part before.
    constexpr int ways = kRowsThreads / M;
    if (whole ? threadIdx.x < M : last_part) {
      const int row = threadIdx.x % M;
      float top = -INFINITY;
      if (whole) {
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) top = fmaxf(top, sm_m[w][row]);
      } else {
#pragma unroll 4
        for (int c = c0 + threadIdx.x / M; c <= c1; c += ways)
          top = fmaxf(top, __ldcg(A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats + M * D + row));
      }
      tops[threadIdx.x / M][row] = top;
    }
    __syncthreads();
    if (whole || last_part) {
      for (int i = threadIdx.x; i < rows * (D / 8); i += kRowsThreads) {
        const int row = i / (D / 8), d = i % (D / 8) * 8;
        float x[8], top = tops[0][row], sum = 0.f;
        if (whole) {
#pragma unroll
          for (int w = 0; w < kRowsWarps; ++w) sum += times_exp2(sm_l[w][row], top == -INFINITY ? 0.f : sm_m[w][row] - top);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = o_sm[row * S::pitch + d + e];
        } else {
#pragma unroll
          for (int w = 1; w < ways; ++w) top = fmaxf(top, tops[w][row]);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const float* part = A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats;
            const float pm = __ldcg(part + M * D + row), pl = __ldcg(part + M * D + M + row);
            const float4 a = __ldcg(reinterpret_cast<const float4*>(part + row * D + d));
            const float4 b = __ldcg(reinterpret_cast<const float4*>(part + row * D + d + 4));
            const float far = top == -INFINITY ? 0.f : pm - top, add = exp2_fast(far);
            sum += times_exp2(pl, far);
            const float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(y[e], add, x[e]);
          }
        }
        const long long at = out_at[row];
        float by = sum == 0.f ? 1.f : 1.f / sum;
        if (E4M3) by *= __uint_as_float((127 - kRowsShift) << 23);
        *reinterpret_cast<uint4*>(A.out + at * D + d) =
            make_uint4(pack_bf16(x[0] * by, x[1] * by), pack_bf16(x[2] * by, x[3] * by), pack_bf16(x[4] * by, x[5] * by),
                       pack_bf16(x[6] * by, x[7] * by));
        if (d == 0 && A.lse)
          A.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum) + (E4M3 ? kRowsShift : 0)) * 0.6931471805599453f;
      }
    }
    if (threadIdx.x == 0 && failed && A.flags) atomicOr(&A.flags[W.row], (uint32_t)SPEC_F_TIMEOUT);
    __syncthreads();
  }
  mbar_settle(&failed);
}

template <int D, bool E4M3, int MT>
static int launch_rows(const AttendArgs& A, const CUtensorMap* maps, cudaStream_t st) {
  using S = RowsShape<D, E4M3, MT>;
  static_assert(S::stages >= 2, "a ring needs two stages");
  const auto kernel = attend_rows_kernel<D, E4M3, MT>;
  static std::atomic<unsigned long long> allowed;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), S::smem, &allowed)) return SPEC_E_CUDA;
  kernel<<<S::ctas * 152, kRowsThreads, S::smem, st>>>(A, maps[0], maps[1]);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <int D, bool E4M3>
static int launch_rows_of(const AttendArgs& A, int rows, const CUtensorMap* maps, cudaStream_t st) {
  // 16 rows where they suffice: 64x1 tokens of group 8 at 8000 105 us, with 32 rows 124; 64x3 of group 4 193 and 226
  return rows <= 16 ? launch_rows<D, E4M3, 1>(A, maps, st) : launch_rows<D, E4M3, 2>(A, maps, st);
}

int launch_attend_rows(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st) {
  if (A.C.D == 128) return e4m3 ? launch_rows_of<128, true>(A, rows, maps, st) : launch_rows_of<128, false>(A, rows, maps, st);
  return e4m3 ? launch_rows_of<64, true>(A, rows, maps, st) : launch_rows_of<64, false>(A, rows, maps, st);
}

}  // namespace specv
