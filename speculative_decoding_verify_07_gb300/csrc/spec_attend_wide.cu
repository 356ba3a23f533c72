// Attention of many query rows over the cache: chunks of a prompt, long drafts,
// wide groups.
//
// Bound by the tensor cores: 4 D operations for each (query row, position).  A
// CTA walks the positions in tiles of 128 with tcgen05: S = Q K^T into tensor
// memory, softmax by one thread a row, P back into tensor memory over S,
// O += P V.  Two groups of four softmax warps keep the matrix unit busy, which
// works for one while the other computes: on two tiles of 128 query rows, or,
// where the item has no more than 128, on every other tile of positions of the
// same rows, with two O that are joined at the end.  P is bf16 (the values are;
// its rounding changes a weight by up to 2^-8), everything else float32.
//
// The maximum only moves when a row's scores pass it by 2^8, so O, which stays
// in tensor memory, is rescaled a few times a row and not at every tile.
//
// Warps: eight for softmax, which take registers from the others to hold a row
// of S; one that issues the matrix instructions; one each that copies keys and
// values by TMA, a box a run of positions within a page; four that make the
// copies ready.  A 16-bit cache lands in the swizzled layout that the matrix unit
// reads, and only the values at the edge of what rows see are looked over.  8-bit
// codes land in half of their stage and are widened in place to bf16 with their
// power-of-two scale (exact), so the rest of the kernel is the same.
//
// Measured: 2x2048 tokens at 9000 positions, 32 query heads of 128, bf16, 415 us,
// 1310 TFLOP/s (70 % of cuBLAS's rate here; by calls back to back 427 us): the matrix
// pipe is busy in 55 % of the cycles and issue slots in 39, and each group's chain
// from scores to weights to products, two in flight, waits for itself.
// 8 bits: 2x1024 at 8000 227 us, 930 TFLOP/s: widening both operands takes as long
// as the softmax.  Heads of 64 have half the products for the same softmax.
#include "spec_attend.cuh"

namespace specv {

constexpr int kWideKT = 128;
constexpr int kNowhere = 0x7fffffff;
constexpr float kWideSlack = 8.f;
constexpr int kWideLarge = 30;       // scores of 2^30 and more are taken for one of that size (see below)
constexpr int kWideWhole = 6;       // items of so few tiles stay in one CTA

template <int D, bool E4M3, bool SPLIT>
struct WideShape {
  static constexpr int QT = SPLIT ? 1 : 2;                    // tiles of query rows
  static constexpr int M = 128 * QT;
  static constexpr int halves = D / 64;                       // 128-byte columns of a bf16 row
  static constexpr int half_tile = kWideKT * 128;
  static constexpr int tile = halves * half_tile;             // 128 rows of Q, K or V
  // what is left of the 227 KB after Q, the alignment and the small arrays, in tiles: keys have the odd one, they are
  // waited for first
  static constexpr int room = (227 * 1024 - 1024 - (E4M3 ? 3584 : 1024) - QT * tile) / tile;
  static constexpr int k_stages = (room + 1) / 2 > 4 ? 4 : (room + 1) / 2;
  static constexpr int v_stages = room / 2 > 4 ? 4 : room / 2;
  static constexpr int smem = 1024 + (QT + k_stages + v_stages) * tile;
  static constexpr int columns = 512;                         // of tensor memory: two S of 128, two O of D
  static constexpr int part_floats = M * (D + 2);
};

constexpr int kWideThreads = 512;      // two groups of softmax warps, one that brings, one of which a warp multiplies
// A group's registers: 2 * 128 * (184 + 72) = 512 * 128, what the block was launched with.
constexpr int kWideMore = 184, kWideLess = 72;

// Shared-memory operand with 128-byte swizzle: address, distance between
// 64-element columns (of a transposed operand) and between groups of 8 rows.
__device__ __forceinline__ uint64_t wide_desc(uint32_t smem, uint32_t columns) {
  return (uint64_t)((smem >> 4) & 0x3fff) | (uint64_t)(columns >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// bf16 x bf16 -> float32, 128 rows by n columns.
__device__ __forceinline__ constexpr uint32_t wide_instr(int n, bool b_transposed) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_transposed ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 | (128u / 16) << 24;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(instr), "r"((uint32_t)accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(instr), "r"((uint32_t)accumulate)
      : "memory");
}
// One thread of the converged warp, and known to the compiler as one: operands
// of the matrix instructions then go straight to uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void mma_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
      "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Whether any thread of the four warps that make tiles ready says so; a barrier among them.
__device__ __forceinline__ bool ready_any(bool mine) {
  uint32_t any;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, 2, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
               : "=r"(any) : "r"((uint32_t)mine) : "memory");
  return any != 0;
}
__device__ __forceinline__ void wide_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }   // the softmax warps

// Two e4m3 codes in the upper bytes of 16-bit halves as bf16, times `scale` (a
// power of two in both halves).  The code's bits, shifted, are a bf16 number
// 2^-120 of its size, which the scale makes up for; the product is exact.
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t high, uint32_t scale) {
  uint32_t w = ((high >> 4) & 0x07f007f0u) | (high & 0x80008000u);
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(scale));
  return w;
}
constexpr uint32_t kWideExp = 134;     // the largest exponent byte whose scale, times 2^120, is a bf16 number

struct WideBars {
  unsigned long long k_raw[4], k_full[4], k_empty[4];      // keys: codes copied, ready, read
  unsigned long long v_raw[4], v_full[4], v_empty[4];      // values: copied, ready, read
  unsigned long long q_full[2], s_full[2], p_half[2], p_full[2], o_full[2];
};

template <int D, bool E4M3, bool SPLIT>
__global__ void __launch_bounds__(kWideThreads, 1)
    attend_wide_kernel(const AttendArgs A, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using S = WideShape<D, E4M3, SPLIT>;
  constexpr int M = S::M, KT = kWideKT, KST = S::k_stages, VST = S::v_stages, QT = S::QT;
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) WideBars bar;
  __shared__ unsigned there[8][4], v_there[8][4];      // which positions of the tile are there, for the last eight tiles
  __shared__ AttendShare share;
  __shared__ uint32_t scales[2][2][E4M3 ? KT : 1];    // 8-bit cache: the last two tiles' scales (in both halves, times 2^120)
  __shared__ uint32_t tmem_base;
  __shared__ int failed, last_part;
  __shared__ int odd_at[16];     // for the last items: the first position whose value is not finite, where that needs care
  unsigned char* const base = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  unsigned char* const k_sm = base + QT * S::tile;
  unsigned char* const v_sm = k_sm + KST * S::tile;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int ready_warp = 8, mma_warp = 12, k_warp = 13, v_warp = 14;
  // one 64-byte row of codes would not begin at a multiple of 128 bytes, where a copy has to land: such rows lie apart
  const int pitch = D == 64 && A.box == 1 ? 128 : D;

  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < 16; ++i) odd_at[i] = kNowhere;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_raw[i], 1);
      mbar_init(&bar.k_full[i], E4M3 ? 128 : 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_raw[i], 1);
      mbar_init(&bar.v_full[i], 128);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 128);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_half[i], 128);
      mbar_init(&bar.p_full[i], 128);
      mbar_init(&bar.o_full[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)), "n"(S::columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tmem_before();
  }
  attend_share<M, KT, kWideThreads, kWideWhole>(A, &share, reinterpret_cast<long long*>(base));   // (shared memory is free yet)
  fence_proxy_async();
  tmem_after();
  const uint32_t tmem = tmem_base;
  AttendWalk<M, KT, true> W(A, share);

  if (warp >= ready_warp && warp < mma_warp) {
    // --------------------------------------------- keys and values made ready
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideLess));
    int n = 0, segment = 0;                      // tiles and items so far
    const int tid = threadIdx.x - ready_warp * 32;
    while (W.next()) {
      const int fewest = attend_sees(A, W.R, attend_token(A, W.qt * M));
      const int limit = attend_sees(A, W.R, attend_token(A, min((W.qt + 1) * M, W.R.n * A.group) - 1));
      if (tid == 0) odd_at[(segment + 6) & 15] = kNowhere;     // (no warp is six items ahead of another)
      // 8-bit cache: this thread's position, its page's entry two tiles ahead and its exponents one tile ahead
      int entry = -1, slot = 0;
      uint32_t ke = 0, ve = 0;
      auto look = [&](int t) {
        const int pos = t * KT + tid;
        entry = pos < limit ? paged_entry(A.C, W.row, pos, &slot) : -1;
      };
      auto fetch = [&]() {
        const int page = paged_page(A.C, entry);
        ke = ve = 0;
        if (page >= 0) {
          const long long e = page * A.C.exp_bytes + (unsigned)(W.head * A.C.page_size + slot);
          ke = max((uint32_t)A.C.k_exp[e], 1u);
          ve = max((uint32_t)A.C.v_exp[e], 1u);
        }
      };
      if (E4M3) {
        look(W.a);
        fetch();
        if (W.a + 1 < W.b) look(W.a + 1);
      }
      for (int t = W.a; t < W.b; ++t, ++n) {
        const int kst = n % KST, vst = n % VST;
        if (E4M3) {
          uint32_t bits[2] = {ke == 0 ? 0u : (ke + 120) << 7, ve == 0 ? 0u : (ve + 120) << 7};
          const bool over = max(ke, ve) > kWideExp;
          if (over) {
            // what does not fit is made up for below; a value of NaN is cleared here and put in at the item's end
            if (ve > kAttendTop) atomicMin(&odd_at[segment & 15], t * KT + tid);
            if (ke > kWideExp) bits[0] = ke < 255 ? (kWideExp + 120) << 7 : 0x7fc0u;
            if (ve > kWideExp) bits[1] = ve <= kAttendTop ? (kWideExp + 120) << 7 : 0u;
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) scales[n & 1][v][E4M3 ? tid : 0] = bits[v] * 0x10001u;
          if (t + 1 < W.b) {
            fetch();
            if (t + 2 < W.b) look(t + 2);
          }
          const bool rest = ready_any(over);       // (and every scale is written)
#pragma unroll 1
          for (int v = 0; v < 2; ++v) {
            unsigned char* const tile = v ? v_sm + vst * S::tile : k_sm + kst * S::tile;
            mbar_await(v ? &bar.v_raw[vst] : &bar.k_raw[kst], (v ? n / VST : n / KST) & 1, &failed);
            // The codes lie in the last 128 D bytes of the stage (in all of it where rows lie apart).  Of 128 dimensions
            // the first 64 go to the other half as they are read; what goes where codes lie is read first.
            unsigned char* const codes = tile + (S::halves - 1) * S::half_tile;
            const int part = tid % 4, row0 = tid / 4;          // 16 codes of rows row0, row0 + 32, ...
            uint32_t scale[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) scale[i] = scales[n & 1][v][E4M3 ? row0 + 32 * i : 0];
#pragma unroll 1
            for (int h = 0; h < S::halves; ++h) {
              uint4 w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(codes + (row0 + 32 * i) * pitch + h * 64 + part * 16);
              if (h == S::halves - 1) asm volatile("bar.sync 2, 128;" ::: "memory");
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                unsigned char* const to = tile + h * S::half_tile + (row0 + 32 * i) * 128;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  uint4 y = make_uint4(e4m3_bf16(__byte_perm(x[2 * j], 0, 0x1404), scale[i]), e4m3_bf16(__byte_perm(x[2 * j], 0, 0x3424), scale[i]),
                                       e4m3_bf16(__byte_perm(x[2 * j + 1], 0, 0x1404), scale[i]), e4m3_bf16(__byte_perm(x[2 * j + 1], 0, 0x3424), scale[i]));
                  *reinterpret_cast<uint4*>(to + (((part * 2 + j) ^ (row0 & 7)) << 4)) = y;
                }
              }
              if (rest) {
                // a scale over 2^7: what it was cut by
#pragma unroll 1
                for (int i = 0; i < 4; ++i) {
                  const int pos = t * KT + row0 + 32 * i;
                  int slot;
                  const int page = pos < limit ? paged_lookup(A.C, W.row, pos, &slot) : -1;
                  uint32_t e = 0;
                  if (page >= 0) e = (v ? A.C.v_exp : A.C.k_exp)[page * A.C.exp_bytes + (unsigned)(W.head * A.C.page_size + slot)];
                  if (e <= kWideExp || e > (v ? kAttendTop : 254u)) continue;
                  const uint32_t more = ((e - kWideExp + 127) << 7) * 0x10001u;
                  for (int j = 0; j < 2; ++j) {
                    uint4* p = reinterpret_cast<uint4*>(tile + h * S::half_tile + (row0 + 32 * i) * 128 + (((part * 2 + j) ^ (row0 & 7)) << 4));
                    uint4 y = *p;
                    asm("mul.rn.bf16x2 %0, %0, %4;\nmul.rn.bf16x2 %1, %1, %4;\nmul.rn.bf16x2 %2, %2, %4;\nmul.rn.bf16x2 %3, %3, %4;"
                        : "+r"(y.x), "+r"(y.y), "+r"(y.z), "+r"(y.w) : "r"(more));
                    *p = y;
                  }
                }
              }
            }
            fence_proxy_async();
            mbar_arrive(v ? &bar.v_full[vst] : &bar.k_full[kst]);
          }
        } else {
          // No value of weight zero may be NaN: positions that are not there are cleared, and what is not finite of
          // those that only some rows see is cleared and remembered.
          mbar_await(&bar.v_raw[vst], n / VST & 1, &failed);
          const unsigned* mask = v_there[n & 7];
          if ((t + 1) * KT > fewest || (mask[0] & mask[1] & mask[2] & mask[3]) != ~0u) {
            int found = kNowhere;
            for (int i = tid; i < KT * S::halves * 8; i += 128) {
              const int k = i / (S::halves * 8), c = i % (S::halves * 8);
              unsigned char* p = v_sm + vst * S::tile + c / 8 * S::half_tile + k * 128 + (c % 8) * 16;   // any order of a row's columns
              if (!(mask[k / 32] >> (k & 31) & 1)) {
                *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
              } else if (t * KT + k >= fewest) {
                uint4 w = *reinterpret_cast<uint4*>(p);
                uint32_t* x = reinterpret_cast<uint32_t*>(&w);
                bool bad = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if ((x[j] & 0x7f80u) == 0x7f80u) x[j] &= 0xffff0000u, bad = true;
                  if ((x[j] & 0x7f800000u) == 0x7f800000u) x[j] &= 0xffffu, bad = true;
                }
                if (bad) {
                  *reinterpret_cast<uint4*>(p) = w;
                  found = min(found, t * KT + k);
                }
              }
            }
            if (found != kNowhere) atomicMin(&odd_at[segment & 15], found);
            fence_proxy_async();
          }
          mbar_arrive(&bar.v_full[vst]);
        }
      }
      ++segment;
    }
  } else if (warp >= mma_warp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideLess));
    if (warp == k_warp || warp == v_warp) {
      // --------------------------------------------- copies of keys or values
      const bool v = warp == v_warp;
      const int stages = v ? VST : KST, boxes = KT / A.box;
      unsigned char* const sm = v ? v_sm : k_sm;
      const CUtensorMap* map = v ? &vmap : &kmap;
      unsigned starts[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) starts[j] = attend_starts(A.box, j);
      int n = 0;
      int next_page[4], next_slot[4];            // this lane's positions of the next tile
      while (W.next()) {
        const int limit = attend_sees(A, W.R, attend_token(A, min((W.qt + 1) * M, W.R.n * A.group) - 1));
        auto look = [&](int t) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int pos = t * KT + 32 * j + lane;
            next_slot[j] = 0;
            next_page[j] = pos < limit ? paged_lookup(A.C, W.row, pos, &next_slot[j]) : -1;
            if (next_page[j] < 0 && pos < limit && A.flags) atomicOr(&A.flags[W.row], (uint32_t)SPEC_F_BAD_IDX);
          }
        };
        look(W.a);
        for (int t = W.a; t < W.b; ++t, ++n) {
          const int st = n % stages;
          int page[4], slot[4];
          unsigned mask[4], copies = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            page[j] = next_page[j];
            slot[j] = next_slot[j];
            mask[j] = __ballot_sync(0xffffffffu, page[j] >= 0);
            copies += __popc(mask[j] & starts[j]);
          }
          if (t + 1 < W.b) look(t + 1);
          const uint32_t bytes = copies * A.box * D * (E4M3 ? 1 : 2);
          unsigned long long* full = v ? &bar.v_raw[st] : E4M3 ? &bar.k_raw[st] : &bar.k_full[st];
          mbar_await(v ? &bar.v_empty[st] : &bar.k_empty[st], (n / stages & 1) ^ 1, &failed);
          if (lane < 4) (v ? v_there : there)[n & 7][lane] = lane == 0 ? mask[0] : lane == 1 ? mask[1] : lane == 2 ? mask[2] : mask[3];
          __syncwarp();
          const bool go = !mbar_given_up(&failed);       // (lanes may differ on it: they meet again whatever it is)
          if (lane == 0 && go) mbar_arrive_expect_tx(full, bytes);
          __syncwarp();
          const uint32_t to = smem_u32(sm + st * S::tile + (E4M3 ? (S::halves - 1) * S::half_tile : 0));
          for (int b0 = 0; b0 < boxes && bytes; b0 += 32) {
            const int at = ((b0 + lane) * A.box) & 127, from = at & 31;
            int p = -1, s = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int pj = __shfl_sync(0xffffffffu, page[j], from), sj = __shfl_sync(0xffffffffu, slot[j], from);
              if (at / 32 == j) p = pj, s = sj;
            }
            if (b0 + lane < boxes && p >= 0 && go) {
              if (E4M3) {
                tma_load_4d(to + at * pitch, map, 0, s, W.head, p, full);
              } else {
#pragma unroll
                for (int h = 0; h < S::halves; ++h) tma_load_4d(to + h * S::half_tile + at * 128, map, h * 64, s, W.head, p, full);
              }
            }
          }
        }
      }
    } else if (warp == mma_warp) {
      // ----------------------------------------------------- matrix products
      // Step i of a segment is for group i % 2: two steps a tile, or one.
      const bool leader = elect_one();
      int n = 0, segment = 0;
      uint32_t p_phase = 0;                      // a bit a group
      constexpr uint32_t s_instr = wide_instr(KT, false), o_instr = wide_instr(D, true);
      constexpr int per = SPLIT ? 1 : 2;
      auto scores = [&](int step) {
        const int group = step & 1, at_n = n + step / per, st = at_n % KST;
        if (step < per || (!SPLIT && step == 1)) mbar_await(&bar.q_full[SPLIT ? 0 : group], segment & 1, &failed);
        mbar_await(&bar.k_full[st], at_n / KST & 1, &failed);
        tmem_after();
        if (leader) {
          const uint64_t a = wide_desc(smem_u32(base + (SPLIT ? 0 : group) * S::tile), 0), b = wide_desc(smem_u32(k_sm + st * S::tile), 0);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t at = (k / 4 * S::half_tile + k % 4 * 32) >> 4;
            mma_ss(tmem + group * 128, a + at, b + at, s_instr, k > 0);
          }
          mma_commit(&bar.s_full[group]);
          if (SPLIT || group == 1) mma_commit(&bar.k_empty[st]);
        }
      };
      auto values = [&](int step) {
        const int group = step & 1, at_n = n + step / per, st = at_n % VST;
        mbar_await(&bar.v_full[st], at_n / VST & 1, &failed);
        const uint64_t b = wide_desc(smem_u32(v_sm + st * S::tile), S::half_tile);
        // the first half of the weights is multiplied while the second is computed
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mbar_await(h ? &bar.p_full[group] : &bar.p_half[group], p_phase >> group & 1, &failed);
          tmem_after();
          if (leader) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              mma_ts(tmem + 256 + group * D, tmem + group * 128 + k * 8, b + (k * 2048 >> 4), o_instr, step > 1 || k > 0);
          }
        }
        p_phase ^= 1u << group;
        if (leader) {
          mma_commit(&bar.o_full[group]);
          if (SPLIT || group == 1) mma_commit(&bar.v_empty[st]);
        }
      };
      while (W.next()) {
        const int steps = (W.b - W.a) * per;
#pragma unroll 1
        for (int step = -2; step < steps; ++step) {
          // the scores run two steps ahead, each in the place of the weights that the products before have read
          if (step >= 0) values(step);
          if (step + 2 < steps) scores(step + 2);
        }
        n += W.b - W.a;
        ++segment;
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideMore));
    const int group = warp / 4, row = threadIdx.x % 128, qt = SPLIT ? 0 : group;   // this thread's row of its query tile
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16), s_at = lanes + group * 128, o_at = lanes + 256;
    // a negative scale turns the queries' signs, so the largest score is that of the largest product
    // (a scale of zero is as good as one of 1e-30, and what is not seen stays at minus infinity)
    const float scale = fmaxf(fabsf(A.scale_log2), 1e-30f);
    const uint32_t turn = A.scale_log2 < 0.f ? 0x80008000u : 0u;
    float* const stats = reinterpret_cast<float*>(base);
    int done = 0, n = 0, segment = 0;          // this group's steps so far; tiles; items
    constexpr int across = D / 8, turns = across;      // lanes a row of Q or of the result, and turns for a warp's 32 rows
    while (W.next()) {
      const AttendRow R = W.R;
      const int item_row = W.row, item_head = W.head, item_qt = W.qt, item_tiles = W.tiles, item_a = W.a, item_b = W.b;
      const bool whole = W.whole();
      const int item = W.item_begin();
      const int mine = item_qt * M + qt * 128 + row, rows = R.n * A.group;
      const bool real = mine < rows;
      const int token = attend_token(A, min(mine, rows - 1)), head = item_head * A.group + min(mine, rows - 1) - token * A.group;
      const int lim = attend_sees(A, R, token), fewest = attend_sees(A, R, attend_token(A, min(item_qt * M + qt * 128, rows - 1)));
      if (!SPLIT || group == 0) {
        // the products with the last Q are done: their results have been waited for
        const unsigned live = __ballot_sync(0xffffffffu, real);
        const long long q_row = (R.first + token) * A.q_token + (long long)head * D;
        uint4 q[turns];
#pragma unroll
        for (int i = 0; i < turns; ++i) {
          const int from = i * (32 / across) + lane / across;
          const long long at = __shfl_sync(0xffffffffu, q_row, from);
          q[i] = make_uint4(0, 0, 0, 0);
          if (live >> from & 1) q[i] = __ldg(reinterpret_cast<const uint4*>(A.q + at) + lane % across);
        }
#pragma unroll
        for (int i = 0; i < turns; ++i) {
          const int r = warp % 4 * 32 + i * (32 / across) + lane / across, c = lane % across;
          q[i].x ^= turn, q[i].y ^= turn, q[i].z ^= turn, q[i].w ^= turn;
          *reinterpret_cast<uint4*>(base + qt * S::tile + c / 8 * S::half_tile + r * 128 + (((c % 8) ^ (r & 7)) << 4)) = q[i];
        }
        fence_proxy_async();
        mbar_arrive(&bar.q_full[SPLIT ? 0 : group]);
      }
      float m = -INFINITY, l = 0.f, by = scale, from = 0.f;     // weights are 2^(by * product + from)
      const int began = done;
      for (int t = item_a + (SPLIT ? group : 0); t < item_b; t += SPLIT ? 2 : 1, ++done) {
        mbar_await(&bar.s_full[group], done & 1, &failed);
        tmem_after();
        uint32_t s[128];
        tmem_ld32(s_at, s);
        tmem_ld32(s_at + 32, s + 32);
        const unsigned* mask = there[(n + t - item_a) & 7];
        const bool edge = (t + 1) * KT > fewest || (mask[0] & mask[1] & mask[2] & mask[3]) != ~0u;
        tmem_wait_ld();
        tmem_ld32(s_at + 64, s + 64);
        tmem_ld32(s_at + 96, s + 96);
        float high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        if (edge) {
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int left = lim - t * KT - c * 32;
            const unsigned seen = mask[c] & (left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen >> i & 1)) s[c * 32 + i] = 0xff800000u;
          }
        }
#pragma unroll
        for (int i = 0; i < 64; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) high[j] = fmaxf(high[j], fmaxf(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 4])));
        tmem_wait_ld();
#pragma unroll
        for (int i = 64; i < 128; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) high[j] = fmaxf(high[j], fmaxf(__uint_as_float(s[i + j]), __uint_as_float(s[i + j + 4])));
        float top = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
        top *= scale;
        float keep = 1.f;
        if (top > m + kWideSlack) {
          keep = exp2_fast(m - top);
          m = top;
          // The multiply-add of the weights leaves what m lost by rounding, 2^6 at 2^30 and soon more than an exponent.
          // From there on a score that is smaller at all is smaller by 2^6: brought to that size by a power of two, the
          // largest keep the weight and all others lose it, as they should.
          const int over = max((int)(__float_as_uint(m) >> 23 & 255) - (127 + kWideLarge), 0);
          const float cut = __uint_as_float((uint32_t)(127 - over) << 23);
          by = scale * cut;
          from = -m * cut;
        }
        if (__any_sync(0xffffffffu, keep != 1.f)) {
          l *= keep;
          if (done > began) {
            mbar_await(&bar.o_full[group], (done - 1) & 1, &failed);
            tmem_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(o_at + group * D + c * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
              tmem_st16(o_at + group * D + c * 16, o);
            }
          }
        }
        const float2 scale2 = make_float2(by, by), from2 = make_float2(from, from);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float2 x = fma2(make_float2(__uint_as_float(s[c * 32 + i]), __uint_as_float(s[c * 32 + i + 1])), scale2, from2);
            x.x = exp2_fast(x.x);
            x.y = exp2_fast(x.y);
            sum[i / 2 & 1] = add2(sum[i / 2 & 1], x);
            p[i / 2] = pack_bf16(x.x, x.y);
          }
          tmem_st16(s_at + c * 16, p);
          if (c == 1) {
            tmem_wait_st();
            tmem_before();
            mbar_arrive(&bar.p_half[group]);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tmem_before();
        mbar_arrive(&bar.p_full[group]);
      }
      n += item_b - item_a;
      // ------------------------------------------------------------ the end
      if (done > began) mbar_await(&bar.o_full[group], (done - 1) & 1, &failed);
      tmem_after();
      if (SPLIT) {
        wide_sync();            // the other group's products with Q are done too: its place is free until the next item
        stats[group * 256 + row] = m;
        stats[group * 256 + 128 + row] = l;
        wide_sync();
      }
      const int odd = odd_at[segment & 15], k1 = min(lim, item_b * KT);
      // this thread's columns of its row: all of them, or half of what two groups have
      constexpr int cols = SPLIT ? D / 2 : D;
      const int d0 = SPLIT ? group * cols : 0;
      float f0 = 1.f, f1 = 0.f;
      bool two = false;
      if (SPLIT) {
        const float m0 = stats[row], m1 = stats[256 + row];
        two = item_b - item_a > 1;
        m = two ? fmaxf(m0, m1) : m0;
        const float ref = m == -INFINITY ? 0.f : m;
        f0 = exp2_fast(m0 - ref);
        f1 = exp2_fast(m1 - ref);
        l = stats[128 + row] * f0 + (two ? stats[384 + row] * f1 : 0.f);
      }
      int c0 = 0, c1 = 0;
      if (!whole) share_parts(share, item, item_tiles, &c0, &c1);
      float* const part = A.parts + ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0)) * S::part_floats;
      const long long out_row = (long long)(R.first + token) * A.hq + head;
      const float inv = l == 0.f ? 1.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < cols / 32; ++c) {
        const int d = d0 + c * 32;
        uint32_t r[32];
        tmem_ld32(o_at + (SPLIT ? 0 : group * D) + d, r);
        tmem_wait_ld();
        float* o = reinterpret_cast<float*>(r);
        if (SPLIT) {
          uint32_t r1[32];
          if (two) tmem_ld32(o_at + D + d, r1);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = o[i] * f0 + (two ? __uint_as_float(r1[i]) * f1 : 0.f);
        }
        if (odd < k1) {
          if (E4M3) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(0x7fc00000u);
          } else {
            for (int k = odd; k < k1; ++k) {
              int slot;
              const int page = paged_lookup(A.C, item_row, k, &slot);
              if (page < 0) continue;
              const uint16_t* v = reinterpret_cast<const uint16_t*>(A.C.v + page * A.C.page_bytes) + ((long long)item_head * A.C.page_size + slot) * D + d;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float x = __uint_as_float((uint32_t)v[i] << 16);
                if (!isfinite(x)) o[i] += x;
              }
            }
          }
        }
        if (!real) {
          // (rows of padding)
        } else if (!whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            __stcg(reinterpret_cast<float4*>(part) + (d + i) / 4 * M + qt * 128 + row, make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const uint4 w = make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                                       pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
            const int cc = (d + i) / 8;
            if (SPLIT) *reinterpret_cast<uint4*>(A.out + out_row * D + d + i) = w;
            else *reinterpret_cast<uint4*>(base + qt * S::tile + cc / 8 * S::half_tile + row * 128 + (((cc % 8) ^ (row & 7)) << 4)) = w;
          }
        }
      }
      if (!SPLIT && whole) {
        // the warp's rows leave by way of Q's place, so that neighbouring lanes write neighbouring columns
        __syncwarp();
#pragma unroll
        for (int i = 0; i < turns; ++i) {
          const int from = i * (32 / across) + lane / across, r = warp % 4 * 32 + from, c = lane % across;
          const long long to = __shfl_sync(0xffffffffu, out_row, from);
          const uint4 w = *reinterpret_cast<const uint4*>(base + qt * S::tile + c / 8 * S::half_tile + r * 128 + (((c % 8) ^ (r & 7)) << 4));
          if (item_qt * M + qt * 128 + r < rows) *(reinterpret_cast<uint4*>(A.out + to * D) + c) = w;
        }
        __syncwarp();
      }
      if (whole && real && d0 == 0 && A.lse) A.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      if (!whole) {
        if (real && d0 == 0) {
          __stcg(part + M * D + qt * 128 + row, m);
          __stcg(part + M * D + M + qt * 128 + row, l);
        }
        __threadfence();
        wide_sync();
        if (threadIdx.x == 0) {
          const unsigned had = atomicAdd(&A.joined[c0], 1u);
          last_part = had == (unsigned)(c1 - c0);
          if (last_part) A.joined[c0] = 0;
          __threadfence();
        }
        wide_sync();
        if (last_part && real) {
          float high = -INFINITY, sum = 0.f;
          for (int c = c0; c <= c1; ++c) high = fmaxf(high, __ldcg(A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats + M * D + qt * 128 + row));
          const float ref = high == -INFINITY ? 0.f : high;
          for (int c = c0; c <= c1; ++c) {
            const float* p = A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats + M * D + qt * 128 + row;
            sum += __ldcg(p + M) * exp2_fast(__ldcg(p) - ref);
          }
          const float by = sum == 0.f ? 1.f : 1.f / sum;
          // neighbouring threads have neighbouring rows, and a part keeps four columns of all rows together
#pragma unroll 1
          for (int d = d0; d < d0 + cols; d += 32) {
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int c = c0; c <= c1; ++c) {
              const float* p = A.parts + ((size_t)c * 2 + (c == c0)) * S::part_floats;
              float4 y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = __ldcg(reinterpret_cast<const float4*>(p) + (d / 4 + i) * M + qt * 128 + row);
              const float f = exp2_fast(__ldcg(p + M * D + qt * 128 + row) - ref);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i].x += y[i].x * f, x[i].y += y[i].y * f, x[i].z += y[i].z * f, x[i].w += y[i].w * f;
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              *reinterpret_cast<uint4*>(A.out + out_row * D + d + 4 * i) =
                  make_uint4(pack_bf16(x[i].x * by, x[i].y * by), pack_bf16(x[i].z * by, x[i].w * by),
                             pack_bf16(x[i + 1].x * by, x[i + 1].y * by), pack_bf16(x[i + 1].z * by, x[i + 1].w * by));
          }
          if (d0 == 0 && A.lse) A.lse[out_row] = sum == 0.f ? -INFINITY : (high + log2f(sum)) * 0.6931471805599453f;
        }
      }
      if (failed && threadIdx.x == 0 && A.flags) atomicOr(&A.flags[item_row], (uint32_t)SPEC_F_TIMEOUT);
      tmem_before();
      ++segment;
      if (SPLIT) wide_sync();      // both O have been read before either is written again
    }
  }
  mbar_settle(&failed);
  tmem_before();
  __syncthreads();
  if (warp == mma_warp) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::columns) : "memory");
  }
}

template <int D, bool E4M3, bool SPLIT>
static int launch_wide(const AttendArgs& A, const CUtensorMap* maps, cudaStream_t st) {
  using S = WideShape<D, E4M3, SPLIT>;
  static_assert(S::v_stages >= 2, "a ring needs two stages");
  const auto kernel = attend_wide_kernel<D, E4M3, SPLIT>;
  static std::atomic<unsigned long long> allowed;
  if (!allow_shared(reinterpret_cast<const void*>(kernel), S::smem, &allowed)) return SPEC_E_CUDA;
  kernel<<<152, kWideThreads, S::smem, st>>>(A, maps[0], maps[1]);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

template <int D, bool E4M3>
static int launch_wide_of(const AttendArgs& A, int rows, const CUtensorMap* maps, cudaStream_t st) {
  // One tile of query rows where it suffices: 16x5 tokens of group 8 over up to 30000 76.8 us, with two tiles 79.7; 32x5 of group 16,
  // heads of 64, 66.5 and 74.0.  Above 128 rows two: 2x2048 tokens 415 us, with one tile 670; 16x17 of group 16 88 and 108.
  return rows <= 128 ? launch_wide<D, E4M3, true>(A, maps, st) : launch_wide<D, E4M3, false>(A, maps, st);
}

int launch_attend_wide(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st) {
  if (A.C.D == 128) return e4m3 ? launch_wide_of<128, true>(A, rows, maps, st) : launch_wide_of<128, false>(A, rows, maps, st);
  return e4m3 ? launch_wide_of<64, true>(A, rows, maps, st) : launch_wide_of<64, false>(A, rows, maps, st);
}

}  // namespace specv
