// What the attention kernels share: arguments, the division of the work over
// CTAs, and tensor maps of the cache.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/spec_verify.h"
#include "spec_device.cuh"
#include "spec_host.h"
#include "spec_paged.cuh"
#include "spec_tma.cuh"

namespace specv {

struct AttendArgs {
  PagedCache C;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  uint32_t* flags;
  long long q_token;     // elements from token to token of q
  int N, group, hq;
  int box;               // cache rows one copy brings: they lie in one page
  float inv_group;
  float scale_log2;      // scale * log2(e): scores are powers of two
  unsigned* joined;      // workspace: per CTA, how many parts of its last item have come
  float* parts;          // workspace: per CTA, two partial results
};

// 8-bit cache: values under a larger exponent byte are taken for NaN, by either kernel.
constexpr unsigned kAttendTop = 221;

// Workspace: a counter a CTA, then the partial results.
constexpr int kAttendCtas = 512;       // no launch has more
constexpr size_t kAttendCounters = kAttendCtas * sizeof(unsigned);

// ------------------------------------------------------- division of the work
//
// An item is (row, cache head, tile of M query rows), query rows being the
// row's (token, head of the group) pairs; its work is the tiles of KT positions
// that its last query row sees, one at least.  The tiles of all items, in the
// order row, head, query tile, position, are divided evenly among the CTAs, so
// a long context is shared by many and short ones are taken in turn.  The parts
// of an item that lie in several CTAs are joined, in the order of their
// positions, by the CTA that finishes last.

struct AttendRow {
  int first, n, kv;     // its packed tokens, and what is cached with them
};

__device__ __forceinline__ AttendRow attend_row(const AttendArgs& A, int r) {
  AttendRow R;
  R.first = __ldg(A.C.cu + r);
  R.n = __ldg(A.C.cu + r + 1) - R.first;
  R.kv = paged_kv_len(A.C, r);
  if (R.first < 0 || R.n < 0 || R.n > A.N - R.first) R.n = 0;
  return R;
}

// a / group, for a >= 0.  (The compiler's division is several times as long, and a
// kernel of several roles is short of instruction cache.)
__device__ __forceinline__ int attend_token(const AttendArgs& A, int a) {
  int q = (int)((float)a * A.inv_group), r = a - q * A.group;
  const int more = (int)((float)r * A.inv_group);      // what the first product's rounding left
  q += more;
  r -= more * A.group;
  return q + (r >= A.group) - (r < 0);
}

// How many positions the row's i-th new token sees; none that the page table cannot hold.
__device__ __forceinline__ int attend_sees(const AttendArgs& A, const AttendRow& R, int i) {
  return max(0, min(R.kv - R.n + i + 1, A.C.max_pages * A.C.page_size));
}

template <int M, int KT>
__device__ __forceinline__ int attend_tiles(const AttendArgs& A, const AttendRow& R, int qt) {
  const int last = min((qt + 1) * M, R.n * A.group) - 1;
  return max(1, (attend_sees(A, R, attend_token(A, last)) + KT - 1) / KT);
}

template <int M>
__device__ __forceinline__ int attend_qtiles(const AttendArgs& A, const AttendRow& R) {
  return (R.n * A.group + M - 1) / M;
}

// The tiles of one head of a row.
template <int M, int KT>
__device__ __forceinline__ long long attend_head_tiles(const AttendArgs& A, int r) {
  const AttendRow R = attend_row(A, r);
  const int qts = attend_qtiles<M>(A, R);
  long long sum = 0;
#pragma unroll 4
  for (int q = 0; q < qts; ++q) sum += attend_tiles<M, KT>(A, R, q);
  return sum;
}

// A CTA's share: tiles [begin, end) of all, of which the first is tile `a` of the
// item (row, head, qt).  Share c begins where an even division would have it begin,
// bound(c), unless that lies inside an item of at most WHOLE tiles or within
// `slack` tiles of the end of a longer one: then at the nearer end of the item,
// since writing and joining the parts of an item takes as long as some tiles.  (A
// share may be empty then.)  With WHOLE = 6 in the wide kernel, whose end of an
// item is the longer one, 5x484 tokens over short contexts take 25.5 us and not 37,
// ragged chunks 138 us and not 148; the few-rows kernel lost 2 % of its long
// contexts by it and has WHOLE = 0.
struct AttendShare {
  int begin, end, row, head, qt, tiles, a;
  int each, more, slack;             // every share has `each` tiles, the first `more` one more
};

// The last share whose bound is not behind a tile.
__device__ __forceinline__ int share_of(const AttendShare& S, int tile) {
  const int high = S.more * (S.each + 1);
  return tile < high ? tile / (S.each + 1) : S.more + (tile - high) / S.each;
}

template <int M, int KT, int THREADS, int WHOLE>
__device__ __forceinline__ void attend_share(const AttendArgs& A, AttendShare* out, long long* sums) {
  const int t = threadIdx.x, each = (A.C.B + THREADS - 1) / THREADS, r0 = min(t * each, A.C.B), r1 = min(r0 + each, A.C.B);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    mine += attend_head_tiles<M, KT>(A, r) * A.C.heads;
    // (no tile is counted, and so nothing looked up, for positions beyond the page table: they have no page)
    const AttendRow R = attend_row(A, r);
    if (R.n > 0 && R.kv > A.C.max_pages * A.C.page_size && blockIdx.x == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
  }
  sums[t] = mine;
  __syncthreads();
  const int used = min(A.C.B, THREADS);
  long long before = 0, all = 0;
#pragma unroll 8
  for (int i = 0; i < used; ++i) {
    const long long s = sums[i];
    before += i < t ? s : 0;
    all += s;
  }
  // (more than 2^31 tiles, tens of terabytes to read, are refused)
  const int total = all > 0x7fffffff ? 0 : (int)all;
  if (all > 0x7fffffff && A.flags && t == 0 && blockIdx.x == 0) atomicOr(&A.flags[0], (uint32_t)SPEC_F_BAD_IDX);
  const int ctas = min((int)gridDim.x, total), cta = min((int)blockIdx.x, ctas);
  const int tiles_each = ctas ? total / ctas : 0, more = total - tiles_each * ctas;
  const int slack = min(WHOLE / 2, tiles_each / 32);      // (1/16 more work for a share that takes in both its ends)
  const int begin = cta * tiles_each + min(cta, more), end = cta < ctas ? begin + tiles_each + (cta < more) : begin;
  if (t == 0) {
    out->each = tiles_each;
    out->more = more;
    out->slack = slack;
    out->begin = begin;
    out->end = end;
  }
  __syncthreads();
#pragma unroll 1
  for (int e = 0; e < (WHOLE ? 2 : 1); ++e) {
    const int x = e ? end : begin;
    if (begin == end || x < before || x >= before + mine) continue;
    int a = x - (int)before, row = r0, per_head;
    for (;; ++row) {
      per_head = (int)attend_head_tiles<M, KT>(A, row);
      if (a < per_head * A.C.heads) break;
      a -= per_head * A.C.heads;
    }
    const AttendRow R = attend_row(A, row);
    const int head = a / per_head;
    a -= head * per_head;
    int qt = 0, tiles;
    for (;; ++qt) {
      tiles = attend_tiles<M, KT>(A, R, qt);
      if (a < tiles) break;
      a -= tiles;
    }
    const int near = tiles <= WHOLE ? tiles : slack;
    const int move = a <= tiles - a ? (a <= near ? -a : 0) : (tiles - a <= near ? tiles - a : 0);
    if (e) {
      out->end = x + move;
    } else {
      out->begin = x + move;
      out->row = row;
      out->head = head;
      out->qt = qt;
      out->tiles = tiles;
      out->a = a + move;
    }
  }
  __syncthreads();
}

// The CTAs that have parts of an item that no CTA has whole: all from *c0 to *c1.
__device__ __forceinline__ void share_parts(const AttendShare& S, int item, int tiles, int* c0, int* c1) {
  *c0 = share_of(S, item + S.slack);
  *c1 = share_of(S, item + tiles - S.slack - 1);
}

// Walks a CTA's share, one segment (a run of position tiles of one item) after
// another.  COUNT: the first item's tiles are counted again and not read from the
// share, which gives the wide kernel the better code (2x2048 tokens 2 % faster) and
// the other the worse (32x5 tokens of group 8, 8 bits, 6 % slower).
template <int M, int KT, bool COUNT>
struct AttendWalk {
  const AttendArgs& A;
  AttendRow R;
  int row, head, qt, tiles;      // the item, and its position tiles
  int a, b;                      // this segment's
  int at, end;                   // the next tile of all, and the share's end
  int next_a;

  __device__ __forceinline__ AttendWalk(const AttendArgs& args, const AttendShare& S)
      : A(args), row(S.row), head(S.head), qt(S.qt), tiles(COUNT ? 0 : S.tiles), a(0), b(0), at(S.begin), end(S.end), next_a(S.a) {
    if (at >= end) return;
    R = attend_row(A, row);
    if (COUNT) tiles = attend_tiles<M, KT>(A, R, qt);
  }
  // The next segment; false at the end of the share.
  __device__ __forceinline__ bool next() {
    if (at >= end) return false;
    if (next_a >= tiles) {
      next_a = 0;
      if (++qt >= attend_qtiles<M>(A, R)) {
        qt = 0;
        if (++head >= A.C.heads) {
          head = 0;
          do R = attend_row(A, ++row); while (R.n == 0);
        }
      }
      tiles = attend_tiles<M, KT>(A, R, qt);
    }
    a = next_a;
    b = min(tiles, a + (end - at));
    at += b - a;
    next_a = b;
    return true;
  }
  __device__ __forceinline__ bool whole() const { return a == 0 && b == tiles; }
  // The first tile of this item among all.
  __device__ __forceinline__ int item_begin() const { return at - b; }
};

// ---------------------------------------------------------------------- copies

// The positions of the j-th 32 of a tile at which boxes of `box` rows begin.
__device__ __forceinline__ unsigned attend_starts(int box, int j) {
  if (box >= 32) return j * 32 % box == 0 ? 1u : 0u;
  return box == 16 ? 0x10001u : box == 8 ? 0x01010101u : box == 4 ? 0x11111111u : box == 2 ? 0x55555555u : ~0u;
}

// A tensor map of one pool: [pages, heads, page_size, head_dim], boxes of up to
// 128 bytes by `box` rows, in the order they have or swizzled as their width asks.
int attend_map(CUtensorMap* map, void* pool, const PagedCache& C, bool e4m3, int box, bool swizzled);

// The launches.  `maps`: keys, values.
int launch_attend_rows(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st);
int launch_attend_wide(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st);

}  // namespace specv
