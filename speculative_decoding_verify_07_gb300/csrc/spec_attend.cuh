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
  R.kv = __ldg(A.C.kv_len + r);
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

// A CTA's share: tiles [begin, end) of all, the first of them at `offset` in row
// `row`.  Each of `ctas` CTAs has `each` tiles, the first `more` one more.
struct AttendShare {
  int begin, end, offset, each, more, row, ctas;
};

__device__ __forceinline__ int share_of(const AttendShare& S, int tile) {
  const int high = S.more * (S.each + 1);
  return tile < high ? tile / (S.each + 1) : S.more + (tile - high) / S.each;
}

template <int M, int KT, int THREADS>
__device__ __forceinline__ void attend_share(const AttendArgs& A, AttendShare* out, long long* sums) {
  const int t = threadIdx.x, each = (A.C.B + THREADS - 1) / THREADS, r0 = min(t * each, A.C.B), r1 = min(r0 + each, A.C.B);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += attend_head_tiles<M, KT>(A, r) * A.C.heads;
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
  const int tiles = ctas ? total / ctas : 0, more = total - tiles * ctas, begin = cta * tiles + min(cta, more);
  if (t == 0) {
    out->ctas = ctas;
    out->each = tiles;
    out->more = more;
    out->begin = begin;
    out->end = cta < ctas ? begin + tiles + (cta < more) : begin;
    out->row = 0;
    out->offset = 0;
  }
  __syncthreads();
  if (total && begin >= before && begin < before + mine) {
    int at = (int)before;
    for (int r = r0; r < r1; ++r) {
      const int w = (int)attend_head_tiles<M, KT>(A, r) * A.C.heads;
      if (begin < at + w) {
        out->row = r;
        out->offset = begin - at;
        break;
      }
      at += w;
    }
  }
  __syncthreads();
}

// Walks a CTA's share, one segment (a run of position tiles of one item) after another.
template <int M, int KT>
struct AttendWalk {
  const AttendArgs& A;
  AttendRow R;
  int row, head, qt, tiles;      // the item, and its position tiles
  int a, b;                      // this segment's
  int at, end;                   // the next tile of all, and the share's end
  int next_a;

  __device__ __forceinline__ AttendWalk(const AttendArgs& args, const AttendShare& S)
      : A(args), row(S.row), head(0), qt(0), tiles(0), a(0), b(0), at(S.begin), end(S.end), next_a(0) {
    if (at >= end) return;
    R = attend_row(A, row);
    int off = S.offset;
    const int per_head = (int)attend_head_tiles<M, KT>(A, row);
    head = off / per_head;
    off -= head * per_head;
    for (;;) {
      tiles = attend_tiles<M, KT>(A, R, qt);
      if (off < tiles) break;
      off -= tiles;
      ++qt;
    }
    next_a = off;
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
