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

// What positions a launch is about: all that a query sees; those that the rows of a group have in common, for all of
// their tokens together; or a row's others.
enum : int { kAll = 0, kCommon = 1, kOwn = 2 };
constexpr int kCommonTile = 128;     // what is taken as common ends with a tile of either kernel

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
  // kCommon: the rows of the cache's view are groups, whose tokens and lengths cu and kv_len have; group g are the
  // batch's rows group_row[g] .. group_row[g + 1] - 1, and the first one's page table is read
  const int32_t* group_row;
  const int32_t* own_from;   // kOwn: the first position of each row that is not common (a multiple of kCommonTile)
  // The results over the common positions by (token, head), each divided by its sum of weights and with the logarithm to
  // base 2 of that.  An item that several CTAs have parts of is in those until they are joined: common_items tells by
  // (head, query tile), those of all groups side by side, the first and the last of these CTAs, or -1.
  float* common;
  float* common_lse;
  float* common_parts;
  int2* common_items;
  int common_rows;           // query rows of a tile
  long long common_tiles;    // query tiles of a head, all groups'
};

// Where the query tiles of group g, whose tokens begin at `first`, begin among all.  (A group's last tile may be begun
// alone: one more for each group.)
__device__ __forceinline__ long long common_tile(const AttendArgs& A, int g, int first) { return (long long)first * A.group / A.common_rows + g; }


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

template <int PART>
struct AttendRow {
  int first, n, kv;     // its packed tokens, and what is cached with them
  int from;             // kOwn: the first position
};

template <int PART>
__device__ __forceinline__ AttendRow<PART> attend_row(const AttendArgs& A, int r) {
  AttendRow<PART> R;
  R.first = __ldg(A.C.cu + r);
  R.n = __ldg(A.C.cu + r + 1) - R.first;
  R.kv = paged_kv_len(A.C, r);
  if (PART == kOwn) R.from = __ldg(A.own_from + r);
  if (R.first < 0 || R.n < 0 || R.n > A.N - R.first) R.n = 0;
  if (PART == kCommon && R.kv == 0) R.n = 0;       // (nothing in common is no work)
  return R;
}

// The batch's row whose page table is read, and flags of a row or of all rows of a group that have tokens.
template <int PART>
__device__ __forceinline__ int attend_cache_row(const AttendArgs& A, int row) {
  return PART == kCommon ? __ldg(A.group_row + row) : row;
}
template <int PART>
__device__ __forceinline__ void attend_flag(const AttendArgs& A, int row, uint32_t flag) {
  if (!A.flags) return;
  if (PART != kCommon) {
    atomicOr(&A.flags[row], flag);
    return;
  }
  const int r1 = __ldg(A.group_row + row + 1);
  for (int r = __ldg(A.group_row + row); r < r1; ++r)
    if (__ldg(A.own_from + r) > 0) atomicOr(&A.flags[r], flag);
}

// The weights with which a query row's results over its own and over the common positions are joined, each given with the
// logarithm to base 2 of its sum of weights, and the logarithm of both.
struct AttendJoin {
  float own, common, lse;
};
__device__ __forceinline__ AttendJoin attend_join(float own, float common) {
  const float top = fmaxf(own, common), ref = top == -INFINITY ? 0.f : top;
  const float a = exp2_fast(own - ref), b = exp2_fast(common - ref), sum = a + b, by = sum == 0.f ? 0.f : 1.f / sum;
  return {a * by, b * by, sum == 0.f ? -INFINITY : top + log2f(sum)};
}

// The next launch of the stream may begin before this one ends, if it was made so; what it reads of this one's results
// waits for its end.
__device__ __forceinline__ void launch_may_follow() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void launch_before_is_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
template <int PART>
__device__ __forceinline__ int attend_sees(const AttendArgs& A, const AttendRow<PART>& R, int i) {
  if (PART == kCommon) return R.kv;
  return max(0, min(R.kv - R.n + i + 1, A.C.max_pages * A.C.page_size));
}

// An item's beginning and end take as long as some tiles, and a row's own positions may be few: they are divided with so
// many before each item's.  (64x3 tokens of 500 own positions on average take 133 us with 4 to 12 in the few-rows kernel
// and 153 with none, 64x3 of 2000 196 and 235; 6 chunks of up to 500 220 and 226 with 3 in the other.  Common positions,
// which are many, gain nothing.)
template <int M, int PART>
constexpr int attend_cost() { return PART != kOwn ? 0 : M <= 32 ? 6 : 3; }

// (kOwn: those from the first position on)
template <int M, int KT, int PART>
__device__ __forceinline__ int attend_tiles(const AttendArgs& A, const AttendRow<PART>& R, int qt) {
  static_assert(kCommonTile % KT == 0, "common positions end with a tile");
  if (PART == kCommon) return R.kv / KT;
  const int last = min((qt + 1) * M, R.n * A.group) - 1;
  const int tiles = (attend_sees(A, R, attend_token(A, last)) + KT - 1) / KT;
  return max(1, PART == kOwn ? tiles - R.from / KT : tiles) + attend_cost<M, PART>();
}

template <int M, int PART>
__device__ __forceinline__ int attend_qtiles(const AttendArgs& A, const AttendRow<PART>& R) {
  return (R.n * A.group + M - 1) / M;
}

// The tiles of one head of a row.
template <int M, int KT, int PART>
__device__ __forceinline__ long long attend_head_tiles(const AttendArgs& A, int r) {
  const AttendRow<PART> R = attend_row<PART>(A, r);
  const int qts = attend_qtiles<M>(A, R);
  if (PART == kCommon) return (long long)qts * (R.kv / KT);
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

template <int M, int KT, int THREADS, int WHOLE, int PART>
__device__ __forceinline__ void attend_share(const AttendArgs& A, AttendShare* out, long long* sums) {
  const int t = threadIdx.x, each = (A.C.B + THREADS - 1) / THREADS, r0 = min(t * each, A.C.B), r1 = min(r0 + each, A.C.B);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    mine += attend_head_tiles<M, KT, PART>(A, r) * A.C.heads;
    // (no tile is counted, and so nothing looked up, for positions beyond the page table: they have no page)
    const AttendRow<PART> R = attend_row<PART>(A, r);
    if (PART != kCommon && R.n > 0 && R.kv > A.C.max_pages * A.C.page_size && blockIdx.x == 0 && A.flags) atomicOr(&A.flags[r], (uint32_t)SPEC_F_BAD_IDX);
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
  // (1/16 more work for a share that takes in both its ends; and no share ends before an item's first tile)
  const int slack = max(min(WHOLE / 2, tiles_each / 32), attend_cost<M, PART>() ? attend_cost<M, PART>() + 1 : 0);
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
      per_head = (int)attend_head_tiles<M, KT, PART>(A, row);
      if (a < per_head * A.C.heads) break;
      a -= per_head * A.C.heads;
    }
    const AttendRow<PART> R = attend_row<PART>(A, row);
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
template <int M, int KT, bool COUNT, int PART>
struct AttendWalk {
  const AttendArgs& A;
  AttendRow<PART> R;
  int row, head, qt, tiles;      // the item, and its position tiles
  int a, b;                      // this segment's, by position
  int from, to;                  // the same from the item's beginning, its cost first
  int at, end;                   // the next tile of all, and the share's end
  int next_a;

  __device__ __forceinline__ AttendWalk(const AttendArgs& args, const AttendShare& S)
      : A(args), row(S.row), head(S.head), qt(S.qt), tiles(COUNT ? 0 : S.tiles), a(0), b(0), at(S.begin), end(S.end), next_a(S.a) {
    if (at >= end) return;
    R = attend_row<PART>(A, row);
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
          do R = attend_row<PART>(A, ++row); while (R.n == 0);
        }
      }
      tiles = attend_tiles<M, KT>(A, R, qt);
    }
    from = next_a;
    to = min(tiles, from + (end - at));
    at += to - from;
    next_a = to;
    constexpr int cost = attend_cost<M, PART>();
    a = max(from - cost, 0) + first();
    b = max(to - cost, 0) + first();
    return true;
  }
  // The tile of positions that the item begins with.
  __device__ __forceinline__ int first() const { return PART == kOwn ? R.from / KT : 0; }
  __device__ __forceinline__ bool whole() const { return from == 0 && to == tiles; }
  // The first tile of this item among all.
  __device__ __forceinline__ int item_begin() const { return at - to; }
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
template <int PART>
int launch_attend_rows(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st);
template <int PART>
int launch_attend_wide(const AttendArgs& A, bool e4m3, int rows, const CUtensorMap* maps, cudaStream_t st);

// A launch that may begin before the last one of the stream has ended (see launch_may_follow).
template <class Kernel, class... Args>
inline int launch_early(Kernel kernel, unsigned ctas, int threads, int smem, cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(ctas);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = st;
  config.attrs = &early;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...) == cudaSuccess ? SPEC_OK : SPEC_E_CUDA;
}

// Whether items of up to `rows` query rows go to the many-rows kernel, and the query rows and the positions of a kernel's tile.
bool attend_is_wide(bool e4m3, long long rows);
int attend_tile_rows(bool e4m3, long long rows);
constexpr int attend_tile_positions(bool wide, bool e4m3) { return wide || e4m3 ? 128 : 64; }

// Either of them, for items of up to `rows` query rows.
template <int PART>
int attend_launch(AttendArgs& A, bool e4m3, long long rows, cudaStream_t st);

// The arguments of spec_attend, checked and laid out; `done`: there is nothing to do.
int attend_check(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens, const spec_cache_t* cache,
                 uint16_t* out, float* lse, uint32_t* flags, void* workspace, AttendArgs* A, bool* done);

}  // namespace specv
