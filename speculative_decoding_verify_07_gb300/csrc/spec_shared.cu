// spec_attend_shared: the attention of rows that have their first positions in common.
//
// What the rows of a group share is one cache for all their tokens: where n rows of T
// tokens read the prompt, n T group query rows a head stand against it, which is a
// product for the tensor cores over bytes that are read once, and not n reads of
// them.  So there are two attentions: of each group's tokens over the common positions
// (no mask: every token is behind all of them), and of each row's tokens over its own,
// causal.  Both are the kernels of spec_attend, which divide their work evenly over the
// device whatever the lengths.  The first leaves its results, divided by their sums,
// and the logarithms of the sums in float32 in the workspace, a long item in the parts
// that its CTAs have, which a launch of its own joins (where one CTA joined an item's
// parts, 8 items of 16,000 positions took as long as 24).  The second, which may begin
// while these end, adds them in as it writes the results.
//
// Measured, 8 heads of 128, group 4, bf16: 64 rows of 3 tokens behind 16,000 common positions
// and up to 1000 of their own 133 us (spec_attend 503): 72 for the common positions (24 items for
// 152 CTAs, each at its beginning and end more than half the time), 5 to 10 to join them, 45 for
// the own ones.  16 groups of 8 rows, 6001 common positions, 8 bits 141 us; 6 chunks of up to 500
// tokens behind 12,345 218 us.
// What is saved is reads, so it pays where the rows behind the first of their groups would
// read some 65,000 common positions or more together, of 8 heads of 128.  In a graph, beside
// spec_attend on the same rows: 64x3 behind 512, 1024 and 2048 positions 53, 53 and 64 us and
// 41, 54 and 83; 8x3 behind 8192 and 16,384 53 and 62 us and 47 and 78; 16 groups of 8, 8 bits,
// behind 512 and 1024 60 and 72 us and 60 and 80; two rows behind 32,768 (heads of 64) still 43
// and 36.  Chunks of prompts are bound by their products, which are the same: 4 of up to
// 500 tokens behind 16,384 185 us and 144.
//
// Common positions end with a multiple of 128, the larger tile of the kernels, so that
// neither has a tile of both kinds; the up to 127 that are left go to each row.
#include <algorithm>

#include "spec_attend.cuh"

namespace specv {

constexpr int kGroupThreads = 1024;

// Finds what each group has in common: shared_len, but nothing behind the first new token of any of its rows or
// beyond the page table, in whole tiles, and nothing for a single row.  A warp a group.  Where that would be more tiles, of
// 2^tile_rows query rows by 2^tile_positions, than the attention over it takes, nothing is in common: the rows' own attention,
// of no fewer, then answers for the call, or refuses it.
static __global__ void __launch_bounds__(kGroupThreads) attend_groups_kernel(const PagedCache C, int N, const int32_t* shared_rows, const int32_t* shared_len,
                                                                      int groups, int group, int tile_rows, int tile_positions, int32_t* group_row,
                                                                      int32_t* group_cu, int32_t* group_len, int32_t* own_from) {
  __shared__ unsigned long long tiles;       // of a head
  if (threadIdx.x == 0) tiles = 0;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  bool ok = true;
  for (int g = threadIdx.x; g < groups; g += kGroupThreads) {
    const int a = __ldg(shared_rows + g), b = __ldg(shared_rows + g + 1);
    ok = ok && a >= 0 && a <= b && b <= C.B;
  }
  ok = __syncthreads_and(ok);
  const int first = ok ? __ldg(shared_rows) : 0, last = ok ? __ldg(shared_rows + groups) : 0;
  for (int r = threadIdx.x; r < C.B; r += kGroupThreads)
    if (r < first || r >= last) own_from[r] = 0;
  for (int g = warp; g < groups; g += kGroupThreads / 32) {
    const int a = ok ? __ldg(shared_rows + g) : 0, b = ok ? __ldg(shared_rows + g + 1) : 0;
    const int t0 = __ldg(C.cu + a), t1 = __ldg(C.cu + b);
    int least = t0 < 0 || t1 > N ? 0 : 0x7fffffff, busy = 0;     // (a row's tokens are among the group's, which are there)
    for (int r = a + lane; r < b; r += 32) {
      const int c0 = __ldg(C.cu + r), c1 = __ldg(C.cu + r + 1);
      if (c0 < t0 || c1 > t1) least = 0;
      if (c0 < c1 && least > 0) {
        least = min(least, paged_kv_len(C, r) - (c1 - c0));
        ++busy;
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    busy = __reduce_add_sync(0xffffffffu, busy);
    int len = 0;
    if (busy > 1) len = max(0, min(min(least, __ldg(shared_len + g)), C.max_pages * C.page_size)) / kCommonTile * kCommonTile;
    for (int r = a + lane; r < b; r += 32) own_from[r] = __ldg(C.cu + r + 1) > __ldg(C.cu + r) ? len : 0;
    if (lane == 0) {
      if (len > 0) atomicAdd(&tiles, (unsigned long long)((((long long)(t1 - t0) * group - 1) >> tile_rows) + 1) * (len >> tile_positions));
      group_len[g] = len;
      group_row[g] = a;
      group_cu[g] = t0;
      if (g == groups - 1) {
        group_row[groups] = b;
        group_cu[groups] = t1;
      }
    }
  }
  __syncthreads();
  if (tiles * C.heads <= 0x7fffffffull) return;
  for (int g = threadIdx.x; g < groups; g += kGroupThreads) group_len[g] = 0;
  for (int r = threadIdx.x; r < C.B; r += kGroupThreads) own_from[r] = 0;
}

constexpr int kPartsThreads = 256;

// Joins the parts of the items that several CTAs have, in the order of their positions: D / 4 lanes a query row.  (A's
// rows are the groups.)
template <int D>
static __global__ void __launch_bounds__(kPartsThreads) attend_parts_kernel(const AttendArgs A) {
  launch_may_follow();
  launch_before_is_done();
  constexpr int L = D / 4;
  const long long all = (long long)A.N * A.hq;
  const int d = threadIdx.x % L * 4;
  for (long long at = ((long long)blockIdx.x * kPartsThreads + threadIdx.x) / L; at < all; at += (long long)gridDim.x * (kPartsThreads / L)) {
    const int token = (int)(at / A.hq), head = (int)(at - (long long)token * A.hq);
    const int g = paged_row(A.C, token);
    if (g < 0 || __ldg(A.C.kv_len + g) == 0) continue;
    const int first = __ldg(A.C.cu + g), kv_head = head / A.group;
    const long long a = (long long)(token - first) * A.group + (head - kv_head * A.group), qt = a / A.common_rows;
    const int local = (int)(a - qt * A.common_rows);
    const int2 ctas = __ldcg(A.common_items + kv_head * A.common_tiles + common_tile(A, g, first) + qt);
    if (ctas.x < 0) continue;
    const long long size = (long long)A.common_rows * (D + 1);
    auto part = [&](int c) { return A.common_parts + (c * 2 + (c == ctas.x)) * size; };
    float top = -INFINITY;
#pragma unroll 8
    for (int c = ctas.x; c <= ctas.y; ++c) top = fmaxf(top, __ldcg(part(c) + A.common_rows * D + local));
    const float ref = top == -INFINITY ? 0.f : top;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 8
    for (int c = ctas.x; c <= ctas.y; ++c) {
      const float w = exp2_fast(__ldcg(part(c) + A.common_rows * D + local) - ref);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(part(c) + (long long)local * D + d));
      sum += w;
      x.x = fmaf(y.x, w, x.x), x.y = fmaf(y.y, w, x.y), x.z = fmaf(y.z, w, x.z), x.w = fmaf(y.w, w, x.w);
    }
    const float by = sum == 0.f ? 1.f : 1.f / sum;
    __stcg(reinterpret_cast<float4*>(A.common + at * D + d), make_float4(x.x * by, x.y * by, x.z * by, x.w * by));
    if (d == 0) __stcg(A.common_lse + at, sum == 0.f ? -INFINITY : top + log2f(sum));
  }
}

static int log2_of(int power) {
  int n = 0;
  while (power >> (n + 1)) ++n;
  return n;
}

// Workspace, behind that of spec_attend (which serves the rows' own positions): the groups' rows, tokens and lengths, the
// rows' first own positions, then the results over the common positions.
struct SharedSpace {
  size_t group_row, group_cu, group_len, own_from, items, lse, out, parts, bytes;

  SharedSpace(size_t base, int N, int B, int heads, int group, int D) {
    const size_t hq = (size_t)heads * group;
    auto take = [&](size_t n) {
      const size_t at = base;
      base = (base + n + 255) / 256 * 256;
      return at;
    };
    base = (base + 255) / 256 * 256;
    group_row = take(((size_t)B + 1) * 4);
    group_cu = take(((size_t)B + 1) * 4);
    group_len = take((size_t)B * 4);
    own_from = take((size_t)B * 4);
    items = take(heads * ((size_t)N * group / 16 + B + 1) * sizeof(int2));      // (16: the query rows of the smallest tile)
    lse = take((size_t)N * hq * 4);
    out = take((size_t)N * hq * D * 4);
    parts = take((size_t)152 * 2 * 256 * (D + 1) * 4);
    bytes = base;
  }
};

}  // namespace specv

extern "C" size_t spec_attend_shared_workspace_size(int N, int B, int heads, int group, int head_dim) {
  const size_t base = spec_attend_workspace_size(heads, group, head_dim);
  if (base == 0 || N < 0 || B < 0 || (long long)heads * group > 65535) return 0;
  return specv::SharedSpace(base, N, B, heads, group, head_dim).bytes;
}

extern "C" int spec_attend_shared(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens,
                                  const spec_cache_t* cache, const int32_t* shared_rows, const int32_t* shared_len, int groups,
                                  uint16_t* out, float* lse, uint32_t* flags, void* workspace, size_t workspace_bytes,
                                  void* cuda_stream) {
  using namespace specv;
  AttendArgs A;
  bool done;
  const int rc = attend_check(q, token_stride, N, group, scale, max_tokens, cache, out, lse, flags, workspace, &A, &done);
  if (rc != SPEC_OK) return rc;
  if (groups < 0 || groups > A.C.B) return SPEC_E_DIM;
  if (done) return SPEC_OK;
  if (groups > 0 && (!shared_rows || !shared_len)) return SPEC_E_NULL;
  if (!paged_aligned(shared_rows, 4) || !paged_aligned(shared_len, 4)) return SPEC_E_ALIGN;
  if (workspace_bytes < spec_attend_shared_workspace_size(N, A.C.B, A.C.heads, group, A.C.D)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  const long long rows = (long long)max_tokens * group;
  if (groups == 0) return attend_launch<kAll>(A, e4m3, rows, st);
  char* const base = static_cast<char*>(workspace);
  const SharedSpace S(spec_attend_workspace_size(A.C.heads, group, A.C.D), N, A.C.B, A.C.heads, group, A.C.D);
  int32_t* const group_row = reinterpret_cast<int32_t*>(base + S.group_row);
  int32_t* const group_cu = reinterpret_cast<int32_t*>(base + S.group_cu);
  int32_t* const group_len = reinterpret_cast<int32_t*>(base + S.group_len);
  int32_t* const own_from = reinterpret_cast<int32_t*>(base + S.own_from);
  A.group_row = group_row;
  A.own_from = own_from;
  A.common = reinterpret_cast<float*>(base + S.out);
  A.common_lse = reinterpret_cast<float*>(base + S.lse);
  A.common_parts = reinterpret_cast<float*>(base + S.parts);
  A.common_items = reinterpret_cast<int2*>(base + S.items);
  // a group's tokens are not known here: as many as each would have of all
  const long long common_rows = ((long long)N + groups - 1) / groups * group;
  A.common_rows = attend_tile_rows(e4m3, common_rows);
  attend_groups_kernel<<<1, kGroupThreads, 0, st>>>(A.C, N, shared_rows, shared_len, groups, group,
                                                    log2_of(A.common_rows),
                                                    log2_of(attend_tile_positions(attend_is_wide(e4m3, common_rows), e4m3)), group_row,
                                                    group_cu, group_len, own_from);
  if (cudaGetLastError() != cudaSuccess) return SPEC_E_CUDA;
  A.common_tiles = (long long)N * group / A.common_rows + groups + 1;
  AttendArgs common = A;
  common.C.B = groups;
  common.C.cu = group_cu;
  common.C.kv_len = group_len;
  int did = attend_launch<kCommon>(common, e4m3, common_rows, st);
  const long long warps = ((long long)N * A.hq * A.C.D + 127) / 128, ctas = std::min((warps + kPartsThreads / 32 - 1) / (kPartsThreads / 32), 152ll * 16);
  if (did == SPEC_OK)
    did = launch_early(A.C.D == 128 ? attend_parts_kernel<128> : attend_parts_kernel<64>, (unsigned)ctas, kPartsThreads, 0, st, common);
  return did != SPEC_OK ? did : attend_launch<kOwn>(A, e4m3, rows, st);
}
