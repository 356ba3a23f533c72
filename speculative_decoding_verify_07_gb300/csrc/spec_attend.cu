// spec_attend: argument checks, tensor maps and the choice between kernels.
#include "spec_attend.cuh"

namespace specv {

TensorMapEncode tensor_map_encoder() {
  static TensorMapEncode fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<TensorMapEncode>(p);
  }();
  return fn;
}

int attend_map(CUtensorMap* map, void* pool, const PagedCache& C, bool e4m3, int box, bool swizzled) {
  const TensorMapEncode encode = tensor_map_encoder();
  if (!encode) return SPEC_E_CUDA;
  const cuuint64_t es = e4m3 ? 1 : 2, row = C.D * es;
  const cuuint64_t dims[4] = {(cuuint64_t)C.D, (cuuint64_t)C.page_size, (cuuint64_t)C.heads, (cuuint64_t)C.pages};
  const cuuint64_t strides[3] = {row, row * C.page_size, (cuuint64_t)C.page_bytes};
  const cuuint32_t width = (cuuint32_t)(row > 128 ? 128 : row);
  const cuuint32_t boxes[4] = {(cuuint32_t)(width / es), (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
  return encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, boxes,
                ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SPEC_OK
             : SPEC_E_CUDA;
}

// Partial results of the launch with the most: 152 CTAs of two parts of 256 rows.
static size_t attend_parts(int D) { return (size_t)152 * 2 * 256 * (D + 2) * sizeof(float); }

}  // namespace specv

extern "C" size_t spec_attend_workspace_size(int heads, int group, int head_dim) {
  if (heads < 1 || heads > 65535 || group < 1 || group > SPEC_MAX_GROUP || (head_dim != 64 && head_dim != 128)) return 0;
  return specv::kAttendCounters + specv::attend_parts(head_dim);
}

extern "C" int spec_attend(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens,
                           const spec_cache_t* cache, uint16_t* out, float* lse, uint32_t* flags, void* workspace,
                           size_t workspace_bytes, void* cuda_stream) {
  using namespace specv;
  AttendArgs A;
  const int rc = paged_check(cache, N, &A.C);
  if (rc != SPEC_OK) return rc;
  if (group < 1 || group > SPEC_MAX_GROUP || max_tokens < 0 || token_stride < 0) return SPEC_E_DIM;
  A.hq = A.C.heads * group;
  const long long dense = (long long)A.hq * A.C.D;
  if (A.hq > 65535 || (token_stride && token_stride < dense)) return SPEC_E_DIM;
  if (N == 0 || A.C.B == 0) return SPEC_OK;
  if (!q || !out || !workspace) return SPEC_E_NULL;
  A.q_token = token_stride ? token_stride : dense;
  if (!paged_aligned(q, 16) || !paged_aligned(out, 16) || A.q_token % 8 || (lse && !paged_aligned(lse, 4)) ||
      (flags && !paged_aligned(flags, 4)) || !paged_aligned(workspace, 256))
    return SPEC_E_ALIGN;
  if (workspace_bytes < spec_attend_workspace_size(A.C.heads, group, A.C.D)) return SPEC_E_WORKSPACE;
  const int arc = check_arch();
  if (arc != SPEC_OK) return arc;
  A.q = q;
  A.out = out;
  A.lse = lse;
  A.flags = flags;
  A.N = N;
  A.group = group;
  A.inv_group = 1.f / group;
  A.scale_log2 = scale * 1.4426950408889634f;
  A.joined = static_cast<unsigned*>(workspace);
  A.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kAttendCounters);
  const bool e4m3 = cache->dtype == SPEC_E4M3;
  // A tile of 16 or 32 query rows at a time, or of 128 or 256.  The few-rows kernel reads the cache again for every
  // 32 rows, the other fills its tile with padding.  In 16 bits 32x5 tokens of group 8 (40 rows) at 8000 take 139 us with
  // many rows, with few 231.  In 8 bits, where the other kernel widens the codes first, neither wins throughout from 33
  // to 64 rows: few rows take 89 us and many 123 with one row of 9 tokens (group 4, one head) at 60000, 47.5 and 58 with
  // 67 ragged ones over 800, 351 and 407 with 32x5 at 8000 in pages of one token; but 220 and 173 with these in pages
  // of 16, and 305 and 206 with 64x8 at 4000.  Up to 32 rows few do (64x4 of group 8 239 us, 328).
  const long long rows = (long long)max_tokens * group;
  const bool wide = rows > (e4m3 ? 64 : 32);
  // the longest run of positions that never leaves a page, up to what is copied at a time
  const int most = wide ? 128 : e4m3 ? 32 : 16;
  A.box = 1;
  while (A.box < most && A.C.page_size % (2 * A.box) == 0) A.box *= 2;
  CUtensorMap maps[2];
  if (A.C.pages > 0) {
    for (int i = 0; i < 2; ++i)
      if (attend_map(&maps[i], i ? A.C.v : A.C.k, A.C, e4m3, A.box, !(wide && e4m3)) != SPEC_OK) return SPEC_E_CUDA;
  }
  const int most_rows = rows > 0x7fffffff ? 0x7fffffff : (int)rows;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
  return wide ? launch_attend_wide(A, e4m3, most_rows, maps, st) : launch_attend_rows(A, e4m3, most_rows, maps, st);
}
