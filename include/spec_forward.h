/*
 * spec_forward.h - the sequence mixers of the target forward around a verify
 * step: the paged cache of keys and values, the attention of a row's new
 * tokens over it, and the gated linear recurrence whose per-token states
 * spec_commit gathers.
 *
 * Source: inclusionAI/AReno PR #550, "What does this PR do?" Phase 2 (one
 * forward verifies k+1 tokens per row; paged KV; the recurrent layers write
 * one state per fed token into the verify-state buffer).
 *
 * The conventions of spec_verify.h hold: device pointers, asynchronous work
 * on cuda_stream, arguments checked before anything is enqueued, status codes,
 * and per-row flag bits for what only the device can see.  Calls may be
 * captured into a CUDA graph.  Included by spec_verify.h.
 */
#ifndef SPEC_FORWARD_H
#define SPEC_FORWARD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of an 8-bit cache, beside SPEC_F32 and SPEC_BF16: OCP e4m3
 * codes under one exponent byte a (token, head). */
#define SPEC_E4M3 2

/* Limits: of the paged cache, and of a row's positions or tokens. */
#define SPEC_MAX_PAGE 4096
#define SPEC_MAX_GROUP 64
#define SPEC_MAX_LENGTH 0x7fffff00

/* A batch's view of a paged cache (a host struct of device pointers).
 *
 * Row r's new tokens are tokens cu_tokens[r] .. cu_tokens[r+1]-1 of the packed
 * arrays [N, ...] that a call takes beside this struct.  kv_len[r] counts the
 * row's cached tokens including its new ones, so with n = cu_tokens[r+1] -
 * cu_tokens[r] its i-th new token has position kv_len[r] - n + i.  Position p
 * is held in page page_table[r, p / page_size], slot p % page_size.
 *   k_pages, v_pages [pages, heads, page_size, head_dim] of dtype (SPEC_BF16
 *     or SPEC_E4M3); page_stride elements from one page to the next (0:
 *     dense), so that layers or keys and values may be interleaved in a pool.
 *   k_exp, v_exp     [pages, heads, page_size] exponent bytes of an SPEC_E4M3
 *     cache (NULL for SPEC_BF16), exp_stride bytes from page to page (0:
 *     dense).  Code c under byte e stands for c * 2^(e - 127); byte 0, which is
 *     never written, is read as 1, and byte 255 stands for a vector of NaN.
 *     Codes 0x7f and 0xff are never written.
 *   page_table [B, max_pages] int32.  Only the entries of positions below
 *     kv_len[r] are read; one outside [0, pages) sets SPEC_F_BAD_IDX.
 *   cu_tokens [B + 1] int32 not decreasing from 0 to at most N; kv_len [B].
 * head_dim is 64 or 128; page_size any number up to SPEC_MAX_PAGE, and
 * max_pages * page_size at most SPEC_MAX_LENGTH. */
typedef struct {
  void* k_pages;
  void* v_pages;
  uint8_t* k_exp;
  uint8_t* v_exp;
  const int32_t* page_table;
  const int32_t* cu_tokens;
  const int32_t* kv_len;
  int64_t page_stride;
  int64_t exp_stride;
  int32_t dtype;
  int32_t B;
  int32_t max_pages;
  int32_t pages;
  int32_t heads;
  int32_t page_size;
  int32_t head_dim;
} spec_cache_t;

/* spec_cache_write - put N new tokens' keys and values into the cache.
 *   k, v  [N, heads, head_dim] of dtype SPEC_F32 or SPEC_BF16, token_stride
 *         elements from token to token (0: dense), each token's heads dense.
 * A 16-bit cache holds the values rounded to bf16.  An 8-bit cache: with s the
 * smallest integer in [-126, 127] for which max|x| <= 448 * 2^s over a head's
 * vector, the codes are x * 2^-s (exact) rounded to e4m3, ties to even, and
 * the byte is s + 127.  A vector with an infinity or a NaN gets byte 255 and
 * zero codes, and its row SPEC_F_NAN.
 *   flags [B] uint32 or NULL, OR-ed: SPEC_F_NAN (a 16-bit cache too, whose
 *         values are kept as they are); SPEC_F_BAD_IDX for a token whose
 *         position is negative or has no valid page (it is skipped).
 * Two tokens of one position race.
 * Errors: SPEC_E_NULL, SPEC_E_DIM, SPEC_E_DTYPE, SPEC_E_ALIGN (k, v, the pools
 * and their strides in multiples of 16 bytes), SPEC_E_ARCH, SPEC_E_CUDA. */
int spec_cache_write(const void* k, const void* v, int dtype, int64_t token_stride, int N,
                     const spec_cache_t* cache, uint32_t* flags, void* cuda_stream);

/* spec_cache_read - the inverse: token i's cached key and value to k[i], v[i]
 * ([N, heads, head_dim] bf16, dense).  To read whole rows pass cu_tokens over
 * kv_len[r] tokens a row.  A token without a valid page reads as zeros and sets
 * SPEC_F_BAD_IDX; a vector under byte 255 reads as NaN.  The values of an 8-bit
 * cache are exact in bf16 (below 2^-126 rounded). */
int spec_cache_read(uint16_t* k, uint16_t* v, int N, const spec_cache_t* cache, uint32_t* flags,
                    void* cuda_stream);

/* Bytes of workspace spec_attend needs for a cache of `heads` heads of
 * head_dim, each read by `group` query heads; 0 when one is out of range.
 * Zero-filled before first use, left reusable by every call; it serves calls
 * of any B, N and lengths on one stream. */
size_t spec_attend_workspace_size(int heads, int group, int head_dim);

/* spec_attend - attention of each row's new tokens over its cache (which
 * already holds them), causal by position:
 *   s_j = scale * q_i . k_j for every position j <= p_i of the row,
 *   out_i = sum_j softmax(s)_j v_j,   lse_i = ln sum_j exp(s_j).
 * Query head h reads cache head h / group.
 *   q    [N, heads * group, head_dim] bf16, token_stride elements a token.
 *   out  [N, heads * group, head_dim] bf16, dense;  lse [N, heads * group]
 *        float32 or NULL.  A token that sees no position (a negative one) gets
 *        zeros and -inf.
 *   max_tokens  the largest number of new tokens of a row, as the host knows
 *        it: it chooses between kernels and is not a limit.
 *   flags [B] uint32 or NULL, OR-ed: SPEC_F_BAD_IDX where a visible position
 *        has no valid page; such positions are left out.  SPEC_F_TIMEOUT where a
 *        wait passed its bound (the row is not to be relied on).  A call of 2^31 and more
 *        tiles of positions writes nothing and sets SPEC_F_BAD_IDX of row 0.
 * Tokens of the packed arrays that belong to no row are not written.
 * What a query does not see never reaches it, infinities and NaN included.
 * Values of an 8-bit cache under exponent bytes above 221 (2^103 and more) are
 * taken for NaN.
 * Scores, their maximum and sum and the output sums are float32.  For the
 * product with the values softmax weights are rounded to bf16, or, with few
 * rows over an 8-bit cache, to fp16 together with the values' scales, where a
 * term of a row 2^-25 below its largest is lost.  One call's results do not
 * depend on timing.
 * Errors: as spec_cache_write, and SPEC_E_WORKSPACE. */
int spec_attend(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens,
                const spec_cache_t* cache, uint16_t* out, float* lse, uint32_t* flags, void* workspace,
                size_t workspace_bytes, void* cuda_stream);

/* Bytes of workspace spec_recur and spec_recur_backward need for B rows of T
 * tokens over D channels (0 when a size is out of range); zero-filled before
 * first use, left reusable by every call.  A workspace serves any shape it is
 * large enough for, on one stream. */
size_t spec_recur_workspace_size(int B, int T, int D);

/* spec_recur - gated linear recurrence, channel by channel:
 *   h_t = exp(g_t) h_{t-1} + x_t,   t = 0 .. len_r - 1.
 * B is at most 65535, T SPEC_MAX_LENGTH, D 2^26.
 *   g, x   [B, T, D] of dtype (SPEC_F32 or SPEC_BF16), channels dense, with
 *          g_row / g_tok (x_row / x_tok) elements from row to row and token to
 *          token (0: the same for all).  g is the logarithm of the decay, at
 *          most 0: above it products of decays may overflow before the state
 *          does.  -inf forgets a finite state.
 *   state  [slots, D] float32 or NULL: h_{-1} of row r is state[slot[r]]
 *          (state[r] where slot is NULL); NULL: zeros.
 *   lens   [B] int32 or NULL (T each): len_r, clamped to [0, T].  g and x
 *          beyond it are not read and h there is zero.
 *   h      [B, T, D] of h_dtype, dense.  In SPEC_F32 it is one layer of
 *          spec_commit's verify_rec with H = Dk = 1, Dv = D.
 *   last   [*, D] float32 or NULL: receives h after the row's last token (its
 *          initial state where len_r is 0) at last_slot[r] (at r where
 *          last_slot is NULL).  It may be `state` with last_slot = slot: a
 *          decode step in place.  last_slots: rows of `last`.
 *   flags  [B] or NULL: SPEC_F_BAD_IDX for a row whose slot or last_slot is out
 *          of range (h is zero, last is left alone); SPEC_F_TIMEOUT for a row
 *          where a wait passed its bound (its h is not to be relied on).
 * The state is float32 throughout.
 * Errors: SPEC_E_NULL, SPEC_E_DIM, SPEC_E_DTYPE, SPEC_E_ALIGN,
 * SPEC_E_WORKSPACE, SPEC_E_ARCH, SPEC_E_CUDA. */
int spec_recur(const void* g, int64_t g_row, int64_t g_tok, const void* x, int64_t x_row, int64_t x_tok,
               int dtype, const float* state, const int32_t* slot, int slots, const int32_t* lens, int B,
               int T, int D, void* h, int h_dtype, float* last, const int32_t* last_slot, int last_slots,
               uint32_t* flags, void* workspace, size_t workspace_bytes, void* cuda_stream);

/* spec_recur_backward - its gradients.  With dh the gradient of h and d_last
 * that of the last state (NULL: zero), from the last token to the first:
 *   l_t = dh_t + exp(g_{t+1}) l_{t+1}   (d_last in the place of the product
 *                                        behind the last token),
 *   dx_t = l_t,   dg_t = exp(g_t) l_t h_{t-1},   d_state = exp(g_0) l_0.
 *   g, dh, dg, dx [B, T, D] of dtype (g strided as above, the others dense);
 *   h [B, T, D] of h_dtype as spec_recur wrote it; state, slot, lens as given
 *   to spec_recur; d_last, d_state [B, D] float32, by row, or NULL (d_state may
 *   be d_last).
 * dg and dx are zero beyond len_r; a row of length 0 has d_state = d_last.
 * dg carries the rounding of h: where float32 gates need more than bf16's 8
 * bits, h is kept in SPEC_F32. */
int spec_recur_backward(const void* g, int64_t g_row, int64_t g_tok, const void* h, int h_dtype,
                        const void* dh, const float* d_last, int dtype, const float* state,
                        const int32_t* slot, int slots, const int32_t* lens, int B, int T, int D, void* dg,
                        void* dx, float* d_state, uint32_t* flags, void* workspace, size_t workspace_bytes,
                        void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_FORWARD_H */
