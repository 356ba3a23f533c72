/*
 * spec_hybrid.h - the further mixers of a hybrid target's forward around a
 * verify step: the short causal convolution and the selective scan of its
 * state space layers, whose per-token states spec_commit gathers, and the
 * attention of several samples of one prompt, which reads the cache of what
 * they have in common once for all of them.
 *
 * Source: inclusionAI/AReno PR #550, "What does this PR do?" Phase 2 (the verify
 * writes a recurrent and a convolution state per fed token) and the group
 * rollouts that it decodes (n samples of a prompt).
 *
 * The conventions of spec_verify.h and spec_forward.h hold: device pointers,
 * asynchronous work on cuda_stream, arguments checked before anything is
 * enqueued, status codes, and per-row flag bits for what only the device can
 * see.  Calls may be captured into a CUDA graph.  Included by spec_verify.h.
 */
#ifndef SPEC_HYBRID_H
#define SPEC_HYBRID_H

#include <stddef.h>
#include <stdint.h>

#include "spec_forward.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_MAX_CONV 8         /* taps of the convolution, two at least */

/* One layer's short causal convolution (a host struct of device pointers).
 *   x        [B, T, C] of dtype (SPEC_F32 or SPEC_BF16), channels dense, x_row /
 *            x_tok elements from row to row and token to token.
 *   weight   [width, C] float32: tap i is that of x_{t - width + 1 + i}.
 *   bias     [C] float32 or NULL.
 *   state    [slots, width - 1, C] of dtype or NULL: the inputs before row r's first
 *            token, the oldest first, are state[slot[r]] (state[r] where slot is
 *            NULL); NULL: zeros.
 *   lens     [B] int32 or NULL (T each): the row's tokens, clamped to [0, T].  x
 *            beyond them is not read; y and states there are zero.
 *   y        [B, T, C] of dtype, dense.
 *   states   [B, T, width - 1, C] of dtype or NULL: the state behind each token.  In
 *            SPEC_BF16 it is one layer of spec_commit's verify_conv with
 *            W = width - 1.
 *   last     [last_slots, width - 1, C] of dtype or NULL: receives the state behind the
 *            row's last token (its initial state where there is none) at
 *            last_slot[r] (at r where last_slot is NULL).  It may be `state` with
 *            last_slot = slot: a decode step in place.  Two rows of one slot race.
 *   flags    [B] uint32 or NULL, OR-ed: SPEC_F_BAD_IDX for a row whose slot or
 *            last_slot is out of range (y and states are zero, last is left alone).
 *   silu     nonzero: y is v / (1 + exp(-v)) of the sum v, otherwise the sum.
 * Outputs overlap no input, but for `last`. */
typedef struct {
  const void* x;
  const float* weight;
  const float* bias;
  const void* state;
  const int32_t* slot;
  const int32_t* lens;
  void* y;
  void* states;
  void* last;
  const int32_t* last_slot;
  uint32_t* flags;
  int64_t x_row;
  int64_t x_tok;
  int32_t dtype;
  int32_t B;
  int32_t T;
  int32_t C;
  int32_t width;
  int32_t slots;
  int32_t last_slots;
  int32_t silu;
} spec_conv_t;

/* spec_conv - y_t[c] = act(bias[c] + sum_i weight[i, c] x_{t - width + 1 + i}[c]),
 * summed in float32.  B is at most 65535, T SPEC_MAX_LENGTH, C 2^26.
 * Errors: SPEC_E_NULL, SPEC_E_DIM, SPEC_E_DTYPE, SPEC_E_ALIGN (each array to its
 * element), SPEC_E_ARCH, SPEC_E_CUDA. */
int spec_conv(const spec_conv_t* conv, void* cuda_stream);

/* One layer's selective scan (a host struct of device pointers).
 *   x, dt, z [B, T, D] of dtype (SPEC_F32 or SPEC_BF16), channels dense, with elements
 *            from row to row and token to token of their own; z may be NULL.
 *   b, c     [B, T, groups, N] of dtype, states dense, with strides of row, token and
 *            group.  Channel d reads group d / (D / groups).
 *   a        [D, N] float32, at most 0: decays are exp(delta a).  With a above zero or
 *            delta below it, products of decays may overflow before the state does.
 *            -inf forgets a finite state (but for a step of 0).
 *   skip, dt_bias  [D] float32 or NULL (zeros).
 *   state    [slots, D, N] float32 or NULL, slot, lens, flags: as in spec_conv_t.
 *   y        [B, T, D] of dtype, dense.
 *   states   [B, T, D, N] float32 or NULL: the state behind each token, one layer
 *            of spec_commit's verify_rec with H = 1, Dk = D, Dv = N.
 *   last     [last_slots, D, N] float32 or NULL, last_slot: as in spec_conv_t.
 *   softplus nonzero: delta = ln(1 + exp(dt + dt_bias)), and 0 where that is below
 *            2^-126 (dt + dt_bias < -87.3, -inf too); otherwise dt + dt_bias.
 * Outputs overlap no input, but for `last`. */
typedef struct {
  const void* x;
  const void* dt;
  const void* z;
  const void* b;
  const void* c;
  const float* a;
  const float* skip;
  const float* dt_bias;
  const float* state;
  const int32_t* slot;
  const int32_t* lens;
  void* y;
  float* states;
  float* last;
  const int32_t* last_slot;
  uint32_t* flags;
  int64_t x_row;
  int64_t x_tok;
  int64_t dt_row;
  int64_t dt_tok;
  int64_t z_row;
  int64_t z_tok;
  int64_t b_row;
  int64_t b_tok;
  int64_t b_group;
  int64_t c_row;
  int64_t c_tok;
  int64_t c_group;
  int32_t dtype;
  int32_t B;
  int32_t T;
  int32_t D;
  int32_t N;
  int32_t groups;
  int32_t slots;
  int32_t last_slots;
  int32_t softplus;
} spec_scan_t;

/* Bytes of workspace spec_scan needs for up to B rows of up to T tokens over D
 * channels of N states (256 at least; 0 when a size is out of range).  Its contents
 * need not be kept or cleared; calls that may overlap take one each. */
size_t spec_scan_workspace_size(int B, int T, int D, int N);

/* spec_scan - the selective scan, for channel d and state n:
 *   h_t[d, n] = exp(delta_t[d] a[d, n]) h_{t-1}[d, n] + delta_t[d] x_t[d] b_t[n],
 *   y_t[d] = (sum_n c_t[n] h_t[d, n] + skip[d] x_t[d]) * (z_t[d] / (1 + exp(-z_t[d]))),
 * the last factor only with z.  A token of delta 0 leaves the state.  N is 8, 16, 32,
 * 64 or 128; B at most 65535, T SPEC_MAX_LENGTH, D 2^24 and a multiple of
 * groups.  States and sums are float32.  A state that has become infinite stays so
 * while the decays of single tokens are 2^-126 and more (below, it may be NaN).
 * state, states, last and a are aligned to 16 bytes, the others to their elements.
 * Errors: SPEC_E_NULL, SPEC_E_DIM, SPEC_E_DTYPE, SPEC_E_ALIGN, SPEC_E_WORKSPACE,
 * SPEC_E_ARCH, SPEC_E_CUDA. */
int spec_scan(const spec_scan_t* scan, void* workspace, size_t workspace_bytes, void* cuda_stream);

/* Bytes of workspace spec_attend_shared needs for up to N new tokens in up to B rows
 * over a cache of `heads` heads of head_dim, each read by `group` query heads; 0 when
 * one is out of range.  Zero-filled before first use, left reusable by every
 * call, for one stream. */
size_t spec_attend_shared_workspace_size(int N, int B, int heads, int group, int head_dim);

/* spec_attend_shared - spec_attend for rows that have their first positions in
 * common, as samples of one prompt have: the same definition, within the same
 * roundings, but what is shared is read once for all of a group's rows.
 *   shared_rows  [groups + 1] int32, not decreasing, within [0, B]: group g are rows
 *                shared_rows[g] .. shared_rows[g+1]-1.  Rows of no group, and all
 *                rows where shared_rows is out of order, share nothing.
 *   shared_len   [groups] int32: the positions that the rows of a group have in
 *                common.  They are read through the page table of the group's first
 *                row; the others' entries of whole tiles of 128 shared positions are
 *                not read.  Where a row's own new tokens begin before shared_len, only
 *                what lies before all of the group's new tokens counts as shared.
 * groups is at most B.  All else is as in spec_attend; out, lse and flags too.
 * What it saves is reads of the cache.  It is the faster call where a group's rows
 * behind the first would read some 65,000 shared positions or more together (of 8
 * heads of 128 in 16 bits): 64 rows behind 1000 positions, 8 behind 12,000.  Below,
 * and for rows of hundreds of new tokens, whose products are what takes time,
 * spec_attend is, with each row's own page table. */
int spec_attend_shared(const uint16_t* q, int64_t token_stride, int N, int group, float scale, int max_tokens,
                       const spec_cache_t* cache, const int32_t* shared_rows, const int32_t* shared_len,
                       int groups, uint16_t* out, float* lse, uint32_t* flags, void* workspace,
                       size_t workspace_bytes, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_HYBRID_H */
