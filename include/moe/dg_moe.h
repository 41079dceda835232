/*
 * dg_moe.h - the steps of a mixture-of-experts block around the grouped GEMMs
 * of dg.h, for AMD Instinct MI355X (gfx950): tokens sorted by expert into the
 * GEMMs' row layouts and back with weights applied, the gated activation
 * between the two GEMMs, the norms before and after the block with its gate
 * and residual scale, and the gradients of all of these. Same library
 * (libdg.so), status codes and conventions as dg.h: every pointer is
 * caller-owned device memory, nothing is allocated, arguments are checked
 * before anything is enqueued, calls enqueue on `stream` (of the current
 * device, where the buffers lie too) and return without synchronising, and
 * all of them are safe to capture in a HIP graph.
 * Activations are BF16, FP8 is OCP E4M3, sums and statistics are float32, and
 * every result is rounded once, to nearest even. Results do not depend on
 * timing: the same inputs give the same bits. The norms and their gradient
 * spread over dg_get_num_cus() compute units (the order of the gradient's
 * column sums goes by their number), the other calls over as many workgroups
 * as they have work for.
 */
#ifndef DG_MOE_H
#define DG_MOE_H

#include "../dg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row layouts of the grouped GEMMs (dg.h). DG_MOE_DENSE: every row is valid. */
#define DG_MOE_DENSE 0
#define DG_MOE_CONTIGUOUS 1
#define DG_MOE_MASKED 2
#define DG_MOE_NOPAD 3

/*
 * Where the slots of a batch of tokens go. Slot (t, j) is token t's j-th
 * choice of expert. Filled by dg_moe_sort (or a dispatch given topk_ids) and
 * read by the other calls; the fields themselves are set by the caller.
 *   layout      DG_MOE_CONTIGUOUS, DG_MOE_MASKED or DG_MOE_NOPAD
 *   max_tokens  most tokens a call may bring
 *   top_k       slots of a token, 1..32
 *   num_groups  groups (local experts) G, 1..4096 (no-padding: 1..2048)
 *   rows        contiguous and no-padding: rows M of the permuted buffers
 *               (contiguous: a multiple of 128); masked: max_m, rows a group;
 *               M and G * max_m below 2^30
 *   hidden      values of a token, a multiple of 128
 *   row_of      [max_tokens][top_k] int32: row of each slot in the permuted
 *               buffer (masked: group * max_m + row), -1 for a dropped slot
 *   group_rows  [G] int32: rows of each group: the no-padding GEMMs'
 *               group_rows and the masked GEMMs' masked_m
 *   grouped_layout  contiguous: [M] int32, each row's group or -1; else NULL
 *   workspace   16-byte aligned, dg_moe_workspace_bytes() bytes; contents
 *               need not be kept between calls. Calls that use one plan must
 *               be ordered (one stream, or events).
 */
typedef struct dg_moe_plan {
  int layout, max_tokens, top_k, num_groups, rows, hidden;
  int32_t* row_of;
  int32_t* group_rows;
  int32_t* grouped_layout;
  void* workspace;
  long long workspace_bytes;
} dg_moe_plan;

/* Bytes of a plan's workspace (from its sizes; the pointers are not read),
 * or -1 if the sizes are not valid. */
long long dg_moe_workspace_bytes(const dg_moe_plan* plan);

/*
 * Sorts the slots by group, stably: a group's slots keep their order
 * t * top_k + j. topk_ids [tokens][top_k] int32 holds each slot's group; an
 * id outside [0, G) drops the slot. Group g's rows are, by layout,
 *   masked:      g * max_m + 0, 1, ...; slots past max_m are dropped;
 *   no-padding:  after the rows of the groups before it;
 *   contiguous:  from the next multiple of 128 after the group before it;
 * and a row at or past M is dropped. Writes row_of[0..tokens), group_rows
 * (rows kept) and, for the contiguous layout, all of grouped_layout.
 * max_tokens * top_k <= 2^22. tokens == 0 gives groups without rows.
 */
dg_status dg_moe_sort(const dg_moe_plan* plan, const int32_t* topk_ids, int tokens, void* stream);

/*
 * Copies each token to the rows of its slots: xp[row_of[t][j]] = x[t].
 *   x [tokens][hidden] BF16; xp [M][hidden] (masked [G][max_m][hidden]) BF16
 * Rows without a token are not written. With topk_ids the slots are sorted
 * first, as by dg_moe_sort; NULL uses the plan as it stands. The gradient of
 * this call is dg_moe_combine without weights.
 */
dg_status dg_moe_dispatch(const dg_moe_plan* plan, const int32_t* topk_ids, const void* x, void* xp, int tokens,
                          void* stream);

/*
 * The same with the token quantised into the GEMMs' LHS operand: per 128
 * values one scale s = max(amax, 1e-4) / 448 (ue8m0 != 0: rounded up to a
 * power of two) and codes e4m3(x / s).
 *   q   [M][hidden] E4M3 (masked [G][max_m][hidden])
 *   sfa [hidden/128][dg_get_tma_aligned_size(M, 4)] float32
 *       (masked [G][hidden/128][dg_get_tma_aligned_size(max_m, 4)])
 * The *_ue8m0 GEMMs and the FP8 x FP4 GEMMs read only a scale's exponent:
 * operands for them need ue8m0 != 0 (a float32 scale's mantissa would be
 * dropped, and the block come out up to a factor of two too small, without an
 * error). Power-of-two scales are right for the other GEMMs too.
 * A NaN in a block makes its scale and codes NaN; an infinity makes the scale
 * infinite, its own code NaN and the others zero.
 */
dg_status dg_moe_dispatch_fp8(const dg_moe_plan* plan, const int32_t* topk_ids, const void* x, void* q, float* sfa,
                              int tokens, int ue8m0, void* stream);

/*
 * Sums a token's rows: y[t] = sum_j weights[t][j] * yp[row_of[t][j]], in
 * slot order in float32. Dropped slots add nothing, whatever their weight; a
 * token without rows gets zeros. weights [tokens][top_k] float32 or NULL for
 * ones. yp [M][hidden] BF16 (masked [G][max_m][hidden]); y [tokens][hidden] BF16.
 */
dg_status dg_moe_combine(const dg_moe_plan* plan, const void* yp, const float* weights, void* y, int tokens,
                         void* stream);

/*
 * Gradient of dg_moe_combine: dyp[row_of[t][j]] = weights[t][j] * dy[t] and
 * dweights[t][j] = sum_c dy[t][c] * yp[row_of[t][j]][c] (0 for a dropped
 * slot). Rows without a token are not written. dweights may be NULL, and yp
 * with it. dyp must not overlap yp or dy.
 */
dg_status dg_moe_combine_bwd(const dg_moe_plan* plan, const void* dy, const void* yp, const float* weights, void* dyp,
                             float* dweights, int tokens, void* stream);

/*
 * Gated activation, quantised into the second GEMM's LHS operand:
 * a = silu(g) * u = g / (1 + exp(-g)) * u, then as in dg_moe_dispatch_fp8.
 *   gu   [m][2 * inner] BF16 (masked [num_groups][m][2 * inner]): g in
 *        columns [0, inner), u in [inner, 2 * inner)
 *   q    [m][inner] E4M3; sfa [inner/128][dg_get_tma_aligned_size(m, 4)]
 *        (masked: each with the leading num_groups)
 *   rows which rows hold tokens: contiguous: grouped_layout [m] (a negative
 *        id holds none); no-padding: group_rows [num_groups]; masked:
 *        masked_m [num_groups]; dense: NULL, every row does. Counts are
 *        clamped as by the GEMMs. Other rows do not influence the result and
 *        are not written.
 * ue8m0 by the GEMM that reads the operand, as for dg_moe_dispatch_fp8.
 * inner % 128 == 0; m % 128 == 0 for the contiguous layout, m <= 2^22;
 * num_groups as in a plan (not read for the dense and contiguous layouts).
 */
dg_status dg_moe_swiglu_fp8(const void* gu, void* q, float* sfa, const int32_t* rows, int layout, int m,
                            int num_groups, int inner, int ue8m0, void* stream);

/* Gradient of the activation: with s = 1 / (1 + exp(-g)),
 *   dgu[:, :inner] = da * u * s * (1 + g * (1 - s)),  dgu[:, inner:] = da * g * s.
 * da [m][inner] BF16, dgu like gu; rows as above. */
dg_status dg_moe_swiglu_bwd(const void* da, const void* gu, void* dgu, const int32_t* rows, int layout, int m,
                            int num_groups, int inner, void* stream);

/* How a gate is spread over [tokens][hidden]. */
#define DG_MOE_GATE_NONE 0     /* ones                                        */
#define DG_MOE_GATE_CHANNEL 1  /* [hidden] float32                            */
#define DG_MOE_GATE_TOKEN 2    /* [tokens] float32                            */
#define DG_MOE_GATE_FULL 3     /* [tokens][hidden] BF16                       */

/*
 * The step between two blocks: the block's output y is normalised, gated and
 * added to the scaled residual stream x, and the result is normalised for
 * the next block. With norm(v; w) = v * rsqrt(mean(v^2) + eps) * w:
 *     h = residual_scale * x + gate * norm(y; post_weight)
 *     n = norm(h; pre_weight)          (of h before it is rounded to BF16)
 *   x, y, h, n [tokens][hidden] BF16; post_weight, pre_weight [hidden] float32
 *   rstd_post, rstd_pre [tokens] float32: the two rsqrt, for the gradient
 * y NULL (before the first block): h is x itself (residual_scale must be 1),
 * h, gate, post_weight and rstd_post must be NULL. post_weight NULL: y enters as
 * it is. n NULL (after the last block): pre_weight and rstd_pre must be NULL.
 * rstd_post and rstd_pre may be NULL where no gradient is wanted. h may be x, and n may be y.
 * hidden % 8 == 0 and at most 16384; tokens <= 2^21; eps >= 0.
 */
typedef struct dg_moe_norm {
  const void* x;
  const void* y;
  const float* post_weight;
  const void* gate;
  const float* pre_weight;
  void* h;
  void* n;
  float* rstd_post;
  float* rstd_pre;
  float residual_scale, eps;
  int gate_kind, tokens, hidden;
} dg_moe_norm;
dg_status dg_moe_block_norm(const dg_moe_norm* args, void* stream);

/* Bytes of the workspace of dg_moe_block_norm_bwd, or -1. */
long long dg_moe_block_norm_workspace_bytes(int tokens, int hidden);

/*
 * Gradient of dg_moe_block_norm. dh [tokens][hidden] BF16 is the gradient
 * that reaches h along the residual stream (NULL: none), dn the one of n
 * (NULL: n was not used). With hn = h * rstd_pre, yn = y * rstd_post:
 *     a = dn * pre_weight;  dH = dh + rstd_pre * (a - hn * mean(a * hn))
 *     dx = residual_scale * dH
 *     dgate = dH * yn * post_weight, summed over what the gate is spread over
 *     b = dH * gate * post_weight;  dy = rstd_post * (b - yn * mean(b * yn))
 *     dpost_weight = sum_t dH * gate * yn;  dpre_weight = sum_t dn * hn
 * (without post_weight: yn * post_weight is y, and dy = dH * gate).
 * dx, dy BF16; dpost_weight, dpre_weight [hidden] float32; dgate like the
 * gate (float32, BF16 for the full gate). y NULL: dy, dgate, dpost_weight,
 * post_weight, gate and rstd_post must be NULL and residual_scale 1. dn NULL:
 * pre_weight, rstd_pre and dpre_weight must be NULL, h is not read and may
 * be NULL. dgate, dpost_weight and dpre_weight may be NULL where not wanted. dx
 * may be dh and dy may be dn. tokens == 0 gives zero weight gradients.
 * workspace: 16-byte aligned, dg_moe_block_norm_workspace_bytes() bytes.
 */
typedef struct dg_moe_norm_bwd {
  const void* dh;
  const void* dn;
  const void* h;
  const void* y;
  const float* post_weight;
  const void* gate;
  const float* pre_weight;
  const float* rstd_post;
  const float* rstd_pre;
  void* dx;
  void* dy;
  float* dpost_weight;
  void* dgate;
  float* dpre_weight;
  void* workspace;
  long long workspace_bytes;
  float residual_scale;
  int gate_kind, tokens, hidden;
} dg_moe_norm_bwd;
dg_status dg_moe_block_norm_bwd(const dg_moe_norm_bwd* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_MOE_H */
