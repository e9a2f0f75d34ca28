/*
 * dg_moe.h - C ABI of libdg, continued: the operators of a mixture-of-experts
 * layer around the grouped FP8 GEMMs of dg.h.
 *
 *   routing      dg_moe_route*: logits -> expert ids and weights, and the
 *                gradient of the weights;
 *   exchange     dg_moe_plan_*, dg_moe_dispatch*: token rows -> quantised
 *                expert rows in the contiguous or masked layout;
 *                dg_moe_combine, dg_moe_combine_bwd: expert rows -> weighted
 *                token rows, and the gradient;
 *   checkpoints  dg_swiglu_quant*, dg_swiglu_bwd, dg_requant_t: the experts'
 *                gated unit with its input kept in 8 bits, and what the
 *                backward pass makes of that (gradient rows and the operands
 *                of dg_k_grouped_nt).
 *
 * A layer's forward pass is route, plan, dispatch, grouped GEMM, swiglu_quant,
 * grouped GEMM, combine; its backward pass combine_bwd, grouped GEMM,
 * swiglu_bwd, grouped GEMM, combine (with no weights), route_bwd, and two
 * K-grouped GEMMs for the weight gradients.
 *
 * Conventions are those of dg.h: device pointers owned by the caller, work
 * enqueued on `stream` and nothing else, graph-capturable, negative dg_status
 * codes decided on the host before any launch, dg_get_last_error_string().
 * Inputs are never written; outputs must not alias inputs.  A call with no
 * tokens or no rows is a successful no-op, except that the plan then
 * describes an empty layout and dg_moe_combine still writes its (zero) rows.
 * Index arrays are read on the device: values out of range name no row, and
 * nothing is accessed out of bounds for any content.  NaN or infinite values
 * in rows that are in use are outside the contract of the quantising entry
 * points (as for dg_quant_1x128); in rows that the layout leaves out they are
 * never looked at.
 *
 * Matrices have at most 65535 * 128 columns (h, hq and what has their width
 * included), byte offsets stay below 2^46; smaller limits stand with the calls.
 *
 * 1x128 codes of float32 values (the gated unit's output and all gradients):
 *   s = amax / 448 in fp32, at least 2^-126, 0 for an all-zero tile;
 *   q = e4m3( v / s ), the quotient within 2 ulp of fp32.
 * Codes of bf16 values (dispatch, the checkpoint) follow dg_quant_1x128 bit
 * for bit.  No value is rounded to bf16 on the way to its code.
 */
#ifndef DG_MOE_H_
#define DG_MOE_H_

#include "dg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* -------------------------------------------------------------- routing -- */

/* Score functions of the router. */
enum { DG_SCORE_SOFTMAX = 0, DG_SCORE_SIGMOID = 1 };

/*
 * Expert routing.  For every token, with logits x[0 .. experts):
 *   s_e   = exp(x_e - max x) / sum_i exp(x_i - max x)     (softmax), or
 *           1 / (1 + exp(-x_e))                           (sigmoid);
 *   key_e = x_e without a bias (the order of the scores, without their
 *           rounding), s_e + bias_e with one;
 *   expert groups (expert_groups > 1): the experts form expert_groups equal
 *           consecutive groups; a group's score is the sum of its group_top
 *           (1 or 2) largest s_e + bias_e, and only the topk_groups groups of
 *           the largest scores take part;
 *   ids   = the topk experts of the largest keys, in descending order;
 *   w_j   = scale * s_ids[j] / sum_i s_ids[i]   (renormalize != 0), or
 *           scale * s_ids[j].
 * Equal keys, and equal group scores, go to the lowest index.  An expert
 * whose logit or bias is -inf is masked: it is never chosen and adds nothing
 * to its group's score, and a group of masked experts is never chosen.  Slots
 * left without an expert get id -1 and weight 0 (all of them, in a row whose
 * experts are all masked).  A key that is NaN is never chosen; a NaN logit
 * makes every softmax score of its token NaN, which then shows in its weights
 * or, where the keys hold scores, leaves the token without experts.
 *   logits  [tokens][ld_logits] float32 (or bf16), ld_logits >= experts
 *   bias    [experts] float32, or NULL
 *   ids     [tokens][topk] int32, weights [tokens][topk] float32
 * Rules: 1 <= experts <= 1024, 1 <= topk <= min(32, experts), expert_groups
 * divides experts and is at most 64, 1 <= topk_groups <= expert_groups,
 * group_top 1 or 2 (DG_ERR_UNSUPPORTED_SHAPE above the maxima,
 * DG_ERR_INVALID_VALUE otherwise); pointers aligned to their element.
 */
int dg_moe_route(const float* logits, const float* bias, int32_t* ids, float* weights, int tokens,
                 int experts, int topk, int64_t ld_logits, int score, int expert_groups,
                 int topk_groups, int group_top, int renormalize, float scale, void* stream);
int dg_moe_route_bf16(const uint16_t* logits, const float* bias, int32_t* ids, float* weights,
                      int tokens, int experts, int topk, int64_t ld_logits, int score,
                      int expert_groups, int topk_groups, int group_top, int renormalize,
                      float scale, void* stream);

/*
 * Gradient of the routing weights with respect to the logits; the choice of
 * experts (and with it the bias and the groups) is held fixed.  With S the
 * sum of the chosen scores (the scores are computed again from the logits)
 * and r_j = s_j / S (0 where S is 0), for the chosen experts:
 *   z_j  = scale * r_j (dw_j - sum_i dw_i r_i)        (renormalize), or
 *          scale * s_j dw_j;
 *   dx_e = z_e (1 - s_e)                              (sigmoid), or
 *          z_e                                        (softmax, renormalize), or
 *          z_e - s_e sum_i z_i                        (softmax),
 * with z_e = 0 for experts that were not chosen.  Slots whose id is not in
 * [0, experts) take no part.  A token's ids must be distinct.
 *   dweights [tokens][topk] float32
 *   dlogits  [tokens][ld_dlogits], of the logits' type; all `experts` columns
 *            are written.
 */
int dg_moe_route_bwd(const float* logits, const int32_t* ids, const float* dweights,
                     float* dlogits, int tokens, int experts, int topk, int64_t ld_logits,
                     int64_t ld_dlogits, int score, int renormalize, float scale, void* stream);
int dg_moe_route_bwd_bf16(const uint16_t* logits, const int32_t* ids, const float* dweights,
                          uint16_t* dlogits, int tokens, int experts, int topk,
                          int64_t ld_logits, int64_t ld_dlogits, int score, int renormalize,
                          float scale, void* stream);

/* ------------------------------------------------------------- exchange -- */

/*
 * Row plan of a layout from the routed ids [tokens][topk]: expert
 * first_expert + g is this device's group g, 0 <= g < num_groups; other ids
 * (and -1) have no row.  Entries (t, j) of a group take its rows in the order
 * of t * topk + j.
 *   rows [tokens][topk] int32: the entry's row in the layout, -1 if none
 *   src  [layout rows] int32: the row's entry t * topk + j, -1 if unused
 * Contiguous layout of m_total rows (a multiple of 128): group g's rows begin
 * at k_offsets[g], each group padded to a multiple of 128 rows; entries whose
 * row would be m_total or more are dropped (row -1).
 *   m_indices [m_total] int32: g for rows in use, -1 for the others (the form
 *             dg_grouped_contiguous takes)
 *   k_offsets [num_groups + 1] int32: starts of the groups and the end of the
 *             last, at most m_total (the form dg_k_grouped_nt takes; rows past
 *             k_offsets[num_groups] belong to no group)
 * Masked layout of [num_groups][m_max] rows: row g * m_max + i; entries past
 * m_max are dropped.
 *   masked_m [num_groups] int32: rows in use, at most m_max (the form
 *             dg_grouped_masked takes)
 * workspace: dg_get_moe_plan_workspace_size(tokens, topk, num_groups) bytes,
 * 16-byte aligned, contents irrelevant; may be NULL when that is 0.  Calls
 * that run at the same time must not share it.
 * Rules: 1 <= topk <= 32, 1 <= num_groups <= 1024, tokens * topk < 2^31,
 * layout rows < 2^31.
 */
int dg_moe_plan_contiguous(const int32_t* ids, int32_t* rows, int32_t* src, int32_t* m_indices,
                           int32_t* k_offsets, int tokens, int topk, int first_expert,
                           int num_groups, int m_total, void* workspace, size_t workspace_bytes,
                           void* stream);
int dg_moe_plan_masked(const int32_t* ids, int32_t* rows, int32_t* src, int32_t* masked_m,
                       int tokens, int topk, int first_expert, int num_groups, int m_max,
                       void* workspace, size_t workspace_bytes, void* stream);
size_t dg_get_moe_plan_workspace_size(int tokens, int topk, int num_groups);

/*
 * Dispatch: row r of the layout becomes the 1x128 codes of token
 * src[r] / topk, bit for bit those of dg_quant_1x128 (dg_quant_1x128_ue8m0).
 * Rows with src[r] outside [0, tokens * topk) are not written.
 *   x   [tokens][ld_x] bf16, ld_x >= cols and a multiple of 8
 *   src [num_groups * rows] int32
 *   q   [num_groups][rows][cols] e4m3
 *   sf  [num_groups][cols/128][ld_sf] fp32 (UE8M0: bytes), ld_sf >= rows, % 4
 * (num_groups = 1, rows = m_total for the contiguous layout.)
 * cols % 128 == 0; x, q, sf 16-byte aligned.
 */
int dg_moe_dispatch(const uint16_t* x, const int32_t* src, uint8_t* q, float* sf, int tokens,
                    int topk, int cols, int rows, int num_groups, int64_t ld_x, int64_t ld_sf,
                    void* stream);
int dg_moe_dispatch_ue8m0(const uint16_t* x, const int32_t* src, uint8_t* q, uint8_t* sf,
                          int tokens, int topk, int cols, int rows, int num_groups, int64_t ld_x,
                          int64_t ld_sf, void* stream);

/*
 * Combine: y[t] = bf16( sum_j w[t][j] * d[rows[t][j]] ), summed in fp32 in the
 * order of j; slots whose row is outside [0, total_rows) add nothing, and a
 * token without rows gets zeros.  weights NULL: all ones (the gradient of
 * dispatch with respect to its tokens).
 *   d [total_rows][ld_d] bf16 (the grouped GEMM's output; for the masked
 *   layout total_rows = num_groups * m_max), y [tokens][ld_y] bf16
 * cols % 8 == 0; ld_d, ld_y >= cols and multiples of 8; d, y 16-byte aligned.
 */
int dg_moe_combine(const uint16_t* d, const int32_t* rows, const float* weights, uint16_t* y,
                   int tokens, int topk, int cols, int total_rows, int64_t ld_d, int64_t ld_y,
                   void* stream);

/*
 * Gradient of the combine over a contiguous layout of m_total rows, from the
 * tokens' gradient dy and the d, rows, src and weights of the forward pass:
 *   dd[r] = w[src[r]] * dy[src[r] / topk]  (fp32), returned as 1x128 codes
 *     dq  [m_total][cols], dsf [cols/128][ld_dsf]: rows of the input-gradient
 *         GEMM; rows not in use are not written
 *     dqt [cols][m_total], dsft [m_total/128][ld_dsft]: the transpose with one
 *         scale per column and 128 rows, an operand of dg_k_grouped_nt; zeros
 *         at rows not in use, and 128-row blocks with no row in use are not
 *         written.  dqt and dsft may both be NULL.
 *   dweights [tokens][topk] = sum_n dy[t][n] * d[rows[t][j]][n], 0 without a row
 * workspace: dg_get_moe_combine_bwd_workspace_size(m_total, cols) bytes,
 * 16-byte aligned, contents irrelevant.
 * cols % 128 == 0, m_total % 128 == 0, m_total < 2^30, m_total * cols < 2^38;
 * ld_dy, ld_d multiples of 8;
 * ld_dsf >= m_total, ld_dsft >= cols, multiples of 4; all pointers but the
 * index arrays', weights' and dweights' 16-byte aligned.
 */
int dg_moe_combine_bwd(const uint16_t* dy, const uint16_t* d, const int32_t* src,
                       const int32_t* rows, const float* weights, uint8_t* dq, float* dsf,
                       uint8_t* dqt, float* dsft, float* dweights, int tokens, int topk, int cols,
                       int m_total, int64_t ld_dy, int64_t ld_d, int64_t ld_dsf, int64_t ld_dsft,
                       void* workspace, size_t workspace_bytes, void* stream);
size_t dg_get_moe_combine_bwd_workspace_size(int m_total, int cols);

/* ---------------------------------------------------------- checkpoints -- */

/*
 * Gated unit of the experts, quantised: h [num_groups][rows][ld_h] bf16 holds
 * `inter` gate columns and then `inter` up columns, and
 *   a = silu(gate) * up,  silu(v) = v / (1 + exp(-v))   (fp32)
 * is returned as 1x128 codes, the next grouped GEMM's operand:
 *   q [num_groups][rows][inter] e4m3, sf [num_groups][inter/128][ld_sf]
 * With hq and hsf (both or neither) it also writes the 8-bit checkpoint of h,
 * bit for bit dg_quant_1x128 of it (a *_qout GEMM that produces h writes the
 * same checkpoint in its epilogue, and these are then left NULL):
 *   hq [num_groups][rows][2 inter] e4m3, hsf [num_groups][2 inter/128][ld_hsf]
 * Rows in use: all (m_indices and masked_m NULL), those with m_indices[r] >= 0
 * (m_indices [rows]; needs num_groups == 1), or the first masked_m[g] of
 * group g (masked_m [num_groups]).  Other rows are not written.
 * inter % 128 == 0, num_groups <= 65535; ld_h >= 2 inter, a multiple of 8; ld_sf, ld_hsf >= rows,
 * multiples of 4; data pointers 16-byte aligned.
 */
int dg_swiglu_quant(const uint16_t* h, const int32_t* m_indices, const int32_t* masked_m,
                    uint8_t* q, float* sf, uint8_t* hq, float* hsf, int rows, int inter,
                    int num_groups, int64_t ld_h, int64_t ld_sf, int64_t ld_hsf, void* stream);
/* The same with UE8M0 scales (the exponent rule of dg_quant_1x128_ue8m0 on
 * the fp32 amax; codes of a / 2^(E-127)), without a checkpoint. */
int dg_swiglu_quant_ue8m0(const uint16_t* h, const int32_t* m_indices, const int32_t* masked_m,
                          uint8_t* q, uint8_t* sf, int rows, int inter, int num_groups,
                          int64_t ld_h, int64_t ld_sf, void* stream);

/*
 * Backward pass of the gated unit from its 8-bit checkpoint, over a
 * contiguous layout of m_total rows.  With gate and up decoded from
 * (hq, hsf), sig = 1 / (1 + exp(-gate)) and da = dact:
 *   d gate = da * up * (sig + gate * sig * (1 - sig)),  d up = da * gate * sig
 * and dh = [d gate | d up], all in fp32, returned as
 *   dq  [m_total][2 inter], dsf [2 inter/128][ld_dsf]: rows of the
 *       input-gradient GEMM; rows not in use are not written
 *   dqt [2 inter][m_total], dsft [m_total/128][ld_dsft]: operand of the first
 *       weight-gradient GEMM (dg_k_grouped_nt)
 *   aqt [inter][m_total], asft [m_total/128][ld_asft]: silu(gate) * up again,
 *       as an operand of the second weight-gradient GEMM; both may be NULL
 * Rows in use: m_indices[r] >= 0, or all with m_indices NULL.  The transposed
 * outputs hold zeros at rows not in use; 128-row blocks with no row in use
 * are not written.
 *   hq [m_total][2 inter] e4m3, hsf [2 inter/128][ld_hsf] fp32
 *   dact [m_total][ld_dact] bf16
 * inter % 128 == 0, m_total % 128 == 0, m_total * inter < 2^45; ld_dact >= inter,
 * % 8; ld_hsf and ld_dsf >= m_total, ld_dsft >= 2 inter, ld_asft >= inter, all % 4; data
 * pointers 16-byte aligned.
 */
int dg_swiglu_bwd(const uint8_t* hq, const float* hsf, const uint16_t* dact,
                  const int32_t* m_indices, uint8_t* dq, float* dsf, uint8_t* dqt, float* dsft,
                  uint8_t* aqt, float* asft, int m_total, int inter, int64_t ld_hsf,
                  int64_t ld_dact, int64_t ld_dsf, int64_t ld_dsft, int64_t ld_asft, void* stream);

/*
 * A row-wise 8-bit checkpoint as a weight-gradient operand: the values of
 * (q [rows][cols], sf [cols/128][ld_sf]) quantised again with one scale per
 * column and 128 rows, transposed:
 *   qt [cols][rows] e4m3, sft [rows/128][ld_sft] fp32
 * Rows in use, zeros and unwritten blocks as for dg_swiglu_bwd.
 * rows % 128 == 0, cols % 128 == 0, rows * cols < 2^38; ld_sf >= rows,
 * ld_sft >= cols, % 4.
 */
int dg_requant_t(const uint8_t* q, const float* sf, const int32_t* m_indices, uint8_t* qt,
                 float* sft, int rows, int cols, int64_t ld_sf, int64_t ld_sft, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_MOE_H_ */
