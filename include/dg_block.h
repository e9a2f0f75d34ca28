/*
 * dg_block.h - C ABI of libdg, continued: what a transformer block needs around
 * the FP8 GEMMs of dg.h and the experts of dg_moe.h.
 *
 *   norms       dg_block_norm*: the junction of two blocks - norm after a
 *               block, gate and residual scale, norm before the next - with
 *               the next GEMM's operand as its result, and its gradient;
 *   balance     dg_moe_balance*: per-expert counts and the load-balance loss
 *               of a router, and its gradient;
 *   epilogue    dg_fp8_gemm_nt_epilogue*: the dense GEMM with bias,
 *               activation and residual; dg_epilogue_bwd: the gradient of what
 *               follows the sum, as operands of the two gradient GEMMs.
 *
 * Conventions are those of dg.h and dg_moe.h: device pointers owned by the
 * caller, work enqueued on `stream` and nothing else, graph-capturable,
 * negative dg_status codes decided on the host before any launch,
 * dg_get_last_error_string().  Inputs are never written; outputs must not
 * alias inputs, or each other, but where a call says so.  A workspace's contents
 * are irrelevant unless stated; calls that run at the same time must not share
 * one.  Byte offsets stay below 2^46.
 *
 * Sums, means and statistics are float32; each result is rounded once, at the
 * end.  1x128 codes of float32 values are those of dg_moe.h (s = amax / 448, at
 * least 2^-126, 0 for an all-zero tile; q = e4m3(v / s)); NaN and infinite
 * values are outside the contract of codes, and show in the other outputs of
 * their row or column.
 */
#ifndef DG_BLOCK_H_
#define DG_BLOCK_H_

#include "dg_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- norms -- */

/* Norms of a row v of n values: v / sqrt(mean v^2 + eps), or
 * (v - mean v) / sqrt(mean (v - mean v)^2 + eps). */
enum { DG_NORM_RMS = 0, DG_NORM_LAYER = 1 };

/* How many values a gate has: none, one a column, one a token. */
enum { DG_GATE_NONE = 0, DG_GATE_COLUMN = 1, DG_GATE_TOKEN = 2 };

/*
 * The junction of two blocks.  With y the output of a block, h the residual
 * stream before it, and * taken column by column:
 *   u = y, or norm(y) * post_weight              (post != 0)
 *   r = res_scale * h + gate * u                 (h NULL: gate * u)
 *   x = norm(r) * weight + bias
 * all in float32.  Results, each left out where its pointer is NULL:
 *   r  bf16, the residual stream after the block
 *   x  bf16
 *   q, sf  the 1x128 codes of x (both or neither), operand of a GEMM
 * x and q come from the float32 r, not from its rounding.  post_weight and
 * weight NULL: ones; bias NULL: none.  A first norm (of an embedding) is the
 * call with h and gate NULL and post 0, a last residual one without x and q.
 *   y [tokens][ld_y] bf16, h [tokens][ld_h] bf16
 *   gate float32 [cols] (gate_kind DG_GATE_COLUMN) or [tokens] (DG_GATE_TOKEN)
 *   post_weight, weight, bias [cols] float32
 *   r [tokens][ld_r], x [tokens][ld_x] bf16; q [tokens][cols] e4m3,
 *   sf [cols/128][ld_sf] float32 (UE8M0: exponent bytes, the rule of
 *   dg_swiglu_quant_ue8m0); entries of sf past the last token are not written.
 * r may be the same matrix as h (with ld_r == ld_h): the stream in place.
 * Rules: cols % 8 == 0 (% 128 == 0 with codes), at most 16384; lds >= cols,
 * multiples of 8; ld_sf >= tokens, a multiple of 4; eps a positive normal number;
 * data pointers and those of [cols] parameters 16-byte aligned, a token gate's
 * 4-byte.  Squares are float32: a normalised row stays below 2^56 in magnitude.
 */
int dg_block_norm(const uint16_t* y, const uint16_t* h, const float* gate, const float* post_weight,
                  const float* weight, const float* bias, uint16_t* r, uint16_t* x, uint8_t* q,
                  float* sf, int tokens, int cols, int64_t ld_y, int64_t ld_h, int64_t ld_r,
                  int64_t ld_x, int64_t ld_sf, int kind, int post, int gate_kind, float res_scale,
                  float eps, void* stream);
int dg_block_norm_ue8m0(const uint16_t* y, const uint16_t* h, const float* gate,
                        const float* post_weight, const float* weight, const float* bias,
                        uint16_t* r, uint16_t* x, uint8_t* q, uint8_t* sf, int tokens, int cols,
                        int64_t ld_y, int64_t ld_h, int64_t ld_r, int64_t ld_x, int64_t ld_sf,
                        int kind, int post, int gate_kind, float res_scale, float eps,
                        void* stream);

/*
 * Its gradient.  dx is the gradient of x, dr the one that reaches r along the
 * residual stream (either may be NULL, for none).  With n = norm(r),
 * s = 1 / sqrt(..) of r, g = dx * weight, and m(..) the mean over the row:
 *   t  = dr + s (g - n m(g n))                   (layer: .. - s m(g))
 *   dh = res_scale * t
 *   dweight = sum over tokens of dx * n,  dbias = sum of dx
 *   dgate   = sum of t * u over tokens (column) or over the row (token)
 *   e  = gate * t
 *   dy = e, or the gradient of norm(y) * post_weight from e as above (post),
 *   dpost_weight = sum over tokens of e * norm(y).
 * Each result is left out where its pointer is NULL, dy alone excepted.  r is
 * read as rounded by the forward pass (with dx), y where post is set or dgate is
 * wanted; either may be NULL where it is not read.
 *   dx, dr, r, y, dy, dh [tokens][ld] bf16; dweight, dbias, dpost_weight [cols],
 *   dgate [cols] or [tokens], float32
 * dweight and dbias need dx, dpost_weight needs post, dgate a gate.  With no
 * tokens the [cols] results are zeros.  The order of the sums is fixed: results
 * do not change from run to run.
 * workspace: dg_get_block_norm_bwd_workspace_size(tokens, cols) bytes, 16-byte
 * aligned; may be NULL where no [cols] result is wanted.
 * Rules as for dg_block_norm; [cols] results 16-byte aligned.
 */
int dg_block_norm_bwd(const uint16_t* dx, const uint16_t* dr, const uint16_t* r, const uint16_t* y,
                      const float* gate, const float* post_weight, const float* weight,
                      uint16_t* dy, uint16_t* dh, float* dweight, float* dbias,
                      float* dpost_weight, float* dgate, int tokens, int cols, int64_t ld_dx,
                      int64_t ld_dr, int64_t ld_r, int64_t ld_y, int64_t ld_dy, int64_t ld_dh,
                      int kind, int post, int gate_kind, float res_scale, float eps,
                      void* workspace, size_t workspace_bytes, void* stream);
size_t dg_get_block_norm_bwd_workspace_size(int tokens, int cols);

/* -------------------------------------------------------------- balance -- */

/*
 * Load balance of a router over sequences.  Sequence s is the tokens
 * seq_offsets[s] .. seq_offsets[s + 1] - 1 (seq_offsets NULL: one sequence of
 * all tokens).  With p the shares of a token's experts,
 *   p_e = softmax of the logits, or s_e / sum_i s_i with s = 1 / (1 + exp(-x)),
 * n the sequence's tokens in use (those with a logit other than -inf) and c_e
 * how often the ids of these name expert e:
 *   f_e = experts * c_e / (topk * n),  P_e = (sum of p_e over its tokens) / n,
 *   loss = coef * mean over sequences of sum_e f_e P_e
 * (a sequence with no token in use adds 0).  The shares of a masked expert
 * (logit -inf) are 0; ids outside [0, experts) are not counted.
 *   logits [tokens][ld_logits] float32 (or bf16), ids [tokens][topk] int32
 *   seq_offsets [num_seqs + 1] int32, not descending, or NULL (num_seqs 1).
 *       Tokens before the first and behind the last take no part.  Other contents
 *       give unspecified results, and nothing is accessed out of bounds.
 *   counts [num_seqs][experts] int32, used [num_seqs] int32 (n), loss [1] float32
 * The order of the sums is fixed: results do not change from run to run.
 * workspace: dg_get_moe_balance_workspace_size(tokens, experts, num_seqs)
 * bytes, 16-byte aligned.
 * Rules: 1 <= experts <= 1024, 1 <= topk <= min(32, experts), 1 <= num_seqs <=
 * 2^20, tokens * topk and num_seqs * experts below 2^31; pointers aligned to
 * their element.  With no tokens the results are zeros.
 */
int dg_moe_balance(const float* logits, const int32_t* ids, const int32_t* seq_offsets,
                   int32_t* counts, int32_t* used, float* loss, int tokens, int experts, int topk,
                   int num_seqs, int64_t ld_logits, int score, float coef, void* workspace,
                   size_t workspace_bytes, void* stream);
int dg_moe_balance_bf16(const uint16_t* logits, const int32_t* ids, const int32_t* seq_offsets,
                        int32_t* counts, int32_t* used, float* loss, int tokens, int experts,
                        int topk, int num_seqs, int64_t ld_logits, int score, float coef,
                        void* workspace, size_t workspace_bytes, void* stream);
size_t dg_get_moe_balance_workspace_size(int tokens, int experts, int num_seqs);

/*
 * Its gradient with respect to the logits (the counts are constants), from the
 * forward pass' counts and used:
 *   a = dloss * coef / (num_seqs * n),  m = sum_i f_i p_i
 *   dlogits_e = add_e + a p_e (f_e - m)                  (softmax), or
 *               add_e + a p_e (1 - s_e) (f_e - m)        (sigmoid)
 *   dloss [1] float32 on the device, or NULL for 1
 *   add   [tokens][ld_add] of the logits' type, or NULL for none; it may be
 *         dlogits itself (with ld_add == ld_dlogits): the gradient of
 *         dg_moe_route_bwd is added to in place
 *   dlogits [tokens][ld_dlogits] of the logits' type; the rows of tokens in no
 *         sequence are not written
 */
int dg_moe_balance_bwd(const float* logits, const int32_t* counts, const int32_t* used,
                       const int32_t* seq_offsets, const float* dloss, const float* add,
                       float* dlogits, int tokens, int experts, int topk, int num_seqs,
                       int64_t ld_logits, int64_t ld_add, int64_t ld_dlogits, int score,
                       float coef, void* stream);
int dg_moe_balance_bwd_bf16(const uint16_t* logits, const int32_t* counts, const int32_t* used,
                            const int32_t* seq_offsets, const float* dloss, const uint16_t* add,
                            uint16_t* dlogits, int tokens, int experts, int topk, int num_seqs,
                            int64_t ld_logits, int64_t ld_add, int64_t ld_dlogits, int score,
                            float coef, void* stream);

/* ------------------------------------------------------------- epilogue -- */

/* Activations: z; max(z, 0); z / (1 + exp(-z)); and the tanh form of the GELU,
 * z / (1 + exp(-t)), t = 2 sqrt(2 / pi) (z + 0.044715 z^3). */
enum { DG_ACT_NONE = 0, DG_ACT_RELU = 1, DG_ACT_SILU = 2, DG_ACT_GELU_TANH = 3 };

/*
 * The dense NT GEMM of dg.h with an epilogue:
 *   z = (the sum that dg_fp8_gemm_nt rounds) + bias[column]
 *   d = bf16( act(z) + residual )
 * in float32, rounded once.
 *   bias     [n] float32, or NULL
 *   residual [m][ld_res] bf16, or NULL
 *   pre      [m][ld_pre] bf16 of z, what dg_epilogue_bwd takes, or NULL
 *   dq, dsf  a quantised copy of d, exactly dg_quant_1x128 of it (UE8M0:
 *            dg_quant_1x128_ue8m0) with the rules of dg_fp8_gemm_nt_qout; both
 *            or neither
 * Everything else as for dg_fp8_gemm_nt (dg_fp8_gemm_nt_ue8m0), the workspace
 * included: dg_get_workspace_size(m, n, k, 1) bytes, zero-filled before its
 * first use.  k == 0: the sum is 0, the epilogue stays.
 * Rules: ld_res, ld_pre >= n, multiples of 8; residual and pre 16-byte, bias
 * 4-byte aligned.
 */
int dg_fp8_gemm_nt_epilogue(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                            const float* bias, const uint16_t* residual, uint16_t* d,
                            uint16_t* pre, uint8_t* dq, float* dsf, int m, int n, int k,
                            int64_t lda, int64_t ldb, int64_t ldd, int64_t ld_sfa, int64_t ld_res,
                            int64_t ld_pre, int64_t ld_dsf, int act, void* workspace,
                            size_t workspace_bytes, void* stream);
int dg_fp8_gemm_nt_ue8m0_epilogue(const uint8_t* a, const uint8_t* sfa, const uint8_t* b,
                                  const uint8_t* sfb, const float* bias, const uint16_t* residual,
                                  uint16_t* d, uint16_t* pre, uint8_t* dq, uint8_t* dsf, int m,
                                  int n, int k, int64_t lda, int64_t ldb, int64_t ldd,
                                  int64_t ld_sfa, int64_t ld_res, int64_t ld_pre, int64_t ld_dsf,
                                  int act, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the epilogue, from the gradient dd of d and the z that the
 * forward pass kept (the gradient of the residual is dd itself):
 *   dz = dd * act'(z)   (float32; act'(0) = 0 for the relu; act' of a NaN is
 *                        NaN, of an infinite z its limit, 0 or 1)
 * returned as
 *   dq  [rows][cols], dsf [cols/128][ld_dsf]: 1x128 codes, rows of the
 *       input-gradient GEMM; entries of dsf past the last row are not written
 *   dqt [cols][rows up to a multiple of 128], dsft [ceil(rows/128)][ld_dsft]:
 *       the transpose with one scale per column and 128 rows, an operand of
 *       dg_k_grouped_nt; zeros past the last row.  Both may be NULL.
 *   dbias [cols] float32 = sum over the rows of dz, or NULL
 *   dd [rows][ld_dd], pre [rows][ld_pre] bf16 (pre NULL with DG_ACT_NONE)
 * With no rows dbias is zeros.  The order of the sums is fixed.
 * workspace: dg_get_epilogue_bwd_workspace_size(rows, cols) bytes, 16-byte
 * aligned; may be NULL where that is 0 or dbias is not wanted.
 * Rules: cols % 128 == 0, at most 65535 * 128; fewer than 2^24 tiles of 128 x
 * 128; ld_dd, ld_pre >= cols, multiples of 8; ld_dsf >= rows, ld_dsft >= cols,
 * multiples of 4; all pointers 16-byte aligned.
 */
int dg_epilogue_bwd(const uint16_t* dd, const uint16_t* pre, uint8_t* dq, float* dsf, uint8_t* dqt,
                    float* dsft, float* dbias, int rows, int cols, int64_t ld_dd, int64_t ld_pre,
                    int64_t ld_dsf, int64_t ld_dsft, int act, void* workspace,
                    size_t workspace_bytes, void* stream);
size_t dg_get_epilogue_bwd_workspace_size(int rows, int cols);

#ifdef __cplusplus
}
#endif

#endif /* DG_BLOCK_H_ */
