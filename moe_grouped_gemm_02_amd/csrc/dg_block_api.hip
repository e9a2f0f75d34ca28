// C ABI of the operators of a transformer block (dg_block.h): argument
// validation and launch parameters.  Every check that can be made on the host is
// made before anything is enqueued; nothing here allocates device memory or
// synchronises the host.  (The GEMM with an epilogue shares the checks of the
// others, in dg_api.hip.)

#include "dg_block.h"

#include <float.h>

#include <utility>

#include "dg_block_internal.h"
#include "dg_moe_internal.h"
#include "dg_status.h"

namespace {

using dg::aligned16;
using dg::below;
using dg::fail;
using dg::ok;

constexpr int64_t kIndexLimit = (int64_t)1 << 31;
constexpr int64_t kByteLimit = (int64_t)1 << 46;
constexpr int kMaxCols = 65535 * 128;
constexpr int kMaxSequences = 1 << 20;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(DG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

#define DG_TRY(call)                      \
  do {                                    \
    const int st_ = (call);               \
    if (st_ != DG_SUCCESS) return st_;    \
  } while (0)

// Leading dimension of a matrix with `rows` rows.
int check_ld(const char* name, int64_t ld, int64_t at_least, int multiple, int64_t rows, int elem) {
  if (ld < at_least)
    return fail(DG_ERR_INVALID_VALUE, "%s=%lld is smaller than %lld", name, (long long)ld, (long long)at_least);
  if (ld % multiple) return fail(DG_ERR_MISALIGNED, "%s must be a multiple of %d", name, multiple);
  if (!below(rows, ld, elem, kByteLimit)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s=%lld is too large", name, (long long)ld);
  return DG_SUCCESS;
}

int check_workspace(void* workspace, size_t given, size_t need) {
  if (need > 0 && (!workspace || given < need))
    return fail(DG_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, given);
  if (!aligned16(workspace)) return fail(DG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  return DG_SUCCESS;
}

// ---------------------------------------------------------------- norms --

int check_norm(int tokens, int cols, int multiple, int kind, int gate_kind, const float* gate, float eps) {
  if (tokens < 0 || cols < 1) return fail(DG_ERR_INVALID_VALUE, "tokens=%d or cols=%d out of range", tokens, cols);
  if (cols % multiple) return fail(DG_ERR_UNSUPPORTED_SHAPE, "cols=%d is not a multiple of %d", cols, multiple);
  if (cols > dg::kMaxNormCols) return fail(DG_ERR_UNSUPPORTED_SHAPE, "cols=%d is larger than %d", cols, dg::kMaxNormCols);
  if (kind != DG_NORM_RMS && kind != DG_NORM_LAYER) return fail(DG_ERR_INVALID_VALUE, "kind=%d is not a norm", kind);
  if (gate_kind < DG_GATE_NONE || gate_kind > DG_GATE_TOKEN)
    return fail(DG_ERR_INVALID_VALUE, "gate_kind=%d is not a kind of gate", gate_kind);
  if ((gate != nullptr) != (gate_kind != DG_GATE_NONE) && tokens > 0)
    return fail(DG_ERR_INVALID_VALUE, "gate and gate_kind=%d do not go together", gate_kind);
  if (!aligned(gate, gate_kind == DG_GATE_COLUMN ? 16 : 4)) return fail(DG_ERR_MISALIGNED, "gate is not aligned");
  if (!(eps >= FLT_MIN && eps <= FLT_MAX)) return fail(DG_ERR_INVALID_VALUE, "eps is not a positive normal number");
  return DG_SUCCESS;
}

int norm_impl(const uint16_t* y, const uint16_t* h, const float* gate, const float* post_weight, const float* weight,
              const float* bias, uint16_t* r, uint16_t* x, uint8_t* q, void* sf, int tokens, int cols, int64_t ld_y,
              int64_t ld_h, int64_t ld_r, int64_t ld_x, int64_t ld_sf, int kind, int post, int gate_kind,
              float res_scale, float eps, void* stream, bool pow2) {
  const bool codes = q || sf;
  DG_TRY(check_norm(tokens, cols, codes ? 128 : 8, kind, gate_kind, gate, eps));
  if (post_weight && !post) return fail(DG_ERR_INVALID_VALUE, "post_weight without post");
  // Matrices without rows may be null, parameters and scales beside them are not.
  if (tokens > 0 && !q != !sf) return fail(DG_ERR_INVALID_VALUE, "q and sf go together");
  if (tokens > 0 && (weight || bias) && !x && !q) return fail(DG_ERR_INVALID_VALUE, "weight or bias without x or q");
  DG_TRY(check_ld("ld_y", ld_y, cols, 8, tokens, 2));
  if (h) DG_TRY(check_ld("ld_h", ld_h, cols, 8, tokens, 2));
  if (r) DG_TRY(check_ld("ld_r", ld_r, cols, 8, tokens, 2));
  if (x) DG_TRY(check_ld("ld_x", ld_x, cols, 8, tokens, 2));
  if (codes) DG_TRY(check_ld("ld_sf", ld_sf, tokens, 4, cols / 128, 4));
  if (r && r == h && ld_r != ld_h) return fail(DG_ERR_INVALID_VALUE, "r in place of h needs ld_r == ld_h");
  if (tokens > 0 && !y) return fail(DG_ERR_INVALID_VALUE, "null y");
  if (tokens > 0 && !r && !x && !q) return fail(DG_ERR_INVALID_VALUE, "no result is wanted");
  for (const void* ptr : {(const void*)y, (const void*)h, (const void*)post_weight, (const void*)weight, (const void*)bias,
                          (const void*)r, (const void*)x, (const void*)q, (const void*)sf})
    if (!aligned16(ptr)) return fail(DG_ERR_MISALIGNED, "data pointers and [cols] parameters must be 16-byte aligned");
  if (tokens == 0) return ok();
  const dg::NormParams p{y,      h,    gate, post_weight, weight, bias, r,     x,                     q,    sf,        tokens,
                         cols,   ld_y, ld_h, ld_r,        ld_x,   ld_sf, kind == DG_NORM_LAYER, post != 0, gate_kind, res_scale, eps};
  return launched(dg::launch_block_norm(p, pow2, static_cast<hipStream_t>(stream)), "block_norm");
}

// -------------------------------------------------------------- balance --

struct BalanceSpace {
  size_t shares, counts, used, loss, arrived, total;
};
BalanceSpace balance_space(int tokens, int experts, int seqs) {
  auto up = [](size_t n) { return (n + 15) / 16 * 16; };
  const size_t slots = (size_t)dg::balance_slots(tokens, seqs), matrix = up(slots * experts * 4);
  BalanceSpace s{};
  s.shares = 0;
  s.counts = matrix;
  s.used = s.counts + matrix;
  s.loss = s.used + up(slots * 4);
  s.arrived = s.loss + up((size_t)seqs * dg::balance_loss_parts(experts) * 8);
  s.total = s.arrived + 16;
  return s;
}

int check_balance(int tokens, int experts, int topk, int seqs, const int32_t* offsets, int64_t ld, int score, int elem) {
  if (tokens < 0) return fail(DG_ERR_INVALID_VALUE, "tokens=%d is negative", tokens);
  if (experts < 1) return fail(DG_ERR_INVALID_VALUE, "experts=%d is not positive", experts);
  if (experts > dg::kMaxExperts)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "experts=%d is larger than %d", experts, dg::kMaxExperts);
  if (topk < 1 || topk > experts) return fail(DG_ERR_INVALID_VALUE, "topk=%d is not in [1, %d]", topk, experts);
  if (topk > dg::kMaxTopk) return fail(DG_ERR_UNSUPPORTED_SHAPE, "topk=%d is larger than %d", topk, dg::kMaxTopk);
  if ((int64_t)tokens * topk >= kIndexLimit) return fail(DG_ERR_UNSUPPORTED_SHAPE, "tokens * topk is 2^31 or more");
  if (seqs < 1) return fail(DG_ERR_INVALID_VALUE, "num_seqs=%d is not positive", seqs);
  if (!offsets && seqs != 1) return fail(DG_ERR_INVALID_VALUE, "num_seqs=%d needs seq_offsets", seqs);
  if (seqs > kMaxSequences || (int64_t)seqs * experts >= kIndexLimit)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "num_seqs=%d of %d experts is too large", seqs, experts);
  if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID)
    return fail(DG_ERR_INVALID_VALUE, "score=%d is not a score function", score);
  return check_ld("ld_logits", ld, experts, 1, tokens, elem);
}

int balance_impl(const void* logits, const int32_t* ids, const int32_t* offsets, int32_t* counts, int32_t* used,
                 float* loss, int tokens, int experts, int topk, int seqs, int64_t ld, int score, float coef,
                 void* workspace, size_t workspace_bytes, void* stream, bool bf16) {
  const int elem = bf16 ? 2 : 4;
  DG_TRY(check_balance(tokens, experts, topk, seqs, offsets, ld, score, elem));
  if (!counts || !used || !loss || (tokens > 0 && (!logits || !ids))) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned(logits, elem) || !aligned(ids, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(used, 4) || !aligned(loss, 4))
    return fail(DG_ERR_MISALIGNED, "pointers must be aligned to their element");
  const BalanceSpace at = balance_space(tokens, experts, seqs);
  DG_TRY(check_workspace(workspace, workspace_bytes, at.total));
  char* ws = static_cast<char*>(workspace);
  dg::BalanceParams p{};
  p.logits = logits, p.ids = ids, p.offsets = offsets, p.counts = counts, p.used = used, p.loss = loss;
  p.share_parts = reinterpret_cast<float*>(ws + at.shares);
  p.count_parts = reinterpret_cast<int32_t*>(ws + at.counts);
  p.used_parts = reinterpret_cast<int32_t*>(ws + at.used);
  p.loss_parts = reinterpret_cast<double*>(ws + at.loss);
  p.arrived = reinterpret_cast<uint32_t*>(ws + at.arrived);
  p.tokens = tokens, p.experts = experts, p.topk = topk, p.seqs = seqs, p.chunk = dg::balance_chunk(tokens);
  p.ld = ld, p.sigmoid = score == DG_SCORE_SIGMOID, p.coef = coef;
  p.coef_mean = (double)coef / seqs, p.experts_per_choice = (double)experts / topk;
  return launched(dg::launch_balance(p, bf16, static_cast<hipStream_t>(stream)), "moe_balance");
}

int balance_bwd_impl(const void* logits, const int32_t* counts, const int32_t* used, const int32_t* offsets,
                     const float* dloss, const void* add, void* dlogits, int tokens, int experts, int topk, int seqs,
                     int64_t ld, int64_t ld_add, int64_t ld_d, int score, float coef, void* stream, bool bf16) {
  const int elem = bf16 ? 2 : 4;
  DG_TRY(check_balance(tokens, experts, topk, seqs, offsets, ld, score, elem));
  DG_TRY(check_ld("ld_dlogits", ld_d, experts, 1, tokens, elem));
  if (add) DG_TRY(check_ld("ld_add", ld_add, experts, 1, tokens, elem));
  if (add && add == dlogits && ld_add != ld_d) return fail(DG_ERR_INVALID_VALUE, "add in place needs ld_add == ld_dlogits");
  if (tokens == 0) return ok();
  if (!logits || !counts || !used || !dlogits) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned(logits, elem) || !aligned(add, elem) || !aligned(dlogits, elem) || !aligned(counts, 4) || !aligned(used, 4) ||
      !aligned(offsets, 4) || !aligned(dloss, 4))
    return fail(DG_ERR_MISALIGNED, "pointers must be aligned to their element");
  dg::BalanceParams p{};
  p.logits = logits, p.counts = const_cast<int32_t*>(counts), p.used = const_cast<int32_t*>(used), p.offsets = offsets;
  p.dloss = dloss, p.add = add, p.dlogits = dlogits;
  p.tokens = tokens, p.experts = experts, p.topk = topk, p.seqs = seqs;
  p.ld = ld, p.ld_add = ld_add, p.ld_d = ld_d, p.sigmoid = score == DG_SCORE_SIGMOID, p.coef = coef;
  return launched(dg::launch_balance_bwd(p, bf16, static_cast<hipStream_t>(stream)), "moe_balance_bwd");
}

}  // namespace

extern "C" {

int dg_block_norm(const uint16_t* y, const uint16_t* h, const float* gate, const float* post_weight, const float* weight,
                  const float* bias, uint16_t* r, uint16_t* x, uint8_t* q, float* sf, int tokens, int cols, int64_t ld_y,
                  int64_t ld_h, int64_t ld_r, int64_t ld_x, int64_t ld_sf, int kind, int post, int gate_kind,
                  float res_scale, float eps, void* stream) {
  return norm_impl(y, h, gate, post_weight, weight, bias, r, x, q, sf, tokens, cols, ld_y, ld_h, ld_r, ld_x, ld_sf, kind,
                   post, gate_kind, res_scale, eps, stream, false);
}

int dg_block_norm_ue8m0(const uint16_t* y, const uint16_t* h, const float* gate, const float* post_weight,
                        const float* weight, const float* bias, uint16_t* r, uint16_t* x, uint8_t* q, uint8_t* sf,
                        int tokens, int cols, int64_t ld_y, int64_t ld_h, int64_t ld_r, int64_t ld_x, int64_t ld_sf,
                        int kind, int post, int gate_kind, float res_scale, float eps, void* stream) {
  return norm_impl(y, h, gate, post_weight, weight, bias, r, x, q, sf, tokens, cols, ld_y, ld_h, ld_r, ld_x, ld_sf, kind,
                   post, gate_kind, res_scale, eps, stream, true);
}

size_t dg_get_block_norm_bwd_workspace_size(int tokens, int cols) {
  if (tokens <= 0 || cols <= 0 || cols > dg::kMaxNormCols) return 0;
  return (size_t)4 * dg::norm_bwd_parts(tokens, cols) * cols * sizeof(float);
}

int dg_block_norm_bwd(const uint16_t* dx, const uint16_t* dr, const uint16_t* r, const uint16_t* y, const float* gate,
                      const float* post_weight, const float* weight, uint16_t* dy, uint16_t* dh, float* dweight,
                      float* dbias, float* dpost_weight, float* dgate, int tokens, int cols, int64_t ld_dx, int64_t ld_dr,
                      int64_t ld_r, int64_t ld_y, int64_t ld_dy, int64_t ld_dh, int kind, int post, int gate_kind,
                      float res_scale, float eps, void* workspace, size_t workspace_bytes, void* stream) {
  DG_TRY(check_norm(tokens, cols, 8, kind, gate_kind, gate, eps));
  if ((dweight || dbias || weight) && !dx && tokens > 0)
    return fail(DG_ERR_INVALID_VALUE, "weight, dweight or dbias without dx");
  if ((post_weight || dpost_weight) && !post) return fail(DG_ERR_INVALID_VALUE, "post_weight or dpost_weight without post");
  if (dgate && gate_kind == DG_GATE_NONE) return fail(DG_ERR_INVALID_VALUE, "dgate without a gate");
  const bool read_y = post || dgate;
  if (dx) DG_TRY(check_ld("ld_dx", ld_dx, cols, 8, tokens, 2));
  if (dr) DG_TRY(check_ld("ld_dr", ld_dr, cols, 8, tokens, 2));
  if (dx) DG_TRY(check_ld("ld_r", ld_r, cols, 8, tokens, 2));
  if (read_y) DG_TRY(check_ld("ld_y", ld_y, cols, 8, tokens, 2));
  DG_TRY(check_ld("ld_dy", ld_dy, cols, 8, tokens, 2));
  if (dh) DG_TRY(check_ld("ld_dh", ld_dh, cols, 8, tokens, 2));
  if (tokens > 0) {
    if (!dx && !dr) return fail(DG_ERR_INVALID_VALUE, "neither dx nor dr is given");
    if (!dy || (dx && !r) || (read_y && !y)) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  }
  for (const void* ptr : {(const void*)dx, (const void*)dr, (const void*)r, (const void*)y, (const void*)post_weight,
                          (const void*)weight, (const void*)dy, (const void*)dh, (const void*)dweight, (const void*)dbias,
                          (const void*)dpost_weight})
    if (!aligned16(ptr)) return fail(DG_ERR_MISALIGNED, "data pointers and [cols] parameters must be 16-byte aligned");
  if (!aligned(dgate, gate_kind == DG_GATE_COLUMN ? 16 : 4)) return fail(DG_ERR_MISALIGNED, "dgate is not aligned");
  const bool sums = dweight || dbias || dpost_weight || (dgate && gate_kind == DG_GATE_COLUMN);
  DG_TRY(check_workspace(workspace, workspace_bytes, sums ? dg_get_block_norm_bwd_workspace_size(tokens, cols) : 0));
  const dg::NormBwdParams p{dx,    dr,   r,     y,     gate,  post_weight, weight, dy, dh, dweight, dbias, dpost_weight, dgate,
                            static_cast<float*>(workspace), tokens, cols, ld_dx, ld_dr, ld_r, ld_y, ld_dy, ld_dh,
                            kind == DG_NORM_LAYER, post != 0, gate_kind, res_scale, eps};
  if (tokens == 0 && !sums) return ok();
  return launched(dg::launch_block_norm_bwd(p, static_cast<hipStream_t>(stream)), "block_norm_bwd");
}

size_t dg_get_moe_balance_workspace_size(int tokens, int experts, int num_seqs) {
  if (tokens < 0 || experts < 1 || experts > dg::kMaxExperts || num_seqs < 1 || num_seqs > kMaxSequences ||
      (int64_t)num_seqs * experts >= kIndexLimit)
    return 0;
  return balance_space(tokens, experts, num_seqs).total;
}

int dg_moe_balance(const float* logits, const int32_t* ids, const int32_t* seq_offsets, int32_t* counts, int32_t* used,
                   float* loss, int tokens, int experts, int topk, int num_seqs, int64_t ld_logits, int score, float coef,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return balance_impl(logits, ids, seq_offsets, counts, used, loss, tokens, experts, topk, num_seqs, ld_logits, score,
                      coef, workspace, workspace_bytes, stream, false);
}

int dg_moe_balance_bf16(const uint16_t* logits, const int32_t* ids, const int32_t* seq_offsets, int32_t* counts,
                        int32_t* used, float* loss, int tokens, int experts, int topk, int num_seqs, int64_t ld_logits,
                        int score, float coef, void* workspace, size_t workspace_bytes, void* stream) {
  return balance_impl(logits, ids, seq_offsets, counts, used, loss, tokens, experts, topk, num_seqs, ld_logits, score,
                      coef, workspace, workspace_bytes, stream, true);
}

int dg_moe_balance_bwd(const float* logits, const int32_t* counts, const int32_t* used, const int32_t* seq_offsets,
                       const float* dloss, const float* add, float* dlogits, int tokens, int experts, int topk,
                       int num_seqs, int64_t ld_logits, int64_t ld_add, int64_t ld_dlogits, int score, float coef,
                       void* stream) {
  return balance_bwd_impl(logits, counts, used, seq_offsets, dloss, add, dlogits, tokens, experts, topk, num_seqs,
                          ld_logits, ld_add, ld_dlogits, score, coef, stream, false);
}

int dg_moe_balance_bwd_bf16(const uint16_t* logits, const int32_t* counts, const int32_t* used,
                            const int32_t* seq_offsets, const float* dloss, const uint16_t* add, uint16_t* dlogits,
                            int tokens, int experts, int topk, int num_seqs, int64_t ld_logits, int64_t ld_add,
                            int64_t ld_dlogits, int score, float coef, void* stream) {
  return balance_bwd_impl(logits, counts, used, seq_offsets, dloss, add, dlogits, tokens, experts, topk, num_seqs,
                          ld_logits, ld_add, ld_dlogits, score, coef, stream, true);
}

size_t dg_get_epilogue_bwd_workspace_size(int rows, int cols) {
  if (rows <= 128 || cols <= 0) return 0;
  return ((size_t)rows + 127) / 128 * cols * sizeof(float);
}

int dg_epilogue_bwd(const uint16_t* dd, const uint16_t* pre, uint8_t* dq, float* dsf, uint8_t* dqt, float* dsft,
                    float* dbias, int rows, int cols, int64_t ld_dd, int64_t ld_pre, int64_t ld_dsf, int64_t ld_dsft,
                    int act, void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0 || cols < 0) return fail(DG_ERR_INVALID_VALUE, "rows=%d or cols=%d is negative", rows, cols);
  if (cols % 128) return fail(DG_ERR_UNSUPPORTED_SHAPE, "cols=%d is not a multiple of 128", cols);
  if (cols > kMaxCols) return fail(DG_ERR_UNSUPPORTED_SHAPE, "cols=%d is larger than %d", cols, kMaxCols);
  const int64_t row_tiles = ((int64_t)rows + 127) / 128;
  if (row_tiles * (cols / 128) >= (int64_t)1 << 24)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "2^24 or more tiles (%d x %d)", rows, cols);
  if (act < DG_ACT_NONE || act > DG_ACT_GELU_TANH) return fail(DG_ERR_INVALID_VALUE, "act=%d is not an activation", act);
  if (!dqt != !dsft) return fail(DG_ERR_INVALID_VALUE, "dqt and dsft go together");
  DG_TRY(check_ld("ld_dd", ld_dd, cols, 8, rows, 2));
  if (act != DG_ACT_NONE) DG_TRY(check_ld("ld_pre", ld_pre, cols, 8, rows, 2));
  DG_TRY(check_ld("ld_dsf", ld_dsf, rows, 4, cols / 128, 4));
  if (dqt) DG_TRY(check_ld("ld_dsft", ld_dsft, cols, 4, row_tiles, 4));
  if (cols == 0) return ok();
  if (rows > 0 && (!dd || !dq || !dsf || (act != DG_ACT_NONE && !pre)))
    return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  for (const void* ptr : {(const void*)dd, (const void*)pre, (const void*)dq, (const void*)dsf, (const void*)dqt,
                          (const void*)dsft, (const void*)dbias})
    if (!aligned16(ptr)) return fail(DG_ERR_MISALIGNED, "all pointers must be 16-byte aligned");
  DG_TRY(check_workspace(workspace, workspace_bytes, dbias ? dg_get_epilogue_bwd_workspace_size(rows, cols) : 0));
  if (rows == 0 && !dbias) return ok();
  const dg::EpilogueBwdParams p{dd,   pre,  dq,    dsf,    dqt,    dsft,    dbias, static_cast<float*>(workspace),
                                rows, cols, ld_dd, ld_pre, ld_dsf, ld_dsft, act};
  return launched(dg::launch_epilogue_bwd(p, static_cast<hipStream_t>(stream)), "epilogue_bwd");
}

}  // extern "C"
