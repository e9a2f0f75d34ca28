// C ABI of the mixture-of-experts operators (dg_moe.h): argument validation
// and launch parameters.  Every check that can be made on the host is made
// before anything is enqueued; nothing here allocates device memory or
// synchronises the host.

#include "dg_moe.h"

#include "dg_moe_internal.h"
#include "dg_status.h"

namespace {

using dg::aligned16;
using dg::below;
using dg::fail;
using dg::ok;

constexpr int64_t kRowLimit = (int64_t)1 << 31;
constexpr int64_t kWorkgroupLimit = (int64_t)1 << 24;  // of 256 threads in one grid dimension
// Byte offsets are 64-bit; a matrix this large is a wrong argument.
constexpr int64_t kByteLimit = (int64_t)1 << 46;
// A row wider than this is a wrong argument.
constexpr int kMaxCols = 65535 * 128;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(DG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

int check_cols(const char* name, int cols, int multiple) {
  if (cols < 0) return fail(DG_ERR_INVALID_VALUE, "%s=%d is negative", name, cols);
  if (cols % multiple) return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s=%d is not a multiple of %d", name, cols, multiple);
  if (cols > kMaxCols) return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s=%d is larger than %d", name, cols, kMaxCols);
  return DG_SUCCESS;
}

// Leading dimension of a row-major matrix of `rows` rows, or of a scale matrix.
int check_ld(const char* name, int64_t ld, int64_t at_least, int multiple, int64_t rows, int elem) {
  if (ld < at_least)
    return fail(DG_ERR_INVALID_VALUE, "%s=%lld is smaller than %lld", name, (long long)ld, (long long)at_least);
  if (ld % multiple) return fail(DG_ERR_MISALIGNED, "%s must be a multiple of %d", name, multiple);
  if (!below(rows, ld, elem, kByteLimit)) return fail(DG_ERR_UNSUPPORTED_SHAPE, "%s=%lld is too large", name, (long long)ld);
  return DG_SUCCESS;
}

int check_entries(int tokens, int topk) {
  if (tokens < 0) return fail(DG_ERR_INVALID_VALUE, "tokens=%d is negative", tokens);
  if (topk < 1) return fail(DG_ERR_INVALID_VALUE, "topk=%d is not positive", topk);
  if (topk > dg::kMaxTopk) return fail(DG_ERR_UNSUPPORTED_SHAPE, "topk=%d is larger than %d", topk, dg::kMaxTopk);
  if ((int64_t)tokens * topk >= kRowLimit) return fail(DG_ERR_UNSUPPORTED_SHAPE, "tokens * topk is 2^31 or more");
  return DG_SUCCESS;
}

int check_layout(int rows, int groups) {
  if (rows < 0 || groups < 1) return fail(DG_ERR_INVALID_VALUE, "rows=%d or num_groups=%d out of range", rows, groups);
  if ((int64_t)rows * groups >= kRowLimit) return fail(DG_ERR_UNSUPPORTED_SHAPE, "2^31 or more layout rows");
  return DG_SUCCESS;
}

// Tiles of 128 x 128.  Kernels that walk over them count with 32 bits; those that
// take a workgroup of 256 threads for each need fewer than 2^32 threads in all.
int check_tiles(int rows, int cols, bool workgroup_each) {
  if ((int64_t)(rows / 128) * (cols / 128) >= (workgroup_each ? kWorkgroupLimit : kRowLimit))
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "2^%d or more tiles (%d x %d)", workgroup_each ? 24 : 31, rows, cols);
  return DG_SUCCESS;
}

#define DG_TRY(call)                      \
  do {                                    \
    const int st_ = (call);               \
    if (st_ != DG_SUCCESS) return st_;    \
  } while (0)

int check_router(int tokens, int experts, int topk, int64_t ld, int score, size_t elem) {
  DG_TRY(check_entries(tokens, topk));
  if (experts < 1) return fail(DG_ERR_INVALID_VALUE, "experts=%d is not positive", experts);
  if (experts > dg::kMaxExperts)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "experts=%d is larger than %d", experts, dg::kMaxExperts);
  if (topk > experts) return fail(DG_ERR_INVALID_VALUE, "topk=%d is larger than experts=%d", topk, experts);
  if (score != DG_SCORE_SOFTMAX && score != DG_SCORE_SIGMOID)
    return fail(DG_ERR_INVALID_VALUE, "score=%d is not a score function", score);
  return check_ld("ld_logits", ld, experts, 1, tokens, (int)elem);
}

int route_impl(const void* logits, const float* bias, int32_t* ids, float* weights, int tokens, int experts, int topk,
               int64_t ld_logits, int score, int expert_groups, int topk_groups, int group_top, int renormalize,
               float scale, void* stream, bool bf16) {
  const size_t elem = bf16 ? 2 : 4;
  DG_TRY(check_router(tokens, experts, topk, ld_logits, score, elem));
  if (expert_groups < 1 || experts % expert_groups)
    return fail(DG_ERR_INVALID_VALUE, "expert_groups=%d does not divide experts=%d", expert_groups, experts);
  if (expert_groups > dg::kMaxExpertGroups)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "expert_groups=%d is larger than %d", expert_groups, dg::kMaxExpertGroups);
  if (topk_groups < 1 || topk_groups > expert_groups)
    return fail(DG_ERR_INVALID_VALUE, "topk_groups=%d is not in [1, %d]", topk_groups, expert_groups);
  if (group_top != 1 && group_top != 2) return fail(DG_ERR_INVALID_VALUE, "group_top=%d is neither 1 nor 2", group_top);
  if (tokens == 0) return ok();
  if (!logits || !ids || !weights) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned(logits, elem) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return fail(DG_ERR_MISALIGNED, "pointers must be aligned to their element");
  dg::RouteParams p{};
  p.logits = logits, p.bias = bias, p.ids = ids, p.weights = weights;
  p.tokens = tokens, p.experts = experts, p.topk = topk, p.ld = ld_logits;
  p.sigmoid = score == DG_SCORE_SIGMOID;
  p.groups = expert_groups, p.topk_groups = topk_groups, p.group_top = group_top;
  p.renormalize = renormalize != 0, p.scale = scale;
  return launched(dg::launch_route(p, bf16, static_cast<hipStream_t>(stream)), "route");
}

int route_bwd_impl(const void* logits, const int32_t* ids, const float* dweights, void* dlogits, int tokens,
                   int experts, int topk, int64_t ld_logits, int64_t ld_dlogits, int score, int renormalize,
                   float scale, void* stream, bool bf16) {
  const size_t elem = bf16 ? 2 : 4;
  DG_TRY(check_router(tokens, experts, topk, ld_logits, score, elem));
  DG_TRY(check_ld("ld_dlogits", ld_dlogits, experts, 1, tokens, (int)elem));
  if (tokens == 0) return ok();
  if (!logits || !ids || !dweights || !dlogits) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned(logits, elem) || !aligned(dlogits, elem) || !aligned(ids, 4) || !aligned(dweights, 4))
    return fail(DG_ERR_MISALIGNED, "pointers must be aligned to their element");
  dg::RouteParams p{};
  p.logits = logits, p.ids = const_cast<int32_t*>(ids), p.dweights = dweights, p.dlogits = dlogits;
  p.tokens = tokens, p.experts = experts, p.topk = topk, p.ld = ld_logits, p.ld_d = ld_dlogits;
  p.sigmoid = score == DG_SCORE_SIGMOID;
  p.renormalize = renormalize != 0, p.scale = scale;
  return launched(dg::launch_route_bwd(p, bf16, static_cast<hipStream_t>(stream)), "route_bwd");
}

int plan_impl(const int32_t* ids, int32_t* rows, int32_t* src, int32_t* m_indices, int32_t* k_offsets,
              int32_t* masked_m, int tokens, int topk, int first_expert, int num_groups, int layout_rows, int m_max,
              bool masked, void* workspace, size_t workspace_bytes, void* stream) {
  DG_TRY(check_entries(tokens, topk));
  if (num_groups > dg::kMaxLocalExperts)
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "num_groups=%d is larger than %d", num_groups, dg::kMaxLocalExperts);
  if (first_expert < 0) return fail(DG_ERR_INVALID_VALUE, "first_expert=%d is negative", first_expert);
  if ((tokens > 0 && (!ids || !rows)) || (layout_rows > 0 && (!src || (!masked && !m_indices))) ||
      (masked ? !masked_m : !k_offsets))
    return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  for (const void* ptr : {(const void*)ids, (const void*)rows, (const void*)src, (const void*)m_indices,
                          (const void*)k_offsets, (const void*)masked_m})
    if (!aligned(ptr, 4)) return fail(DG_ERR_MISALIGNED, "index arrays must be 4-byte aligned");
  const size_t need = dg::plan_workspace_bytes((int64_t)tokens * topk, num_groups);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DG_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (!aligned16(workspace)) return fail(DG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  dg::PlanParams p{};
  p.ids = ids, p.rows = rows, p.src = src, p.m_indices = m_indices, p.k_offsets = k_offsets, p.masked_m = masked_m;
  p.hist = static_cast<int32_t*>(workspace);
  p.entries = tokens * topk, p.first = first_expert, p.groups = num_groups;
  p.masked = masked, p.m_max = m_max, p.layout_rows = layout_rows;
  p.by_m_max = dg::divisor(m_max);
  return launched(dg::launch_plan(p, static_cast<hipStream_t>(stream)), "plan");
}

int dispatch_impl(const uint16_t* x, const int32_t* src, uint8_t* q, void* sf, int tokens, int topk, int cols,
                  int rows, int num_groups, int64_t ld_x, int64_t ld_sf, void* stream, bool pow2) {
  DG_TRY(check_entries(tokens, topk));
  DG_TRY(check_layout(rows, num_groups));
  DG_TRY(check_cols("cols", cols, 128));
  DG_TRY(check_ld("ld_x", ld_x, cols, 8, tokens, 2));
  DG_TRY(check_ld("ld_sf", ld_sf, rows, 4, (int64_t)num_groups * (cols / 128), 4));
  if (tokens == 0 || rows == 0 || cols == 0) return ok();
  if (!x || !src || !q || !sf) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(x) || !aligned16(q) || !aligned16(sf) || !aligned(src, 4))
    return fail(DG_ERR_MISALIGNED, "x, q and sf must be 16-byte aligned, src 4-byte aligned");
  const dg::DispatchParams p{x, src, q, sf, tokens, topk, cols, rows, num_groups, ld_x, ld_sf,
                             dg::divisor(topk), dg::divisor(rows)};
  return launched(dg::launch_dispatch(p, pow2, static_cast<hipStream_t>(stream)), "dispatch");
}

int swiglu_impl(const uint16_t* h, const int32_t* m_indices, const int32_t* masked_m, uint8_t* q, void* sf,
                uint8_t* hq, float* hsf, int rows, int inter, int num_groups, int64_t ld_h, int64_t ld_sf,
                int64_t ld_hsf, void* stream, bool pow2) {
  DG_TRY(check_layout(rows, num_groups));
  DG_TRY(check_cols("inter", inter, 128));
  if (inter > kMaxCols / 2) return fail(DG_ERR_UNSUPPORTED_SHAPE, "inter=%d is larger than %d", inter, kMaxCols / 2);
  if (num_groups > 65535) return fail(DG_ERR_UNSUPPORTED_SHAPE, "num_groups=%d is larger than 65535", num_groups);
  if (m_indices && masked_m) return fail(DG_ERR_INVALID_VALUE, "m_indices and masked_m given together");
  if (m_indices && num_groups != 1) return fail(DG_ERR_INVALID_VALUE, "m_indices needs num_groups == 1");
  if (!hq != !hsf) return fail(DG_ERR_INVALID_VALUE, "hq and hsf go together");
  DG_TRY(check_ld("ld_h", ld_h, 2 * (int64_t)inter, 8, (int64_t)rows * num_groups, 2));
  DG_TRY(check_ld("ld_sf", ld_sf, rows, 4, (int64_t)num_groups * (inter / 128), 4));
  if (hq) DG_TRY(check_ld("ld_hsf", ld_hsf, rows, 4, (int64_t)num_groups * (inter / 64), 4));
  if (rows == 0 || inter == 0) return ok();
  if (!h || !q || !sf) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(h) || !aligned16(q) || !aligned16(sf) || !aligned16(hq) || !aligned16(hsf) || !aligned(m_indices, 4) ||
      !aligned(masked_m, 4))
    return fail(DG_ERR_MISALIGNED, "data pointers must be 16-byte aligned, index arrays 4-byte aligned");
  const dg::SwigluParams p{h, m_indices, masked_m, q, sf, hq, hsf, rows, inter, num_groups, ld_h, ld_sf, ld_hsf};
  return launched(dg::launch_swiglu_quant(p, pow2, static_cast<hipStream_t>(stream)), "swiglu_quant");
}

}  // namespace

extern "C" {

int dg_moe_route(const float* logits, const float* bias, int32_t* ids, float* weights, int tokens, int experts,
                 int topk, int64_t ld_logits, int score, int expert_groups, int topk_groups, int group_top,
                 int renormalize, float scale, void* stream) {
  return route_impl(logits, bias, ids, weights, tokens, experts, topk, ld_logits, score, expert_groups, topk_groups,
                    group_top, renormalize, scale, stream, false);
}

int dg_moe_route_bf16(const uint16_t* logits, const float* bias, int32_t* ids, float* weights, int tokens,
                      int experts, int topk, int64_t ld_logits, int score, int expert_groups, int topk_groups,
                      int group_top, int renormalize, float scale, void* stream) {
  return route_impl(logits, bias, ids, weights, tokens, experts, topk, ld_logits, score, expert_groups, topk_groups,
                    group_top, renormalize, scale, stream, true);
}

int dg_moe_route_bwd(const float* logits, const int32_t* ids, const float* dweights, float* dlogits, int tokens,
                     int experts, int topk, int64_t ld_logits, int64_t ld_dlogits, int score, int renormalize,
                     float scale, void* stream) {
  return route_bwd_impl(logits, ids, dweights, dlogits, tokens, experts, topk, ld_logits, ld_dlogits, score,
                        renormalize, scale, stream, false);
}

int dg_moe_route_bwd_bf16(const uint16_t* logits, const int32_t* ids, const float* dweights, uint16_t* dlogits,
                          int tokens, int experts, int topk, int64_t ld_logits, int64_t ld_dlogits, int score,
                          int renormalize, float scale, void* stream) {
  return route_bwd_impl(logits, ids, dweights, dlogits, tokens, experts, topk, ld_logits, ld_dlogits, score,
                        renormalize, scale, stream, true);
}

int dg_moe_plan_contiguous(const int32_t* ids, int32_t* rows, int32_t* src, int32_t* m_indices, int32_t* k_offsets,
                           int tokens, int topk, int first_expert, int num_groups, int m_total, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (num_groups < 1 || m_total < 0)
    return fail(DG_ERR_INVALID_VALUE, "m_total=%d or num_groups=%d out of range", m_total, num_groups);
  if (m_total % 128) return fail(DG_ERR_UNSUPPORTED_SHAPE, "m_total=%d is not a multiple of 128", m_total);
  return plan_impl(ids, rows, src, m_indices, k_offsets, nullptr, tokens, topk, first_expert, num_groups, m_total, 0,
                   false, workspace, workspace_bytes, stream);
}

int dg_moe_plan_masked(const int32_t* ids, int32_t* rows, int32_t* src, int32_t* masked_m, int tokens, int topk,
                       int first_expert, int num_groups, int m_max, void* workspace, size_t workspace_bytes,
                       void* stream) {
  DG_TRY(check_layout(m_max, num_groups));
  return plan_impl(ids, rows, src, nullptr, nullptr, masked_m, tokens, topk, first_expert, num_groups,
                   m_max * num_groups, m_max, true, workspace, workspace_bytes, stream);
}

size_t dg_get_moe_plan_workspace_size(int tokens, int topk, int num_groups) {
  if (tokens < 0 || topk < 1 || topk > dg::kMaxTopk || num_groups < 1 || num_groups > dg::kMaxLocalExperts ||
      (int64_t)tokens * topk >= kRowLimit)
    return 0;
  return dg::plan_workspace_bytes((int64_t)tokens * topk, num_groups);
}

int dg_moe_dispatch(const uint16_t* x, const int32_t* src, uint8_t* q, float* sf, int tokens, int topk, int cols,
                    int rows, int num_groups, int64_t ld_x, int64_t ld_sf, void* stream) {
  return dispatch_impl(x, src, q, sf, tokens, topk, cols, rows, num_groups, ld_x, ld_sf, stream, false);
}

int dg_moe_dispatch_ue8m0(const uint16_t* x, const int32_t* src, uint8_t* q, uint8_t* sf, int tokens, int topk,
                          int cols, int rows, int num_groups, int64_t ld_x, int64_t ld_sf, void* stream) {
  return dispatch_impl(x, src, q, sf, tokens, topk, cols, rows, num_groups, ld_x, ld_sf, stream, true);
}

int dg_moe_combine(const uint16_t* d, const int32_t* rows, const float* weights, uint16_t* y, int tokens, int topk,
                   int cols, int total_rows, int64_t ld_d, int64_t ld_y, void* stream) {
  DG_TRY(check_entries(tokens, topk));
  if (total_rows < 0) return fail(DG_ERR_INVALID_VALUE, "total_rows=%d is negative", total_rows);
  DG_TRY(check_cols("cols", cols, 8));
  DG_TRY(check_ld("ld_d", ld_d, cols, 8, total_rows, 2));
  DG_TRY(check_ld("ld_y", ld_y, cols, 8, tokens, 2));
  if (tokens == 0 || cols == 0) return ok();
  if ((total_rows > 0 && !d) || !rows || !y) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(d) || !aligned16(y) || !aligned(rows, 4) || !aligned(weights, 4))
    return fail(DG_ERR_MISALIGNED, "d and y must be 16-byte aligned, rows and weights 4-byte aligned");
  const dg::CombineParams p{d, rows, weights, y, tokens, topk, cols, total_rows, ld_d, ld_y};
  return launched(dg::launch_combine(p, static_cast<hipStream_t>(stream)), "combine");
}

size_t dg_get_moe_combine_bwd_workspace_size(int m_total, int cols) {
  if (m_total <= 0 || cols <= 0) return 0;
  return (size_t)m_total * ((size_t)cols / 128) * sizeof(float);
}

int dg_moe_combine_bwd(const uint16_t* dy, const uint16_t* d, const int32_t* src, const int32_t* rows,
                       const float* weights, uint8_t* dq, float* dsf, uint8_t* dqt, float* dsft, float* dweights,
                       int tokens, int topk, int cols, int m_total, int64_t ld_dy, int64_t ld_d, int64_t ld_dsf,
                       int64_t ld_dsft, void* workspace, size_t workspace_bytes, void* stream) {
  DG_TRY(check_entries(tokens, topk));
  DG_TRY(check_layout(m_total, 1));
  if (m_total % 128) return fail(DG_ERR_UNSUPPORTED_SHAPE, "m_total=%d is not a multiple of 128", m_total);
  DG_TRY(check_cols("cols", cols, 128));
  DG_TRY(check_tiles(m_total, cols, true));
  if (m_total / 64 >= kWorkgroupLimit)  // a workgroup for 64 rows sums the weights' gradient
    return fail(DG_ERR_UNSUPPORTED_SHAPE, "m_total=%d is 2^30 or more", m_total);
  if (!dqt != !dsft) return fail(DG_ERR_INVALID_VALUE, "dqt and dsft go together");
  DG_TRY(check_ld("ld_dy", ld_dy, cols, 8, tokens, 2));
  DG_TRY(check_ld("ld_d", ld_d, cols, 8, m_total, 2));
  DG_TRY(check_ld("ld_dsf", ld_dsf, m_total, 4, cols / 128, 4));
  if (dqt) DG_TRY(check_ld("ld_dsft", ld_dsft, cols, 4, m_total / 128, 4));
  if (tokens == 0 || cols == 0) return ok();
  if (!rows || !dweights || !weights || !dy || (m_total > 0 && (!d || !src || !dq || !dsf)))
    return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(dy) || !aligned16(d) || !aligned16(dq) || !aligned16(dsf) || !aligned16(dqt) || !aligned16(dsft) ||
      !aligned(src, 4) || !aligned(rows, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return fail(DG_ERR_MISALIGNED, "dy, d, codes and scales must be 16-byte aligned, the others 4-byte aligned");
  const size_t need = dg_get_moe_combine_bwd_workspace_size(m_total, cols);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(DG_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (!aligned16(workspace)) return fail(DG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  const dg::CombineBwdParams p{dy,     d,    src,  rows,    weights, dq,   dsf,    dqt,     dsft, dweights, static_cast<float*>(workspace),
                               tokens, topk, cols, m_total, ld_dy,   ld_d, ld_dsf, ld_dsft, dg::divisor(topk)};
  return launched(dg::launch_combine_bwd(p, static_cast<hipStream_t>(stream)), "combine_bwd");
}

int dg_swiglu_quant(const uint16_t* h, const int32_t* m_indices, const int32_t* masked_m, uint8_t* q, float* sf,
                    uint8_t* hq, float* hsf, int rows, int inter, int num_groups, int64_t ld_h, int64_t ld_sf,
                    int64_t ld_hsf, void* stream) {
  return swiglu_impl(h, m_indices, masked_m, q, sf, hq, hsf, rows, inter, num_groups, ld_h, ld_sf, ld_hsf, stream,
                     false);
}

int dg_swiglu_quant_ue8m0(const uint16_t* h, const int32_t* m_indices, const int32_t* masked_m, uint8_t* q,
                          uint8_t* sf, int rows, int inter, int num_groups, int64_t ld_h, int64_t ld_sf,
                          void* stream) {
  return swiglu_impl(h, m_indices, masked_m, q, sf, nullptr, nullptr, rows, inter, num_groups, ld_h, ld_sf, 0, stream,
                     true);
}

int dg_swiglu_bwd(const uint8_t* hq, const float* hsf, const uint16_t* dact, const int32_t* m_indices, uint8_t* dq,
                  float* dsf, uint8_t* dqt, float* dsft, uint8_t* aqt, float* asft, int m_total, int inter,
                  int64_t ld_hsf, int64_t ld_dact, int64_t ld_dsf, int64_t ld_dsft, int64_t ld_asft, void* stream) {
  DG_TRY(check_layout(m_total, 1));
  if (m_total % 128) return fail(DG_ERR_UNSUPPORTED_SHAPE, "m_total=%d is not a multiple of 128", m_total);
  DG_TRY(check_cols("inter", inter, 128));
  if (inter > kMaxCols / 2) return fail(DG_ERR_UNSUPPORTED_SHAPE, "inter=%d is larger than %d", inter, kMaxCols / 2);
  DG_TRY(check_tiles(m_total, inter, false));
  if (!aqt != !asft) return fail(DG_ERR_INVALID_VALUE, "aqt and asft go together");
  DG_TRY(check_ld("ld_hsf", ld_hsf, m_total, 4, inter / 64, 4));
  DG_TRY(check_ld("ld_dact", ld_dact, inter, 8, m_total, 2));
  DG_TRY(check_ld("ld_dsf", ld_dsf, m_total, 4, inter / 64, 4));
  DG_TRY(check_ld("ld_dsft", ld_dsft, 2 * (int64_t)inter, 4, m_total / 128, 4));
  if (aqt) DG_TRY(check_ld("ld_asft", ld_asft, inter, 4, m_total / 128, 4));
  if (m_total == 0 || inter == 0) return ok();
  if (!hq || !hsf || !dact || !dq || !dsf || !dqt || !dsft) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(hq) || !aligned16(hsf) || !aligned16(dact) || !aligned16(dq) || !aligned16(dsf) || !aligned16(dqt) ||
      !aligned16(dsft) || !aligned16(aqt) || !aligned16(asft) || !aligned(m_indices, 4))
    return fail(DG_ERR_MISALIGNED, "data pointers must be 16-byte aligned, m_indices 4-byte aligned");
  const dg::SwigluBwdParams p{hq,  hsf,  dact,    m_indices, dq,     dsf,     dqt,    dsft,    aqt,
                              asft, m_total, inter, ld_hsf,    ld_dact, ld_dsf, ld_dsft, ld_asft};
  return launched(dg::launch_swiglu_bwd(p, static_cast<hipStream_t>(stream)), "swiglu_bwd");
}

int dg_requant_t(const uint8_t* q, const float* sf, const int32_t* m_indices, uint8_t* qt, float* sft, int rows,
                 int cols, int64_t ld_sf, int64_t ld_sft, void* stream) {
  DG_TRY(check_layout(rows, 1));
  if (rows % 128) return fail(DG_ERR_UNSUPPORTED_SHAPE, "rows=%d is not a multiple of 128", rows);
  DG_TRY(check_cols("cols", cols, 128));
  DG_TRY(check_tiles(rows, cols, true));
  DG_TRY(check_ld("ld_sf", ld_sf, rows, 4, cols / 128, 4));
  DG_TRY(check_ld("ld_sft", ld_sft, cols, 4, rows / 128, 4));
  if (rows == 0 || cols == 0) return ok();
  if (!q || !sf || !qt || !sft) return fail(DG_ERR_INVALID_VALUE, "null pointer argument");
  if (!aligned16(q) || !aligned16(sf) || !aligned16(qt) || !aligned16(sft) || !aligned(m_indices, 4))
    return fail(DG_ERR_MISALIGNED, "data pointers must be 16-byte aligned, m_indices 4-byte aligned");
  const dg::RequantParams p{q, sf, m_indices, qt, sft, rows, cols, ld_sf, ld_sft};
  return launched(dg::launch_requant_t(p, static_cast<hipStream_t>(stream)), "requant_t");
}

}  // extern "C"
