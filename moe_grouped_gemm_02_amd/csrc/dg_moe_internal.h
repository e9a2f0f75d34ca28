// Internal host/device interface of the mixture-of-experts operators
// (dg_moe.h): what dg_moe_api.hip has checked and the kernels rely on.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;
constexpr int kMaxExpertGroups = 64;
constexpr int kMaxLocalExperts = 1024;

// Division of numbers below 2^31 by a constant 1 <= d < 2^31: e / d is e for
// d = 1 and otherwise (e * mul >> 32) >> shift, with mul = ceil(2^(31 + l) / d),
// 2^l the power of two at or above d, and shift = l - 1: mul / 2^(31 + l) is above
// 1 / d by less than 2^-(31 + l), which e < 2^31 times it cannot carry past the
// next quotient.
struct Divisor {
  uint32_t mul, shift;  // mul 0: d = 1
};
inline Divisor divisor(uint32_t d) {
  if (d <= 1) return {0, 0};
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), l - 1};
}

// A launch of 2^32 threads or more along one dimension of its grid is not made, or
// loses those past 2^32 without an error: workgroups of up to 256 threads that are
// counted by tokens are spread over two dimensions, x first.
struct GridXY {
  unsigned x, y;
};
inline GridXY spread(int64_t workgroups) {
  constexpr int64_t kMost = (int64_t)1 << 23;
  return workgroups <= kMost ? GridXY{(unsigned)workgroups, 1u} : GridXY{(unsigned)kMost, (unsigned)((workgroups + kMost - 1) / kMost)};
}

struct RouteParams {
  const void* logits;  // [tokens][ld], fp32 or bf16
  const float* bias;   // null: none
  int32_t* ids;        // backward: read
  float* weights;
  const float* dweights;
  void* dlogits;
  int tokens, experts, topk;
  int64_t ld, ld_d;
  int sigmoid;  // 0: softmax
  int groups, topk_groups, group_top;
  // Set by the launch: experts of a group, log2 of its lanes, whether those hold its experts.
  int per_group, group_shift, group_whole;
  Divisor by_group;
  int renormalize;
  float scale;
};
hipError_t launch_route(const RouteParams& p, bool bf16, hipStream_t stream);
hipError_t launch_route_bwd(const RouteParams& p, bool bf16, hipStream_t stream);

struct PlanParams {
  const int32_t* ids;
  int32_t* rows;
  int32_t* src;
  int32_t* m_indices;  // contiguous only
  int32_t* k_offsets;  // contiguous only
  int32_t* masked_m;   // masked only
  int32_t* hist;       // [blocks + 1][groups] counts
  int blocks;          // of 1024 entries (set by the launch)
  int scanned;         // whether hist holds sums over the blocks before (set by the launch)
  int entries;         // tokens * topk
  int first, groups;
  int masked, m_max;   // masked layout and its rows per group
  int layout_rows;
  Divisor by_m_max;  // masked only
};
size_t plan_workspace_bytes(int64_t entries, int groups);
hipError_t launch_plan(const PlanParams& p, hipStream_t stream);

struct DispatchParams {
  const uint16_t* x;
  const int32_t* src;
  uint8_t* q;
  void* sf;
  int tokens, topk, cols, rows, groups;
  int64_t ld_x, ld_sf;
  Divisor by_topk, by_rows;
};
hipError_t launch_dispatch(const DispatchParams& p, bool pow2, hipStream_t stream);

struct CombineParams {
  const uint16_t* d;
  const int32_t* rows;
  const float* weights;  // null: ones
  uint16_t* y;
  int tokens, topk, cols, total_rows;
  int64_t ld_d, ld_y;
};
hipError_t launch_combine(const CombineParams& p, hipStream_t stream);

struct CombineBwdParams {
  const uint16_t* dy;
  const uint16_t* d;
  const int32_t* src;
  const int32_t* rows;
  const float* weights;
  uint8_t* dq;
  float* dsf;
  uint8_t* dqt;  // null: no transposed codes
  float* dsft;
  float* dweights;
  float* dots;  // [cols / 128][m_total] partial sums of the weights' gradient
  int tokens, topk, cols, m_total;
  int64_t ld_dy, ld_d, ld_dsf, ld_dsft;
  Divisor by_topk;
};
hipError_t launch_combine_bwd(const CombineBwdParams& p, hipStream_t stream);

struct SwigluParams {
  const uint16_t* h;
  const int32_t* m_indices;  // at most one of the two is given
  const int32_t* masked_m;
  uint8_t* q;
  void* sf;
  uint8_t* hq;  // null: no checkpoint
  float* hsf;
  int rows, inter, groups;
  int64_t ld_h, ld_sf, ld_hsf;
};
hipError_t launch_swiglu_quant(const SwigluParams& p, bool pow2, hipStream_t stream);

struct SwigluBwdParams {
  const uint8_t* hq;
  const float* hsf;
  const uint16_t* dact;
  const int32_t* m_indices;  // null: every row in use
  uint8_t* dq;
  float* dsf;
  uint8_t* dqt;
  float* dsft;
  uint8_t* aqt;  // null: not wanted
  float* asft;
  int m_total, inter;
  int64_t ld_hsf, ld_dact, ld_dsf, ld_dsft, ld_asft;
};
hipError_t launch_swiglu_bwd(const SwigluBwdParams& p, hipStream_t stream);

struct RequantParams {
  const uint8_t* q;
  const float* sf;
  const int32_t* m_indices;
  uint8_t* qt;
  float* sft;
  int rows, cols;
  int64_t ld_sf, ld_sft;
};
hipError_t launch_requant_t(const RequantParams& p, hipStream_t stream);

}  // namespace dg
