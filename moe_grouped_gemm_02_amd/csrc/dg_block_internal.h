// Internal host/device interface of the operators of dg_block.h: what
// dg_block_api.hip has checked and the kernels rely on.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dg {

constexpr int kMaxNormCols = 16384;

struct NormParams {
  const uint16_t* y;
  const uint16_t* h;         // null: no residual
  const float* gate;         // by gate_kind
  const float* post_weight;  // null: ones
  const float* weight;       // null: ones
  const float* bias;         // null: none
  uint16_t* r;               // null: not wanted, as the next two
  uint16_t* x;
  uint8_t* q;
  void* sf;
  int tokens, cols;
  int64_t ld_y, ld_h, ld_r, ld_x, ld_sf;
  int layer, post, gate_kind;
  float res_scale, eps;
};
hipError_t launch_block_norm(const NormParams& p, bool pow2, hipStream_t stream);

struct NormBwdParams {
  const uint16_t* dx;  // null: none
  const uint16_t* dr;  // null: none
  const uint16_t* r;
  const uint16_t* y;
  const float* gate;
  const float* post_weight;
  const float* weight;
  uint16_t* dy;
  uint16_t* dh;        // null: not wanted, as the next four
  float* dweight;
  float* dbias;
  float* dpost_weight;
  float* dgate;
  float* parts;        // [4][norm_bwd_parts(tokens, cols)][cols] partial sums
  int tokens, cols;
  int64_t ld_dx, ld_dr, ld_r, ld_y, ld_dy, ld_dh;
  int layer, post, gate_kind;
  float res_scale, eps;
};
int norm_bwd_parts(int tokens, int cols);
hipError_t launch_block_norm_bwd(const NormBwdParams& p, hipStream_t stream);

// Sums over the parts of up to four matrices [parts][cols] into vectors [cols]
// (null: none), in the order of the parts.  cols % 8 == 0.
struct ColumnSums {
  const float* from[4];
  float* to[4];
  int count, parts, cols;
};
hipError_t launch_column_sums(const ColumnSums& c, hipStream_t stream);

struct BalanceParams {
  const void* logits;  // [tokens][ld], fp32 or bf16
  const int32_t* ids;
  const int32_t* offsets;  // null: one sequence of all tokens
  int32_t* counts;         // backward: read
  int32_t* used;           // backward: read
  float* loss;
  const float* dloss;  // null: 1
  const void* add;     // null: none
  void* dlogits;
  // Workspace: partial sums of the shares and counts [slots][experts], tokens in
  // use [slots], parts of the loss and how many of them are there.
  float* share_parts;
  int32_t* count_parts;
  int32_t* used_parts;
  double* loss_parts;
  uint32_t* arrived;
  int tokens, experts, topk, seqs;
  int chunk;  // tokens of a workgroup (forward)
  int64_t ld, ld_add, ld_d;
  int sigmoid;
  float coef;
  double coef_mean, experts_per_choice;  // forward: coef / seqs, experts / topk
};
// Tokens of a forward workgroup, and the rows of its partial sums.
int balance_chunk(int tokens);
int64_t balance_slots(int tokens, int seqs);
int balance_loss_parts(int experts);
hipError_t launch_balance(const BalanceParams& p, bool bf16, hipStream_t stream);
hipError_t launch_balance_bwd(const BalanceParams& p, bool bf16, hipStream_t stream);

struct EpilogueBwdParams {
  const uint16_t* dd;
  const uint16_t* pre;
  uint8_t* dq;
  float* dsf;
  uint8_t* dqt;  // null: no transposed codes
  float* dsft;
  float* dbias;  // null: not wanted
  float* parts;  // [row tiles][cols] partial sums
  int rows, cols;
  int64_t ld_dd, ld_pre, ld_dsf, ld_dsft;
  int act;
};
hipError_t launch_epilogue_bwd(const EpilogueBwdParams& p, hipStream_t stream);

}  // namespace dg
