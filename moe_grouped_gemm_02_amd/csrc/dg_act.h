// Activation functions of a product's epilogue and their slopes, in float32,
// and the rounding of a pair of values to bf16.
#pragma once

#include <type_traits>

#include "dg_block.h"
#include "dg_math.h"
#include "dg_tile.h"

namespace dg {

// Two values rounded to bf16 (to nearest even, NaN quiet), the first one low.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{lo, hi}), v2b));
}

// The tanh form of the GELU is z / (1 + e^-t), t = 2 sqrt(2 / pi) (z + 0.044715 z^3):
// (1 + tanh(u)) / 2 is the sigmoid of 2 u, which keeps its relative accuracy
// for negative z.
constexpr float kGelu1 = 1.5957691216057308f, kGelu3 = 0.071354816272600247f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kGelu1Log2e = 2.302208198144325f, kGelu3Log2e = 0.1029432395800235f;  // t in powers of 2

// Values that are rounded to bf16 next: z / (1 + 2^-u) as z w (w / (1 + w^2)) with
// w = 2^(u / 2), by the hardware's 2^x and reciprocal, within 2^-21 and |u| 2^-23 of
// themselves.  Neither factor leaves the normal range before the result does: 2^-u alone
// would be infinite from u = -128 on, where SiLU(-89) = -2e-37 is still a bf16 number
// (GEMM of 4096 x 4096 x 7168 with GELU: 122.2 us, 121.4 with 2^-u; 128.1 with exp2f and a
// quotient).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  auto gated = [](float v, float half) {  // half: u / 2
    const float w = __builtin_amdgcn_exp2f(fminf(half, 60.0f));  // past that 1 / (1 + 2^-u) is 1
    return v * (w * __builtin_amdgcn_rcpf(fmaf(w, w, 1.0f))) * w;
  };
  if constexpr (ACT == DG_ACT_RELU) return z < 0.0f ? 0.0f : z;
  else if constexpr (ACT == DG_ACT_SILU) return gated(z, z * (0.5f * kLog2e));
  else if constexpr (ACT == DG_ACT_GELU_TANH) return gated(z, z * fmaf(0.5f * kGelu3Log2e, z * z, 0.5f * kGelu1Log2e));
  else return z;
}

// The slope of a NaN is NaN, that of an infinite z the limit, 0 or 1.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == DG_ACT_RELU) {
    return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
  } else if constexpr (ACT == DG_ACT_SILU) {
    const float slope = silu_slope(z, 1.0f, z, sigmoid(z));
    return z == z ? slope : z;  // the ranges that sigmoid() cuts take a NaN for a number
  } else if constexpr (ACT == DG_ACT_GELU_TANH) {
    // Up to +-10 t log2(e) lies in +-125.97, where the hardware's 2^x and its reciprocal are
    // in the normal range and z^2 is finite; past that the slope is 1 or below 2^-117.
    // log2(e) is part of the constants: two roundings of t, as without it, and none of a
    // product with it (16384 x 4096: 91.5 us, and 95.5 with the exponent split off before).
    const float v = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -10.0f), 10.0f), v2 = v * v;
    const float e = __builtin_amdgcn_exp2f(v * fmaf(kGelu3Log2e, v2, kGelu1Log2e));
    const float n = reciprocal(1.0f + e);  // 1 - sigmoid
    return e * n * fmaf(v * n, fmaf(3.0f * kGelu3, v2, kGelu1), 1.0f);
  } else {
    return 1.0f;
  }
}

// f with the activation as a type.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case DG_ACT_RELU: f(std::integral_constant<int, DG_ACT_RELU>{}); break;
    case DG_ACT_SILU: f(std::integral_constant<int, DG_ACT_SILU>{}); break;
    case DG_ACT_GELU_TANH: f(std::integral_constant<int, DG_ACT_GELU_TANH>{}); break;
    default: f(std::integral_constant<int, DG_ACT_NONE>{}); break;
  }
}

}  // namespace dg
