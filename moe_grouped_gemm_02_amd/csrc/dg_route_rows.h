// Rows of a router's logits in the registers of a wave: lane l holds experts
// V l .. V l + V - 1, with V the power of two that covers all experts.
#pragma once

#include "dg_math.h"

namespace dg {
namespace {

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ void narrow(float& to, float v) { to = v; }
__device__ __forceinline__ void narrow(uint16_t& to, float v) {
  to = (uint16_t)(v == v ? f32_to_bf16_rne(v) : 0x7FC0u);
}

// V consecutive elements as one access of up to 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
  T v[V];
};

// The lane's V logits, -inf past the last expert.  VEC: rows and their length
// allow whole vectors (decided on the host); otherwise the wave reads them in
// order and hands them out through its 64 V words of shared memory (32768 rows of
// 500: 41 us, 60 with each lane reading its own).  The two steps apart, for rows that
// are read ahead: fetch_row, and arrange_row on what it read.
template <bool VEC, typename T, int V>
__device__ __forceinline__ void fetch_row(const T* row, int experts, int lane, float (&x)[V]) {
  if constexpr (VEC) {
    const int e0 = lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = -INFINITY;
    if (e0 < experts) {
      const Pack<T, V> in = *reinterpret_cast<const Pack<T, V>*>(row + e0);
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = widen(in.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      x[i] = e < experts ? widen(row[e]) : -INFINITY;
    }
  }
}
template <bool VEC, int V>
__device__ __forceinline__ void arrange_row(int lane, float* lds, float (&x)[V]) {
  if constexpr (!VEC && V > 1) {
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) lds[i * 64 + lane] = x[i];
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = lds[lane * V + i];
  }
}
template <bool VEC, typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int experts, int lane, float* lds, float (&x)[V]) {
  fetch_row<VEC>(row, experts, lane, x);
  arrange_row<VEC>(lane, lds, x);
}

// s = 1 / (1 + e^-x) and 1 - s, each with its own relative accuracy: the smaller
// one is e^-|x| times the larger, not a difference from 1.
__device__ __forceinline__ void both_sigmoids(float x, float& s, float& rest) {
  const float e = x == x ? exp_to_80(-fabsf(x)) : x;
  const float large = reciprocal(1.0f + e), small = e * large;
  s = x < 0.0f ? small : large;
  rest = x < 0.0f ? large : small;
}

}  // namespace
}  // namespace dg
