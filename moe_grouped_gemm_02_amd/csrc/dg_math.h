// Elementary functions of the mixture-of-experts kernels, and reductions that
// stay in the registers of a wave.
#pragma once

#include <utility>

#include "dg_device.h"
#include "dg_moe_internal.h"

namespace dg {

// 1 / d for normal d, within about half an ulp: the hardware's (1 ulp) and one
// Newton step.
__device__ __forceinline__ float reciprocal(float d) {
  const float y = __builtin_amdgcn_rcpf(d);
  return fmaf(fmaf(-d, y, 1.0f), y, y);
}

// exp(v) for v in [-150, 80] (others as the nearer end; not for NaN): 2^k 2^f
// with k the integer next to v log2(e), so that f carries none of the rounding
// of that product and results below the normal range come out rounded, not as
// zero.
__device__ __forceinline__ float exp_to_80(float v) {
  v = __builtin_amdgcn_fmed3f(v, -150.0f, 80.0f);
  const float k = __builtin_rintf(v * 1.44269504088896340736f);
  const float f = fmaf(v, 1.44269504088896340736f, -k);
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(f), (int)k);
}

// sigmoid(v) = e^v / (1 + e^v): the e^v in front keeps its relative accuracy
// for large negative v.
struct Sigmoid {
  float e, n, sig;  // e^v, 1 / (1 + e^v), their product
};
__device__ __forceinline__ Sigmoid sigmoid(float v) {
  const float e = exp_to_80(v);
  const float n = reciprocal(1.0f + e);
  return {e, n, e * n};
}

// e / d for e below 2^31 (see Divisor).
__device__ __forceinline__ uint32_t divided(uint32_t e, Divisor d) {
  return d.mul ? __umulhi(e, d.mul) >> d.shift : e;
}

// Between a lane's write to shared memory and another lane of the same wave
// reading it: the hardware keeps a wave's accesses in order, this keeps the
// compiler from moving or forwarding them.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Stores of results larger than the L2s, which nothing reads back through them:
// marked as streaming they leave the cached inputs alone (calls of 32768 x 7168:
// plan and dispatch 117 us, against 128 with plain stores; requantised transpose
// 83.6 and 91.5, combine gradient 252 and 274; gated unit of 32768 x 2048 79 and
// 81.7).
__device__ __forceinline__ void store_streaming(void* p, uint4 v) {
  __builtin_nontemporal_store(v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w}, static_cast<v4i*>(p));
}
__device__ __forceinline__ void store_streaming(void* p, uint2 v) {
  typedef int v2i __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(v2i{(int)v.x, (int)v.y}, static_cast<v2i*>(p));
}
// Short results stay in the L2s for the kernel that takes them next.
template <bool STREAMING>
__device__ __forceinline__ void store(void* p, uint4 v) {
  if constexpr (STREAMING) store_streaming(p, v);
  else *static_cast<uint4*>(p) = v;
}
// Loads of values that are used once (combine of 32110 rows x 7168: 95 us, against
// 107.7 with plain loads; requantised transpose 83.6 and 86.5, gated unit's
// backward 151 and 158).
__device__ __forceinline__ uint4 load_streaming4(const void* p) {
  const v4i v = __builtin_nontemporal_load(static_cast<const v4i*>(p));
  return make_uint4((uint32_t)v.x, (uint32_t)v.y, (uint32_t)v.z, (uint32_t)v.w);
}
__device__ __forceinline__ uint2 load_streaming2(const void* p) {
  typedef int v2i __attribute__((ext_vector_type(2)));
  const v2i v = __builtin_nontemporal_load(static_cast<const v2i*>(p));
  return make_uint2((uint32_t)v.x, (uint32_t)v.y);
}

// f(0) .. f(N - 1) with the index as a type, for what must be a constant.
template <int... I, typename F>
__device__ __forceinline__ void for_each_index(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void for_each_index(F&& f) {
  for_each_index(std::make_integer_sequence<int, N>{}, f);
}

// v of the lane that CTRL names, inside a row of 16 lanes or from one row to the
// next; 0 where that lane does not exist.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E;                  // quad_perm
constexpr int kHalfMirror = 0x141, kRowMirror = 0x140;     // the other quad of 8 lanes, the other half of 16
constexpr int kRowLane0 = 0x150;                           // + n: lane n of the row, to all of it
constexpr int kBroadcast15 = 0x142, kBroadcast31 = 0x143;  // a row's last lane to the next row, lane 31 to rows 2, 3

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(lane_value(__float_as_uint(v), lane));
}

// Order of a float as an unsigned number: larger value, larger number, -0 like
// +0; 0 for -inf and NaN.  (Maxima of unsigned numbers take a row operation as
// an operand, without the quieting of NaN that float maxima bring.)
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t o = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
  return v > -INFINITY ? o : 0u;
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Over the 64 lanes of the wave, as a uniform value.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = umax(v, dpp<kXor1>(v));
  v = umax(v, dpp<kXor2>(v));
  v = umax(v, dpp<kHalfMirror>(v));
  v = umax(v, dpp<kRowMirror>(v));
  v = umax(v, dpp<kBroadcast15>(v));
  v = umax(v, dpp<kBroadcast31>(v));
  return lane_value(v, 63);
}
// Over the 16 lanes of a row, in each of them.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  return v + dpp<kRowMirror>(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

}  // namespace dg
