// Expert routing for gfx950: scores, grouped top-k and weights, and the
// gradient of the weights with respect to the logits.
//
// One wave holds one token: expert e sits in lane e % 64, register e / 64, so
// a load of 64 consecutive logits is coalesced for any row stride and any
// number of experts, and every reduction stays inside the wave.

#include "dg_device.h"
#include "dg_moe_internal.h"

namespace dg {
namespace {

constexpr int kWaves = 4;  // tokens of a workgroup

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return bf16_bits_to_f32(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  *p = (uint16_t)(v == v ? f32_to_bf16_rne(v) : 0x7FC0u);
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Order of a float as an unsigned number: larger value, larger number, -0
// like +0; 0 for values that are never chosen (-inf and NaN).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  const uint32_t o = (u >> 31) ? ~u : (u | 0x80000000u);
  return v > -INFINITY ? o : 0u;
}

// Scores of the wave's token: lane l holds experts l + 64 i.
template <int V>
__device__ __forceinline__ void scores(const float (&x)[V], float (&s)[V], int experts, int lane, bool sigmoid) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = 1.0f / (1.0f + expf(-x[i]));
    return;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) top = fmaxf(top, x[i]);
  top = wave_max(top);
  if (top == -INFINITY) top = 0.0f;  // nothing but masked experts: every score is 0
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s[i] = lane + 64 * i < experts ? expf(x[i] - top) : 0.0f;
    total += s[i];
  }
  total = wave_sum(total);
  if (total == 0.0f) total = 1.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] /= total;
}

template <typename T, int V>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteParams p) {
  __shared__ float keys[kWaves][64 * V];
  __shared__ uint32_t gkeys[kWaves][kMaxExpertGroups];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float x[V], s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.experts ? load_logit(row + e) : -INFINITY;
  }
  scores<V>(x, s, p.experts, lane, p.sigmoid != 0);

  uint32_t key[V];  // 0: cannot be chosen
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    const float biased = p.bias && e < p.experts ? s[i] + p.bias[e] : s[i];
    key[i] = x[i] > -INFINITY ? order_of(p.bias ? biased : x[i]) : 0u;
    if (p.groups > 1) keys[wave][e] = x[i] > -INFINITY ? biased : -INFINITY;
  }

  if (p.groups > 1) {
    // Lane g scores group g; a group stays where fewer than topk_groups others
    // come before it.
    const int per = p.experts / p.groups;
    __builtin_amdgcn_wave_barrier();
    uint32_t mine = 0;
    if (lane < p.groups) {
      float a = -INFINITY, b = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const float v = keys[wave][lane * per + i];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      if (p.group_top == 2 && b > -INFINITY) a += b;
      mine = order_of(a);
      gkeys[wave][lane] = mine;
    }
    __builtin_amdgcn_wave_barrier();
    int before = 0;
    if (lane < p.groups)
      for (int g = 0; g < p.groups; ++g) {
        const uint32_t other = gkeys[wave][g];
        before += other > mine || (other == mine && g < lane);
      }
    const uint64_t kept = __ballot(lane < p.groups && before < p.topk_groups && mine != 0u);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane + 64 * i;
      if (e < p.experts && !((kept >> (e / per)) & 1)) key[i] = 0u;
    }
  }

  // topk rounds of a maximum over (key, lowest expert).
  int my_id = -1;
  float my_score = 0.0f, total = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint64_t c = key[i] ? ((uint64_t)key[i] << 32) | (uint32_t)~(lane + 64 * i) : 0ull;
      best = c > best ? c : best;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint64_t other = __shfl_xor((unsigned long long)best, off, 64);
      best = other > best ? other : best;
    }
    if (best == 0) break;  // the same in every lane
    const int e = (int)~(uint32_t)best;
    float sc = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == lane + 64 * i) {
        sc = s[i];
        key[i] = 0u;
      }
    sc = __shfl(sc, e & 63, 64);
    total += sc;
    if (lane == j) {
      my_id = e;
      my_score = sc;
    }
  }
  if (lane < p.topk) {
    float w = p.scale * my_score;
    if (p.renormalize) w = total > 0.0f || total != total ? w / total : 0.0f;
    p.ids[t * p.topk + lane] = my_id;
    p.weights[t * p.topk + lane] = w;
  }
}

template <typename T, int V>
__global__ __launch_bounds__(64 * kWaves) void route_bwd_kernel(RouteParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kWaves + wave;
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float x[V], s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    x[i] = e < p.experts ? load_logit(row + e) : -INFINITY;
  }
  scores<V>(x, s, p.experts, lane, p.sigmoid != 0);

  int id = -1;
  float dw = 0.0f;
  if (lane < p.topk) {
    id = p.ids[t * p.topk + lane];
    if (id < 0 || id >= p.experts) id = -1;
    dw = id >= 0 ? p.dweights[t * p.topk + lane] : 0.0f;
  }
  // Lane j takes the score of its expert.
  float sel = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    const int e = __shfl(id, j, 64);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i == (e >> 6)) v = s[i];
    v = __shfl(v, e & 63, 64);
    if (lane == j && e >= 0) sel = v;
  }
  float g = p.scale * dw;
  if (p.renormalize) {
    const float total = wave_sum(sel);
    if (total != 0.0f) g = (g - wave_sum(g * sel) / total) / total;
  }
  if (id < 0) g = 0.0f;
  float full[V];
#pragma unroll
  for (int i = 0; i < V; ++i) full[i] = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    const int e = __shfl(id, j, 64);
    const float v = __shfl(g, j, 64);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == lane + 64 * i) full[i] = v;
  }
  const float mean = p.sigmoid ? 0.0f : wave_sum(g * sel);
  T* out = static_cast<T*>(p.dlogits) + t * p.ld_d;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    const float dx = p.sigmoid ? full[i] * s[i] * (1.0f - s[i]) : s[i] * (full[i] - mean);
    if (e < p.experts) store_logit(out + e, dx);
  }
}

template <typename T>
hipError_t pick(const RouteParams& p, bool bwd, hipStream_t stream) {
  const dim3 grid((unsigned)(((int64_t)p.tokens + kWaves - 1) / kWaves)), block(64 * kWaves);
  auto go = [&](auto fwd, auto grad) {
    if (bwd) hipLaunchKernelGGL(grad, grid, block, 0, stream, p);
    else hipLaunchKernelGGL(fwd, grid, block, 0, stream, p);
  };
  const int v = (p.experts + 63) / 64;
  if (v <= 1) go(route_kernel<T, 1>, route_bwd_kernel<T, 1>);
  else if (v <= 2) go(route_kernel<T, 2>, route_bwd_kernel<T, 2>);
  else if (v <= 4) go(route_kernel<T, 4>, route_bwd_kernel<T, 4>);
  else if (v <= 8) go(route_kernel<T, 8>, route_bwd_kernel<T, 8>);
  else go(route_kernel<T, 16>, route_bwd_kernel<T, 16>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams& p, bool bf16, hipStream_t stream) {
  return bf16 ? pick<uint16_t>(p, false, stream) : pick<float>(p, false, stream);
}

hipError_t launch_route_bwd(const RouteParams& p, bool bf16, hipStream_t stream) {
  return bf16 ? pick<uint16_t>(p, true, stream) : pick<float>(p, true, stream);
}

}  // namespace dg
