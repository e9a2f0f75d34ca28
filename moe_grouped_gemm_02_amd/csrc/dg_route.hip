// Expert routing for gfx950: scores, grouped top-k and weights, and the
// gradient of the weights with respect to the logits.
//
// One wave holds one token, lane l experts V l .. V l + V - 1 with V the power
// of two that covers all experts, so that a row is one vector load a lane, the
// order of lanes and registers is the order of the experts (ties), and every
// reduction stays in registers (row operations and readlane, no shared memory).
// A token is read once.  What bounds the choice is the issue of vector
// instructions, 376 a token of 256 experts in groups (17 a round of the top-k, 11
// a sigmoid): 32768 tokens in 21.6 us, 59 us with shuffles for the row operations
// and 64-bit keys.  The gradient is bound by memory and by its start: it writes 34
// MB and reads the lines of the chosen logits in 10.2 us.

#include "dg_math.h"
#include "dg_moe_internal.h"
#include "dg_route_rows.h"

namespace dg {
namespace {

constexpr int kWaves = 4;  // tokens of a workgroup

// 1 / (1 + e^-x) within 2 ulp: the hardware's reciprocal without its Newton
// step.
__device__ __forceinline__ float score_sigmoid(float x) {
  const float e = exp_to_80(x);
  return e * __builtin_amdgcn_rcpf(1.0f + e);
}

// Scores of the wave's token.
template <int V>
__device__ __forceinline__ void scores(const float (&x)[V], float (&s)[V], bool sigmoid_scores) {
  if (sigmoid_scores) {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = score_sigmoid(x[i]);
    return;
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) most = umax(most, order_of(x[i]));
  most = wave_max(most);
  const float top = most ? of_order(most) : 0.0f;  // nothing but masked experts: every score is 0
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float d = x[i] - top;
    const float e = exp_to_80(d);
    s[i] = d == d ? e : d;
    total += s[i];
  }
  total = wave_sum(total);
  const float inv = total == 0.0f ? 0.0f : reciprocal(total);
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] *= inv;
}

// The two largest of two sorted pairs.
__device__ __forceinline__ void merge_top2(uint32_t& a, uint32_t& b, uint32_t a2, uint32_t b2) {
  b = umax(umin(a, a2), umax(b, b2));
  a = umax(a, a2);
}

// BIAS, GROUPS: whether the call has them.
template <bool VEC, typename T, int V, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteParams p) {
  __shared__ float lds[kWaves][64 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + wave;
  if (t >= p.tokens) return;
  float x[V], s[V], bias[V];
  uint32_t key[V];  // 0: cannot be chosen
  int idx[V];
  load_row<VEC>(static_cast<const T*>(p.logits) + t * p.ld, p.experts, lane, lds[wave], x);
  if constexpr (BIAS) load_row<VEC>(p.bias, p.experts, lane, lds[wave], bias);
  scores<V>(x, s, p.sigmoid != 0);
#pragma unroll
  for (int i = 0; i < V; ++i) lds[wave][lane * V + i] = s[i];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (BIAS) s[i] += bias[i];
    const uint32_t k = order_of(BIAS || GROUPS ? s[i] : x[i]);
    key[i] = (!BIAS && !GROUPS) || x[i] > -INFINITY ? k : 0u;
    idx[i] = i;
  }

  if constexpr (GROUPS) {
    // Two largest keys of each group by its 2^group_shift lanes: those that hold
    // the group's experts where that many lanes hold them and no others, otherwise
    // an equal share of the wave, which looks at them in shared memory (256 experts
    // in 8 groups, 32768 tokens: 21.6 us, and 24.2 by shared memory).
    uint32_t a = 0, b = 0;
    const int lanes = 1 << p.group_shift, sub = lane & (lanes - 1);
    const int mine = lane >> p.group_shift;  // the lane's group
    if (p.group_whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) merge_top2(a, b, key[i], 0u);
    } else {
      __shared__ uint32_t keys[kWaves][64 * V];
#pragma unroll
      for (int i = 0; i < V; ++i) keys[wave][lane * V + i] = key[i];
      wave_fence();
      if (mine < p.groups)
        for (int i = sub; i < p.per_group; i += lanes) merge_top2(a, b, keys[wave][mine * p.per_group + i], 0u);
    }
    if (p.group_shift > 0) merge_top2(a, b, dpp<kXor1>(a), dpp<kXor1>(b));
    if (p.group_shift > 1) merge_top2(a, b, dpp<kXor2>(a), dpp<kXor2>(b));
    if (p.group_shift > 2) merge_top2(a, b, dpp<kHalfMirror>(a), dpp<kHalfMirror>(b));
    if (p.group_shift > 3) merge_top2(a, b, dpp<kRowMirror>(a), dpp<kRowMirror>(b));
    if (p.group_shift > 4) merge_top2(a, b, __shfl_xor(a, 16, 64), __shfl_xor(b, 16, 64));
    const uint32_t score = a == 0u ? 0u : p.group_top == 2 && b != 0u ? order_of(of_order(a) + of_order(b)) : a;
    int before = 0;  // groups that come first
    if (p.groups <= lanes) {
      // Each lane of a group looks at one other group (23.1 us with the loop below).
      const uint32_t other = (uint32_t)__shfl((int)score, sub << p.group_shift, 64);
      const bool first = sub < p.groups && (other > score || (other == score && sub < mine));
      before = __popcll((__ballot(first) >> (lane - sub)) & ((1ull << lanes) - 1ull));
    } else {
      for (int g = 0; g < p.groups; ++g) {
        const uint32_t other = lane_value(score, g << p.group_shift);
        before += other > score || (other == score && g < mine);
      }
    }
    const bool stays = before < p.topk_groups && mine < p.groups && score != 0u;
    const uint64_t kept = __ballot(stays);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bool in = stays;
      if (!p.group_whole) {
        const int g = (int)divided(lane * V + i, p.by_group);
        in = g < p.groups && ((kept >> (g << p.group_shift)) & 1);
      }
      // Without a bias the groups go by scores, the experts by their logits.
      const uint32_t k = BIAS ? key[i] : order_of(x[i]);
      key[i] = in ? k : 0u;
    }
  }

  // Largest first within the lane, equal keys in order: as many passes as
  // experts are wanted.
#pragma unroll
  for (int pass = 0; pass < V - 1; ++pass) {
    if (pass < p.topk) {
#pragma unroll
      for (int i = V - 2; i >= pass; --i) {
        const uint32_t a = key[i], b = key[i + 1];
        const int ia = idx[i], ib = idx[i + 1];
        const bool swap = b > a;
        key[i] = umax(a, b), key[i + 1] = umin(a, b);
        idx[i] = swap ? ib : ia, idx[i + 1] = swap ? ia : ib;
      }
    }
  }
  // Each round takes the largest head of all lanes, the lowest lane among
  // equals, and moves that lane's list up; the order of its registers is kept as
  // four bits each.
  uint64_t order = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) order |= (uint64_t)idx[i] << (4 * i);
  int id = -1;
  for (int j = 0; j < p.topk; ++j) {
    const uint32_t best = wave_max(key[0]);
    if (best == 0u) break;
    const uint64_t heads = __ballot(key[0] == best);
    const int from = __builtin_ctzll(heads);
    const int e = from * V + (__builtin_amdgcn_readlane((int)order, from) & 15);
    id = __builtin_amdgcn_inverse_ballot_w64(1ull << j) ? e : id;
    const bool pop = __builtin_amdgcn_inverse_ballot_w64(heads & -heads);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t same = key[i], next = i + 1 < V ? key[i + 1] : 0u;
      key[i] = pop ? next : same;
    }
    if (V > 8) order = pop ? order >> 4 : order;
    else order = pop ? (uint32_t)order >> 4 : (uint32_t)order;
  }
  wave_fence();
  float w = id >= 0 ? lds[wave][id] : 0.0f;
  if (p.renormalize) {
    const float total = wave_sum(w);
    w = total > 0.0f || total != total ? w / total : 0.0f;
  }
  if (lane < p.topk) {
    p.ids[t * p.topk + lane] = id;
    p.weights[t * p.topk + lane] = p.scale * w;
  }
}

// The sigmoid's gradient touches the chosen experts alone and reads only their
// logits; the softmax's needs the row.  The row of the outputs is put together
// in shared memory.
template <bool VEC, typename T, int V, bool SIGMOID>
__global__ __launch_bounds__(64 * kWaves) void route_bwd_kernel(RouteParams p) {
  __shared__ float lds[kWaves][64 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kWaves + wave;
  if (t >= p.tokens) return;
  const T* row = static_cast<const T*>(p.logits) + t * p.ld;
  float* mine = lds[wave] + lane * V;
  int id = lane < p.topk ? p.ids[t * p.topk + lane] : -1;
  if (id >= p.experts) id = -1;
  const float dw = id >= 0 ? p.dweights[t * p.topk + lane] : 0.0f;
  float x[V], s[V], sel = 0.0f, rest = 0.0f;
  if constexpr (SIGMOID) {
    if (id >= 0) both_sigmoids(widen(row[id]), sel, rest);
  } else {
    load_row<VEC>(row, p.experts, lane, lds[wave], x);
    scores<V>(x, s, false);
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] = s[i];
    wave_fence();
    if (id >= 0) sel = lds[wave][id];
  }
  // g: the scores' gradient, or, renormalised, that of the scores' logarithms:
  // s / S comes first, since the chosen scores' sum S may be so small that a
  // quotient by it leaves float32.
  float g = p.scale * dw;
  if (p.renormalize) {
    const float total = wave_sum(sel);
    const float r = total != 0.0f ? sel / total : 0.0f;
    g = p.scale * r * (dw - wave_sum(dw * r));
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < V; ++i) mine[i] = 0.0f;
  wave_fence();
  if (id >= 0) lds[wave][id] = !SIGMOID ? g : (p.renormalize ? g : g * sel) * rest;
  wave_fence();
  // Renormalised softmax weights depend on the chosen logits alone: 0 at the others.
  const bool chosen_alone = SIGMOID || p.renormalize;
  const float mean = chosen_alone ? 0.0f : wave_sum(g * sel);
  T* to = static_cast<T*>(p.dlogits) + t * p.ld_d;
  float out[V];
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = chosen_alone ? mine[i] : s[i] * (mine[i] - mean);
  if constexpr (VEC) {
    Pack<T, V> pack;
#pragma unroll
    for (int i = 0; i < V; ++i) narrow(pack.v[i], out[i]);
    if (lane * V < p.experts) *reinterpret_cast<Pack<T, V>*>(to + lane * V) = pack;
  } else {
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) mine[i] = out[i];
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * 64 + lane;
      if (e < p.experts) narrow(to[e], lds[wave][e]);
    }
  }
}

template <bool VEC, typename T, int V>
void go(const RouteParams& p, bool bwd, hipStream_t stream) {
  const GridXY by_token = spread(((int64_t)p.tokens + kWaves - 1) / kWaves);
  const dim3 grid(by_token.x, by_token.y), block(64 * kWaves);
  if (!bwd) {
    if (p.bias && p.groups > 1) hipLaunchKernelGGL((route_kernel<VEC, T, V, true, true>), grid, block, 0, stream, p);
    else if (p.bias) hipLaunchKernelGGL((route_kernel<VEC, T, V, true, false>), grid, block, 0, stream, p);
    else if (p.groups > 1) hipLaunchKernelGGL((route_kernel<VEC, T, V, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((route_kernel<VEC, T, V, false, false>), grid, block, 0, stream, p);
  } else if (p.sigmoid) hipLaunchKernelGGL((route_bwd_kernel<VEC, T, V, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((route_bwd_kernel<VEC, T, V, false>), grid, block, 0, stream, p);
}

// Whole vectors: no ragged last lane, and every row starts on a vector (32768 rows
// of 256: 21.4 us, and 22.8 through shared memory).
template <typename T, int V>
void go(RouteParams p, bool bwd, hipStream_t stream) {
  if (!bwd && p.groups > 1) {
    p.per_group = p.experts / p.groups;
    p.by_group = divisor(p.per_group);
    p.group_shift = 6;
    while (p.groups > 64 >> p.group_shift) --p.group_shift;
    for (int shift = 0; shift < 6; ++shift)
      if (p.per_group == V << shift) p.group_shift = shift, p.group_whole = 1;
  }
  constexpr size_t kAlign = alignof(Pack<T, V>);
  auto fits = [&](const void* at, int64_t ld) {
    return reinterpret_cast<uintptr_t>(at) % kAlign == 0 && ld * sizeof(T) % kAlign == 0;
  };
  const bool vec = p.experts % V == 0 && fits(p.logits, p.ld) && (!bwd || fits(p.dlogits, p.ld_d)) &&
                   reinterpret_cast<uintptr_t>(p.bias) % alignof(Pack<float, V>) == 0;
  if (vec) go<true, T, V>(p, bwd, stream);
  else go<false, T, V>(p, bwd, stream);
}

template <typename T>
hipError_t pick(const RouteParams& p, bool bwd, hipStream_t stream) {
  const int v = (p.experts + 63) / 64;
  if (v <= 1) go<T, 1>(p, bwd, stream);
  else if (v <= 2) go<T, 2>(p, bwd, stream);
  else if (v <= 4) go<T, 4>(p, bwd, stream);
  else if (v <= 8) go<T, 8>(p, bwd, stream);
  else go<T, 16>(p, bwd, stream);
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
