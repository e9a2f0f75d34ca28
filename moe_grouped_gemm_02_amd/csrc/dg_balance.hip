// Load balance of a router over sequences for gfx950: the experts' counts and
// the loss in two launches, the gradient in one.
//
// A wave holds a token's logits, lane l experts V l .. V l + V - 1.  A workgroup
// has a chunk of consecutive tokens, finds the sequence of its first one and walks
// from sequence to sequence.  Forward it leaves, for every sequence that meets the
// chunk, a row of sums over their common tokens: chunk b and sequence s share row
// b + s (both only grow along the tokens, so no two pairs have the same), and a
// second launch adds the rows of each sequence in their order.  32768 tokens of 256
// fp32 experts: 8.5 + 6.6 us (13.4 + 6.5 with every score formed as the gradient's), and
// 20 for the gradient with one to add to, 101 MB at 5 TB/s.  Of bf16 logits, half of
// the bytes, 9.8 + 6.6 us and 16.2, with the vector units busy 56 and 75 % of the time:
// their scores take the same instructions.

#include "dg_block_internal.h"
#include "dg_math.h"
#include "dg_moe_internal.h"
#include "dg_route_rows.h"
#include "dg_turns.h"

namespace dg {
namespace {

// Sequence ends, brought into [0, tokens].
struct Sequences {
  const int32_t* offsets;
  int count, tokens;
  __device__ __forceinline__ int at(int s) const {
    if (!offsets) return s == 0 ? 0 : tokens;
    return min(max(offsets[s], 0), tokens);
  }
  // The first sequence that ends behind token t (count: none): the wave looks at 64
  // places at a time, each the last of an equal part of what is left.
  __device__ __forceinline__ int of(int t, int lane) const {
    int lo = 0, hi = count;
    while (lo < hi) {
      const int part = (hi - lo + 63) / 64;
      const int last = (int)min((int64_t)lo + (int64_t)(lane + 1) * part, (int64_t)hi) - 1;
      const uint64_t behind = __ballot(at(last + 1) > t);
      if (behind == 0) return hi;
      const int k = __builtin_ctzll(behind);
      hi = (int)lane_value((uint32_t)last, k);
      lo += k * part;
    }
    return hi;
  }
};

// f(s, from, to) for each sequence s with tokens in [t0, t1), and those; the same in
// every wave.  A wave holds the ends of 64 sequences at a time, so that the step from
// one sequence to the next reads no memory.  t grows with every turn whatever the
// offsets hold: the sequence that is found or taken ends behind it.
template <typename F>
__device__ __forceinline__ void for_sequences(const Sequences& q, int t0, int t1, int lane, F&& f) {
  int t = t0;
  for (int first = q.of(t, lane); first < q.count; first = q.of(t, lane)) {
    const int s = first + lane;
    const int end = s < q.count ? q.at(s + 1) : -1;
    t = max(t, q.at(first));
    while (t < t1) {
      const uint64_t behind = __ballot(end > t);
      if (behind == 0) break;
      const int k = __builtin_ctzll(behind);
      const int to = min((int)lane_value((uint32_t)end, k), t1);
      f(first + k, t, to);
      t = to;
    }
    if (t >= t1) return;
  }
}

// Shares p of the wave's token, and for sigmoid scores 1 minus the score (1 for
// softmax).  Scores are taken relative to the largest one where all are small, so
// that tokens whose scores leave float32 have shares like any other.  True where
// some logit is not -inf.
template <int V>
__device__ __forceinline__ bool shares(const float (&x)[V], float (&p)[V], float (&rest)[V], bool sigmoid_scores) {
  uint32_t most = 0;
  bool open = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    most = umax(most, order_of(x[i]));
    open |= !(x[i] == -INFINITY);
  }
  most = wave_max(most);
  const float top = most ? of_order(most) : 0.0f;
  float total = 0.0f;
  if (sigmoid_scores) {
#pragma unroll
    for (int i = 0; i < V; ++i) both_sigmoids(x[i], p[i], rest[i]);
    if (top < 0.0f) {  // s_e / s_max up to a factor that cancels: e^(x - top) (1 - s)
#pragma unroll
      for (int i = 0; i < V; ++i) p[i] = exp_to_80(x[i] - top) * rest[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) total += p[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = x[i] - top, e = exp_to_80(d);
      p[i] = d == d ? e : d;
      rest[i] = 1.0f;
      total += p[i];
    }
  }
  total = wave_sum(total);
  const float inv = total == 0.0f ? 0.0f : reciprocal(total);
#pragma unroll
  for (int i = 0; i < V; ++i) p[i] *= inv;
  return __ballot(open) != 0;
}

// Rows as they nearly always are: no NaN, the largest logit finite and, for sigmoid
// scores, one of them not negative, so that no score has to be taken relative to
// another one.  top: the largest logit (softmax).
template <int V>
__device__ __forceinline__ bool ordinary(const float (&x)[V], bool sigmoid_scores, float& top) {
  float most = x[0];
  bool nan = x[0] != x[0];
#pragma unroll
  for (int i = 1; i < V; ++i) most = fmaxf(most, x[i]);
#pragma unroll
  for (int i = 1; i < V; i += 2) nan |= __builtin_isunordered(x[i], x[i + 1 < V ? i + 1 : i]);
  if (__ballot(nan)) return false;
  if (sigmoid_scores) return __ballot(most >= 0.0f) != 0;
  const uint32_t all = wave_max(order_of(most));
  top = of_order(all);
  return all != 0 && top < INFINITY;
}

constexpr float kLog2e = 1.44269504088896340736f;

// What shares of an ordinary row are proportional to, for sums over tokens: the
// hardware's 2^x of the product as it was rounded, within |x| 2^-24 of the value, and
// 0 where that is below the normal range.
template <int V>
__device__ __forceinline__ float weights(const float (&x)[V], float top, bool sigmoid_scores, float (&p)[V]) {
  float total = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = sigmoid_scores ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x[i]))
                          : __builtin_amdgcn_exp2f(kLog2e * (x[i] - top));
    total += p[i];
  }
  return wave_sum(total);
}

// The same within 3 ulp, results below the normal range included, and that times
// the slope's factor: s (1 - s) is the same on both sides of 0.
template <int V>
__device__ __forceinline__ void slopes(const float (&x)[V], float top, bool sigmoid_scores, float (&p)[V], float (&g)[V]) {
  auto e_to = [](float v) {  // exp_to_80 of v <= 0 that is a number
    v = fmaxf(v, -150.0f);
    const float k = __builtin_rintf(v * kLog2e);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f(fmaf(v, kLog2e, -k)), (int)k);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (sigmoid_scores) {
      const float e = e_to(-fabsf(x[i])), large = __builtin_amdgcn_rcpf(1.0f + e), small = e * large;
      p[i] = x[i] < 0.0f ? small : large;
      g[i] = small * large;
    } else {
      p[i] = g[i] = e_to(x[i] - top);
    }
  }
}

// Workgroup: a chunk of tokens, its waves one token after another, the next one read
// ahead (four ahead measure the same, and take registers).  At most 256 chunks: few rows
// for the second launch to add (32768 x 256: 6.5 us there, against 12.6 with 1024
// chunks of 4 waves, which take as long here), one workgroup a CU, which reads its 131 KB at
// what a CU reaches.
constexpr int kSumWaves = 16, kMostChunks = 256;

template <bool VEC, typename T, int V>
__global__ __launch_bounds__(64 * kSumWaves) void balance_kernel(BalanceParams p) {
  __shared__ float sums[kSumWaves][64 * V];
  __shared__ int counts[64 * V];
  __shared__ int used[kSumWaves];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.arrived = 0;
  const Sequences seqs = {p.offsets, p.seqs, p.tokens};
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = t0 + p.chunk;
  for_sequences(seqs, (int)t0, (int)(t1 < p.tokens ? t1 : p.tokens), lane, [&](int s, int from, int to) {
    for (int e = threadIdx.x; e < p.experts; e += 64 * kSumWaves) counts[e] = 0;
    float sum[V] = {}, next[V];
    int here = 0, next_id = -1;
    auto fetch = [&](int t) {
      fetch_row<VEC>(static_cast<const T*>(p.logits) + (int64_t)t * p.ld, p.experts, lane, next);
      if (lane < p.topk) next_id = p.ids[(int64_t)t * p.topk + lane];
    };
    Turns<kSumWaves> turn(from, to, wave);
    if (turn.here()) fetch(turn.row());
    __syncthreads();
    for (; turn.here(); turn.next()) {
      float x[V], share[V], top = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = next[i];
      const int id = next_id;
      if (turn.has_next()) fetch(turn.next_row());
      arrange_row<VEC>(lane, sums[wave], x);
      float inv = 1.0f;
      if (ordinary<V>(x, p.sigmoid != 0, top)) {
        inv = reciprocal(p.sigmoid ? weights<V>(x, top, true, share) : weights<V>(x, top, false, share));
      } else {
        float rest[V];
        if (!shares<V>(x, share, rest, p.sigmoid != 0)) continue;
      }
      ++here;
      if ((uint32_t)id < (uint32_t)p.experts) atomicAdd(&counts[id], 1);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] = fmaf(share[i], inv, sum[i]);
    }
    wave_fence();
#pragma unroll
    for (int i = 0; i < V; ++i) sums[wave][lane * V + i] = sum[i];
    if (lane == 0) used[wave] = here;
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < p.experts; e += 64 * kSumWaves) {
      float all = sums[0][e];
#pragma unroll
      for (int w = 1; w < kSumWaves; ++w) all += sums[w][e];
      p.share_parts[row * p.experts + e] = all;
      p.count_parts[row * p.experts + e] = counts[e];
    }
    if (threadIdx.x == 0) {
      int all = 0;
#pragma unroll
      for (int w = 0; w < kSumWaves; ++w) all += used[w];
      p.used_parts[row] = all;
    }
    __syncthreads();
  });
}

// Workgroup (s, y): 64 experts of sequence s, ROWS threads for each, which share the
// rows of the sequence's chunks.  The last workgroup to arrive adds up the loss; it
// reads what the others left past its own L2.  Sums are 64 bits here, where the chunks'
// float32 ones come together, and the loss is rounded once (of 120 calls of 8191 to 1.2M
// tokens the largest error is 8e-8 of the loss, and 1e-7 with float32 throughout, in the
// same time).
constexpr int kExperts = 64;

__device__ __forceinline__ double wave_sum64(double v) {
  auto step = [&](auto ctrl) {
    const uint64_t u = __double_as_longlong(v);
    const uint32_t lo = dpp<decltype(ctrl)::value>((uint32_t)u), hi = dpp<decltype(ctrl)::value>((uint32_t)(u >> 32));
    v += __longlong_as_double(((uint64_t)hi << 32) | lo);
  };
  step(std::integral_constant<int, kXor1>{});
  step(std::integral_constant<int, kXor2>{});
  step(std::integral_constant<int, kHalfMirror>{});
  step(std::integral_constant<int, kRowMirror>{});
  auto row = [&](int lane) {
    const uint64_t u = __double_as_longlong(v);
    return __longlong_as_double(((uint64_t)lane_value((uint32_t)(u >> 32), lane) << 32) | lane_value((uint32_t)u, lane));
  };
  return (row(0) + row(16)) + (row(32) + row(48));
}

template <int ROWS>
__global__ __launch_bounds__(kExperts * ROWS) void balance_sum_kernel(BalanceParams p) {
  __shared__ double shares[ROWS][kExperts];
  __shared__ int counts[ROWS][kExperts];
  __shared__ int used_sum;
  __shared__ bool last;
  constexpr int kThreads = kExperts * ROWS;
  const int tid = threadIdx.x, at = tid % kExperts, part = tid / kExperts;
  const int s = blockIdx.x, e = blockIdx.y * kExperts + at;
  const Sequences seqs = {p.offsets, p.seqs, p.tokens};
  const int begin = seqs.at(s), end = seqs.at(s + 1);
  const int64_t first = begin / p.chunk, rows = end > begin ? (end - 1) / p.chunk - first + 1 : 0;
  if (tid == 0) used_sum = 0;
  __syncthreads();
  double share = 0.0;
  int count = 0, used = 0;
  if (e < p.experts) {
#pragma unroll 8
    for (int64_t r = part; r < rows; r += ROWS) {
      const int64_t from = (first + s + r) * p.experts + e;
      share += p.share_parts[from];
      count += p.count_parts[from];
    }
  }
  for (int64_t r = tid; r < rows; r += kThreads) used += p.used_parts[first + s + r];
  if (used) atomicAdd(&used_sum, used);
  shares[part][at] = share, counts[part][at] = count;
  __syncthreads();
  if (part == 0) {
#pragma unroll
    for (int k = 1; k < ROWS; ++k) share += shares[k][at], count += counts[k][at];
    used = used_sum;
    if (e < p.experts) p.counts[(int64_t)s * p.experts + e] = count;
    if (e == 0) p.used[s] = used;
    // f_e P_e = experts c_e / (topk n) times share / n
    double sum = wave_sum64(used ? (double)count * share : 0.0);
    if (at == 0) {
      if (used) sum *= p.experts_per_choice / ((double)used * used);
      __hip_atomic_store(&p.loss_parts[(int64_t)s * gridDim.y + blockIdx.y], sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // The store goes past the L2 and is waited for, like the reads below: no cache as a
      // whole has to be written back or dropped (8191 x 72: 7.2 -> 5.9 us).
      asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
      last = __hip_atomic_fetch_add(p.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  double sum = 0.0;
  for (int64_t k = tid; k < (int64_t)gridDim.x * gridDim.y; k += kThreads)
    sum += __hip_atomic_load(&p.loss_parts[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  sum = wave_sum64(sum);
  if (at == 0) shares[part][0] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int k = 1; k < ROWS; ++k) sum += shares[k][0];
    *p.loss = (float)(p.coef_mean * sum);
  }
}

// Waves and tokens of a workgroup of the gradient (32768 x 256 with a gradient to add to:
// 16 tokens 20 us, 32 tokens 21; the same with all of a wave's rows read before its
// sequence is known: the other waves cover that wait).
constexpr int kWaves = 4, kBwdChunk = 16;

template <bool VEC, typename T, int V>
__global__ __launch_bounds__(64 * kWaves) void balance_bwd_kernel(BalanceParams p) {
  __shared__ float rows[kWaves][64 * V];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Sequences seqs = {p.offsets, p.seqs, p.tokens};
  const float dloss = p.dloss ? *p.dloss : 1.0f;
  const int64_t t0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kBwdChunk, t1 = t0 + kBwdChunk;
  if (t0 >= p.tokens) return;
  for_sequences(seqs, (int)t0, (int)(t1 < p.tokens ? t1 : p.tokens), lane, [&](int s, int from, int to) {
    const int used = p.used[s];
    const float n = (float)used;
    const float a = used > 0 ? dloss * p.coef / ((float)p.seqs * n) : 0.0f;
    const float per = used > 0 ? (float)p.experts / ((float)p.topk * n) : 0.0f;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = lane * V + i;
      f[i] = e < p.experts ? per * (float)p.counts[(int64_t)s * p.experts + e] : 0.0f;
    }
    for (Turns<kWaves> turn(from, to, wave); turn.here(); turn.next()) {
      const int t = turn.row();
      float x[V], add[V], share[V], g[V], top = 0.0f;
      load_row<VEC>(static_cast<const T*>(p.logits) + (int64_t)t * p.ld, p.experts, lane, rows[wave], x);
      if (p.add) load_row<VEC>(static_cast<const T*>(p.add) + (int64_t)t * p.ld_add, p.experts, lane, rows[wave], add);
      const bool usual = ordinary<V>(x, p.sigmoid != 0, top);
      if (usual) {
        p.sigmoid ? slopes<V>(x, top, true, share, g) : slopes<V>(x, top, false, share, g);
      } else {
        float rest[V];
        shares<V>(x, share, rest, p.sigmoid != 0);
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = share[i] * rest[i];
      }
      float total = 0.0f, mean = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) total += share[i], mean = fmaf(f[i], share[i], mean);
      total = wave_sum(total);
      const float inv = usual ? reciprocal(total) : 1.0f;
      mean = wave_sum(mean) * inv;
      const float scale = a * inv;
      float out[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        out[i] = scale * (g[i] * (f[i] - mean));
        if (p.add) out[i] += add[i];
      }
      T* to_row = static_cast<T*>(p.dlogits) + (int64_t)t * p.ld_d;
      if constexpr (VEC) {
        Pack<T, V> pack;
#pragma unroll
        for (int i = 0; i < V; ++i) narrow(pack.v[i], out[i]);
        if (lane * V < p.experts) *reinterpret_cast<Pack<T, V>*>(to_row + lane * V) = pack;
      } else {
        wave_fence();
#pragma unroll
        for (int i = 0; i < V; ++i) rows[wave][lane * V + i] = out[i];
        wave_fence();
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = i * 64 + lane;
          if (e < p.experts) narrow(to_row[e], rows[wave][e]);
        }
      }
    }
  });
}

template <bool VEC, typename T, int V>
void go(const BalanceParams& p, bool bwd, hipStream_t stream) {
  if (bwd) {
    const GridXY grid = spread(((int64_t)p.tokens + kBwdChunk - 1) / kBwdChunk);
    hipLaunchKernelGGL((balance_bwd_kernel<VEC, T, V>), dim3(grid.x, grid.y), dim3(64 * kWaves), 0, stream, p);
  } else {
    const int64_t chunks = ((int64_t)p.tokens + p.chunk - 1) / p.chunk;
    hipLaunchKernelGGL((balance_kernel<VEC, T, V>), dim3((unsigned)(chunks > 0 ? chunks : 1)), dim3(64 * kSumWaves),
                       0, stream, p);
  }
}

// Whole vectors: no ragged last lane, and every row starts on a vector.
template <typename T, int V>
void go(const BalanceParams& p, bool bwd, hipStream_t stream) {
  constexpr size_t kAlign = alignof(Pack<T, V>);
  auto fits = [&](const void* at, int64_t ld) {
    return reinterpret_cast<uintptr_t>(at) % kAlign == 0 && ld * sizeof(T) % kAlign == 0;
  };
  const bool vec = p.experts % V == 0 && fits(p.logits, p.ld) &&
                   (!bwd || (fits(p.dlogits, p.ld_d) && (!p.add || fits(p.add, p.ld_add))));
  if (vec) go<true, T, V>(p, bwd, stream);
  else go<false, T, V>(p, bwd, stream);
}

template <typename T>
void pick(const BalanceParams& p, bool bwd, hipStream_t stream) {
  const int v = (p.experts + 63) / 64;
  if (v <= 1) go<T, 1>(p, bwd, stream);
  else if (v <= 2) go<T, 2>(p, bwd, stream);
  else if (v <= 4) go<T, 4>(p, bwd, stream);
  else if (v <= 8) go<T, 8>(p, bwd, stream);
  else go<T, 16>(p, bwd, stream);
}

}  // namespace

int balance_chunk(int tokens) {
  const int64_t share = ((int64_t)tokens + kMostChunks - 1) / kMostChunks;
  return share <= kSumWaves ? kSumWaves : (int)((share + kSumWaves - 1) / kSumWaves * kSumWaves);
}

int64_t balance_slots(int tokens, int seqs) {
  const int64_t chunk = balance_chunk(tokens);
  return ((int64_t)tokens + chunk - 1) / chunk + seqs;
}

int balance_loss_parts(int experts) { return (experts + kExperts - 1) / kExperts; }

hipError_t launch_balance(const BalanceParams& p, bool bf16, hipStream_t stream) {
  if (bf16) pick<uint16_t>(p, false, stream);
  else pick<float>(p, false, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid(p.seqs, balance_loss_parts(p.experts));
  const int64_t chunks_of_one = ((int64_t)p.tokens / p.seqs) / p.chunk;
  if (chunks_of_one > 16) hipLaunchKernelGGL(balance_sum_kernel<16>, grid, dim3(kExperts * 16), 0, stream, p);
  else hipLaunchKernelGGL(balance_sum_kernel<4>, grid, dim3(kExperts * 4), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_balance_bwd(const BalanceParams& p, bool bf16, hipStream_t stream) {
  if (bf16) pick<uint16_t>(p, true, stream);
  else pick<float>(p, true, stream);
  return hipGetLastError();
}

}  // namespace dg
