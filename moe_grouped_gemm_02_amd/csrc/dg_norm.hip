// The junction of two transformer blocks for gfx950: the norm after a block,
// gate and residual scale, the norm before the next block with the next GEMM's
// operand as its result, and the gradient of all of it.
//
// A team of threads (a wave, or a workgroup) holds one row, thread i chunks i,
// i + TEAM, .. of 8 values, so that loads and stores are whole 16-byte vectors
// side by side, 16 lanes own the 128 values of a code tile, and a row is read
// once, whatever its norms need: statistics are sums over the team, by row
// operations inside a wave and through shared memory between waves.

#include "dg_act.h"
#include "dg_block_internal.h"
#include "dg_math.h"
#include "dg_tile.h"

namespace dg {
namespace {

__device__ __forceinline__ void widen8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    f[2 * c] = __uint_as_float(w[c] << 16);
    f[2 * c + 1] = __uint_as_float(w[c] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// 1 / sqrt(a) for normal a: the hardware's (1 ulp) and one Newton step.
__device__ __forceinline__ float inverse_root(float a) {
  const float y = __builtin_amdgcn_rsqf(a);
  return fmaf(y * 0.5f, fmaf(-a * y, y, 1.0f), y);
}

// Sums over a team of N values each: a row of 16 lanes, two of them, a wave, or a
// workgroup.  Two calls one after another use different
// words of shared memory (`turn`), so that one barrier a call is enough: the words
// of a call are written again behind the barrier of the next one, which every wave
// passes after it has read them.
template <int TEAM>
struct TeamSums {
  static constexpr int kWaves = TEAM > 64 ? TEAM / 64 : 1;
  float words[2][kWaves][3];
};

template <int TEAM, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], TeamSums<TEAM>& lds, int& turn) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if constexpr (TEAM >= 64) v[n] = wave_sum(v[n]);
    else v[n] = row_sum(v[n]);
    if constexpr (TEAM == 32) v[n] += __shfl_xor(v[n], 16, 64);
  }
  if constexpr (TEAM > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) lds.words[turn][wave][n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      float sum = lds.words[turn][0][n];
#pragma unroll
      for (int w = 1; w < TEAM / 64; ++w) sum += lds.words[turn][w][n];
      v[n] = sum;
    }
    turn ^= 1;
  }
}

// The thread's chunks of a row.
template <int TEAM, int V>
struct Chunks {
  int lane, count;  // place in the team; chunks of the row
  __device__ __forceinline__ int at(int i) const { return i * TEAM + lane; }
  // Only the last of a thread's chunks can lie past the row's end (the host picks the
  // least V).
  __device__ __forceinline__ bool in(int i) const { return i < V - 1 || at(i) < count; }
};

template <int TEAM, int V>
__device__ __forceinline__ void load_chunks(const uint16_t* row, const Chunks<TEAM, V>& c, uint4 (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = c.in(i) ? load_streaming4(row + c.at(i) * 8) : make_uint4(0, 0, 0, 0);
}

template <bool STREAMING>
__device__ __forceinline__ void store8(uint16_t* to, const float (&f)[8]) {
  store<STREAMING>(to, narrow8(f));
}

// v = v w with the chunk's columns of w, v without w.
template <int TEAM, int V>
__device__ __forceinline__ void times_columns(const float* w, const Chunks<TEAM, V>& c, float (&v)[V][8]) {
  if (!w) return;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (!c.in(i)) continue;
    float k[8];
    load8(w + c.at(i) * 8, k);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= k[e];
  }
}

// A layer norm takes the mean first and the squares of what is left, since a single pass
// would lose rows with a large mean.  Of rows whose values hardly differ, the roundings of
// the mean would stay in every value (7168 times 1000: 2^-14, which the root of eps makes
// 0.06), so that what they leave of the mean, `rest`, is taken off too:
// * bf16 values of two neighbouring powers of two are multiples of 2^-9 of the largest, and
//   the sum of up to 2^14 of them is exact, so that the division's remainder is all of it.
//   (Others differ by a quarter of the largest, so that their root is at least 2^-9 of it.)
// * Float32 values have a sum that was rounded: what is left is summed with the squares.
//   sum (v - m)^2 of what is left, with its mean m = sum v^2 - m sum v
__device__ __forceinline__ float squares_around(float squares, float sum, float mean) {
  return fmaxf(fmaf(-sum, mean, squares), 0.0f);
}

// norm(v) = scale v + shift.  A layer norm's mean is taken off v here, and what that
// leaves of it is the shift.
struct Affine {
  float scale, shift;
};
// BF16: the values are those of a bf16 row.
template <bool LAYER, bool BF16, int TEAM, int V>
__device__ __forceinline__ Affine norm_of(float (&v)[V][8], const Chunks<TEAM, V>& c, float inv_cols, float eps,
                                          TeamSums<TEAM>& lds, int& turn) {
  if constexpr (LAYER) {
    float sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] += v[i][e];
    team_sums<TEAM>(sum, lds, turn);
    const float cols = (float)(c.count * 8), mean = sum[0] / cols;
    float s[BF16 ? 1 : 2] = {};  // squares, sum of what is left
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = c.in(i) ? v[i][e] - mean : 0.0f;
        v[i][e] = d, s[0] = fmaf(d, d, s[0]);
        if constexpr (!BF16) s[1] += d;
      }
    team_sums<TEAM>(s, lds, turn);
    float left = fmaf(-mean, cols, sum[0]);
    if constexpr (!BF16) left = s[1];
    const float rest = left * inv_cols;
    const float scale = inverse_root(fmaf(squares_around(s[0], left, rest), inv_cols, eps));
    return {scale, -rest * scale};
  } else {
    float squares[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) squares[0] = fmaf(v[i][e], v[i][e], squares[0]);
    team_sums<TEAM>(squares, lds, turn);
    return {inverse_root(fmaf(squares[0], inv_cols, eps)), 0.0f};
  }
}
template <bool LAYER>
__device__ __forceinline__ float normed(float v, const Affine& n) {
  return LAYER ? fmaf(v, n.scale, n.shift) : v * n.scale;
}

// Codes of 8 values x + rest (rest: what the rounding of x left), a tile of 128 by 16
// lanes.  The quotient takes in both residuals, so that a code differs from that of the
// exact value only where that lies within a rounding of a boundary (of 294M codes of
// normal rows 273 differ, and 318 with the quotient of the rounded value alone).
template <bool POW2>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const float (&rest)[8], float& s, uint32_t& e) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) m = fmaxf(m, fmaxf(fabsf(x[i] + rest[i]), fabsf(x[i + 1] + rest[i + 1])));
  uint32_t u = __float_as_uint(m);  // not negative: ordered like its bits
  u = umax(u, dpp<kXor1>(u));
  u = umax(u, dpp<kXor2>(u));
  u = umax(u, dpp<kHalfMirror>(u));
  u = umax(u, dpp<kRowMirror>(u));
  const float amax = __uint_as_float(u);
  if constexpr (POW2) {
    e = ue8m0_exponent_f32(amax);
    const int up = 127 - (int)e;
    auto q = [&](int j) { return __builtin_ldexpf(x[j] + rest[j], up); };
    return make_uint2(e4m3_of4(q(0), q(1), q(2), q(3)), e4m3_of4(q(4), q(5), q(6), q(7)));
  } else {
    const TileScale t = tile_scale(amax);
    s = t.s;
    auto q = [&](int j) {
      const float p = x[j] * t.inv;
      return fmaf(fmaf(-t.s, p, x[j]) + rest[j], t.inv, p);
    };
    return make_uint2(e4m3_of4(q(0), q(1), q(2), q(3)), e4m3_of4(q(4), q(5), q(6), q(7)));
  }
}

// The team's number in its workgroup, in a scalar register where a wave has one.
template <int TEAM>
__device__ __forceinline__ int team_of_thread() {
  const int team = threadIdx.x / TEAM;
  return TEAM < 64 ? team : __builtin_amdgcn_readfirstlane(team);
}

// Threads of a workgroup: teams smaller than 256 threads share one.
template <int TEAM>
constexpr int kNormThreads = TEAM < 256 ? 256 : TEAM;
template <int TEAM>
constexpr int kBwdThreads = TEAM < 256 ? 512 : TEAM;

// Bound by the memory: everything is read once and written once (16384 x 7168 with both
// norms, gate, r and codes: 205 us, 5.2 TB/s, where a copy of 256 MiB reaches 5.2; one
// row: 3.6 us, the launch).  The teams are the smallest that hold a row in 16 values a
// thread, since a row's sums wait for its last load and other rows have to fill that
// time: 512 threads for 7168 columns 207 us, 256 threads of 32 values 216, 1024 of 8
// 262; 375000 rows of 128 columns 62 us by 16 lanes, 160 by a wave.
// STREAMING: results larger than the L2s, which nothing reads back through them
// (store_streaming; 4096 x 7168 with r, bf16 rows and codes: 49.0 us, and 54.5 with
// plain stores).
template <bool POW2, bool STREAMING, bool LAYER, int TEAM, int V>
__global__ __launch_bounds__(kNormThreads<TEAM>) void norm_kernel(NormParams p) {
  constexpr int kTeams = kNormThreads<TEAM> / TEAM;
  static_assert(kTeams == 1 || TEAM <= 64, "teams that share a workgroup need no barrier");
  __shared__ TeamSums<TEAM> lds;
  int turn = 0;
  const Chunks<TEAM, V> c = {(int)threadIdx.x % TEAM, p.cols / 8};
  const float inv_cols = 1.0f / (float)p.cols;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  for (int64_t t = (int64_t)blockIdx.x * kTeams + team_of_thread<TEAM>(); t < p.tokens; t += step) {
    uint4 y[V], h[V];
    load_chunks(p.y + t * p.ld_y, c, y);
    if (p.h) load_chunks(p.h + t * p.ld_h, c, h);
    float v[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) widen8(y[i], v[i]);
    if (p.post) {
      const Affine n = norm_of<LAYER, true>(v, c, inv_cols, p.eps, lds, turn);
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = !LAYER || c.in(i) ? normed<LAYER>(v[i][e], n) : 0.0f;
      times_columns(p.post_weight, c, v);
    }
    if (p.gate_kind == DG_GATE_COLUMN) {
      times_columns(p.gate, c, v);
    } else if (p.gate_kind == DG_GATE_TOKEN) {
      const float g = p.gate[t];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= g;
    }
    if (p.h) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float f[8];
        widen8(h[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = fmaf(p.res_scale, f[e], v[i][e]);
      }
    }
    if (p.r) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c.in(i)) store8<STREAMING>(p.r + t * p.ld_r + c.at(i) * 8, v[i]);
    }
    if (!p.x && !p.q) continue;
    const Affine norm = norm_of<LAYER, false>(v, c, inv_cols, p.eps, lds, turn);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int at = c.at(i);
      float w[8], x[8], rest[8];
      if (p.weight && c.in(i)) {
        load8(p.weight + at * 8, w);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = normed<LAYER>(v[i][e], norm), of_n = fmaf(v[i][e], norm.scale, -n);
        x[e] = n * w[e];
        rest[e] = fmaf(LAYER ? of_n + norm.shift : of_n, w[e], fmaf(n, w[e], -x[e]));
      }
      if (p.bias && c.in(i)) {
        float b[8];
        load8(p.bias + at * 8, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // x + b = sum + what its rounding leaves (exact in float32, whichever is larger)
          const float sum = x[e] + b[e], of_b = sum - x[e];
          rest[e] += (x[e] - (sum - of_b)) + (b[e] - of_b);
          x[e] = sum;
        }
      }
      if (p.x && c.in(i)) store8<STREAMING>(p.x + t * p.ld_x + at * 8, x);
      if (!p.q) continue;
      // 16 lanes own a tile; those past the row's end are whole tiles.
      float s;
      uint32_t exponent;
      const uint2 codes = encode8<POW2>(x, rest, s, exponent);
      if (!c.in(i)) continue;
      store<STREAMING>(p.q + t * p.cols + at * 8, codes);
      if (at % 16 == 0) {
        const int64_t sf_at = (int64_t)(at / 16) * p.ld_sf + t;
        if constexpr (POW2) static_cast<uint8_t*>(p.sf)[sf_at] = (uint8_t)exponent;
        else static_cast<float*>(p.sf)[sf_at] = s;
      }
    }
  }
}

// What a thread reads of one row of the gradient.
template <int V>
struct NormBwdRaw {
  uint4 dx[V], dr[V], r[V], y[V];
};

template <int TEAM, int V>
__device__ __forceinline__ void load_raw(const NormBwdParams& p, int64_t t, bool read_y, const Chunks<TEAM, V>& c, NormBwdRaw<V>& raw) {
  if (p.dx) {
    load_chunks(p.dx + t * p.ld_dx, c, raw.dx);
    load_chunks(p.r + t * p.ld_r, c, raw.r);
  }
  if (p.dr) load_chunks(p.dr + t * p.ld_dr, c, raw.dr);
  if (read_y) load_chunks(p.y + t * p.ld_y, c, raw.y);
}

// The parameters' columns (ones without a parameter), where reading them again for
// each row waits for nothing but itself: loads from memory come back in order, so a
// row's parameters would wait for the next row, which is on its way (16384 x 7168: 264
// us, and 349 with parameters from memory).  In registers, or in shared memory, first
// and second halves of the chunks apart, so that lanes side by side read 16 bytes side
// by side; rows of more than 12288 values, which are not read ahead, take them from
// memory (there is room for them in shared memory: not tried).
enum ColumnsIn { kRegisters, kShared, kMemory };
template <int TEAM, int V>
constexpr ColumnsIn kColumnsIn = TEAM * V > 1536 ? kMemory : V == 1 ? kRegisters : kShared;
template <int TEAM, int V>
struct ColumnsLds {
  float4 half[2][kColumnsIn<TEAM, V> == kShared ? V * TEAM : 1];
};
template <int TEAM, int V>
struct Columns {
  const float* from;
  const ColumnsLds<TEAM, V>& lds;
  float kept[8];
  // The whole workgroup calls it; a barrier follows before the first get().
  __device__ __forceinline__ Columns(const float* w, ColumnsLds<TEAM, V>& to, const Chunks<TEAM, V>& c) : from(w), lds(to) {
    if constexpr (kColumnsIn<TEAM, V> == kRegisters) read(c, 0, kept);
    if constexpr (kColumnsIn<TEAM, V> == kShared) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v[8];
        read(c, i, v);
        to.half[0][c.at(i)] = make_float4(v[0], v[1], v[2], v[3]);
        to.half[1][c.at(i)] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
  }
  __device__ __forceinline__ void read(const Chunks<TEAM, V>& c, int i, float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
    if (from && c.in(i)) load8(from + c.at(i) * 8, v);
  }
  __device__ __forceinline__ void get(const Chunks<TEAM, V>& c, int i, float (&v)[8]) const {
    if constexpr (kColumnsIn<TEAM, V> == kRegisters) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = kept[e];
    } else if constexpr (kColumnsIn<TEAM, V> == kShared) {
      const float4 a = lds.half[0][c.at(i)], b = lds.half[1][c.at(i)];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      read(c, i, v);
    }
  }
};

// The sums of a column gradient over a team's rows: in registers, or, where two norms
// of rows of more than 12288 values leave none for them, each thread's in its own words
// of shared memory (16384 columns, both norms and a column gate: 3.6 TB/s, and 1.7 with
// sums that spill).  With one norm they stay in registers, and with the gradient of a bias
// or of a gate some 20 registers spill (16384 columns: 4.4 TB/s, 3.6 to 4.1 so); shared memory
// would hold these sums too.
template <int TEAM, int V, bool POST>
constexpr bool kSumsInLds = POST && TEAM * V > 1536;
template <int TEAM, int V, bool LDS>
struct ColumnAcc {
  float kept[LDS ? 1 : V][8] = {};
  float4* half;  // [2][V * TEAM], as ColumnsLds
  __device__ __forceinline__ ColumnAcc(float4* lds, const Chunks<TEAM, V>& c) : half(lds) {
    if constexpr (LDS) {
#pragma unroll
      for (int i = 0; i < V; ++i) half[c.at(i)] = half[V * TEAM + c.at(i)] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
  __device__ __forceinline__ void add(const Chunks<TEAM, V>& c, int i, const float (&a)[8], const float (&b)[8]) {
    if constexpr (LDS) {
      float v[8];
      get(c, i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(a[e], b[e], v[e]);
      half[c.at(i)] = make_float4(v[0], v[1], v[2], v[3]);
      half[V * TEAM + c.at(i)] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) kept[i][e] = fmaf(a[e], b[e], kept[i][e]);
    }
  }
  __device__ __forceinline__ void get(const Chunks<TEAM, V>& c, int i, float (&v)[8]) const {
    if constexpr (LDS) {
      const float4 a = half[c.at(i)], b = half[V * TEAM + c.at(i)];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = kept[i][e];
    }
  }
};

// Gradient.  Each team walks down the rows and keeps the sums over its rows of the
// column gradients; they leave once, as a row of partial sums of the workgroup, so that
// the sums need no atomics and their order is fixed.  Bound by the memory: 16384 x 7168
// with both norms 262 us, 5.4 TB/s; 4.9 to 5.6 TB/s up to 8192 columns (calls of a few
// thousand short rows are two launches: 4095 x 1000 3.1 TB/s), and above, where
// registers run short, 3.7 to 5.4 up to 12288 and 3.3 to 4.4 up to 16384.  The next row is
// read while this one is worked on.  POST, LAYER: as in the call; EXTRA: whether the
// gradients of a bias or of a column gate are wanted (registers for two more sums).
template <int TEAM, int V, bool POST, bool LAYER, bool EXTRA>
__global__ __launch_bounds__(kBwdThreads<TEAM>) void norm_bwd_kernel(NormBwdParams p) {
  constexpr int kTeams = kBwdThreads<TEAM> / TEAM;
  __shared__ TeamSums<TEAM> lds;
  int turn = 0;
  const Chunks<TEAM, V> c = {(int)threadIdx.x % TEAM, p.cols / 8};
  const float inv_cols = 1.0f / (float)p.cols;
  const bool read_y = POST || p.dgate;
  // A second row where the registers hold it.
  constexpr bool kAhead = TEAM * V <= 1024 || (TEAM * V <= 1536 && !(POST && EXTRA));
  __shared__ ColumnsLds<TEAM, V> columns[3];
  const Columns<TEAM, V> weight(p.weight, columns[0], c), post_weight(POST ? p.post_weight : nullptr, columns[1], c),
      gate(p.gate_kind == DG_GATE_COLUMN ? p.gate : nullptr, columns[2], c);
  __syncthreads();
  constexpr bool kLds = kSumsInLds<TEAM, V, POST>;
  __shared__ float4 sums[kLds ? 2 : 1][kLds ? 2 * V * TEAM : 1];
  ColumnAcc<TEAM, V, kLds> dw(sums[0], c), dpw(sums[kLds ? 1 : 0], c);
  ColumnAcc<TEAM, V, false> db(nullptr, c), dg(nullptr, c);
  NormBwdRaw<V> raw = {}, next = {};
  const int64_t step = (int64_t)gridDim.x * kTeams;
  int64_t t = (int64_t)blockIdx.x * kTeams + team_of_thread<TEAM>();
  if (kAhead && t < p.tokens) load_raw(p, t, read_y, c, next);
  for (; t < p.tokens; t += step) {
    if constexpr (kAhead) {
      raw = next;
      if (t + step < p.tokens) load_raw(p, t + step, read_y, c, next);
    } else {
      load_raw(p, t, read_y, c, raw);
    }
    // The sums that both norms' statistics need, together: the mean first (layer),
    // then squares and products with what is left (of bf16 values, see squares_around).
    float mean_r = 0.0f, mean_y = 0.0f, mean_g = 0.0f, left_r = 0.0f, left_y = 0.0f;
    if constexpr (LAYER) {
      float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float a[8], b[8], w[8];
        if (p.dx) {
          widen8(raw.r[i], a);
          widen8(raw.dx[i], b);
          weight.get(c, i, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] += a[e], s[2] = fmaf(b[e], w[e], s[2]);
        }
        if (POST) {
          widen8(raw.y[i], a);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[1] += a[e];
        }
      }
      team_sums<TEAM>(s, lds, turn);
      const float cols = (float)p.cols;
      mean_r = s[0] / cols, mean_y = s[1] / cols, mean_g = s[2] * inv_cols;
      left_r = fmaf(-mean_r, cols, s[0]), left_y = fmaf(-mean_y, cols, s[1]);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};  // squares of r, products of g and r, squares of y
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!c.in(i)) continue;
      float a[8], b[8], w[8];
      if (p.dx) {
        widen8(raw.r[i], a);
        widen8(raw.dx[i], b);
        weight.get(c, i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = a[e] - mean_r;
          s[0] = fmaf(d, d, s[0]);
          s[1] = fmaf(b[e] * w[e], d, s[1]);
        }
      }
      if (POST) {
        widen8(raw.y[i], a);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = a[e] - mean_y;
          s[2] = fmaf(d, d, s[2]);
        }
      }
    }
    if (p.dx || POST) team_sums<TEAM>(s, lds, turn);
    float rest_r = 0.0f, rest_y = 0.0f;
    if constexpr (LAYER) {
      rest_r = left_r * inv_cols, rest_y = left_y * inv_cols;
      s[0] = squares_around(s[0], left_r, rest_r), s[2] = squares_around(s[2], left_y, rest_y);
      s[1] = fmaf(-mean_g, left_r, s[1]);  // rest_r times the sum of g
    }
    const float kr = inverse_root(fmaf(s[0], inv_cols, p.eps));
    const float ky = POST ? inverse_root(fmaf(s[2], inv_cols, p.eps)) : 1.0f;
    const float gn = s[1] * inv_cols * kr;  // mean of g n
    const float shift_r = -rest_r * kr, shift_y = -rest_y * ky;  // norm(v) = (v - mean) k + shift
    const float token_gate = p.gate_kind == DG_GATE_TOKEN ? p.gate[t] : 1.0f;
    float tot[V][8];  // t, then e
    float after[3] = {0.0f, 0.0f, 0.0f};  // sums of e post_weight, of that times n(y), of t u
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (p.dr) widen8(raw.dr[i], tot[i]);
      else {
#pragma unroll
        for (int e = 0; e < 8; ++e) tot[i][e] = 0.0f;
      }
      if (!c.in(i)) continue;
      if (p.dx) {
        float n[8], b[8], w[8];
        widen8(raw.r[i], n);
        widen8(raw.dx[i], b);
        weight.get(c, i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          n[e] = fmaf(n[e] - mean_r, kr, shift_r);
          if constexpr (EXTRA) db.kept[i][e] += b[e];
          tot[i][e] = fmaf(kr, fmaf(-n[e], gn, fmaf(b[e], w[e], -mean_g)), tot[i][e]);
        }
        dw.add(c, i, b, n);
      }
      if (p.dh) {
        float out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) out[e] = p.res_scale * tot[i][e];
        store8<true>(p.dh + t * p.ld_dh + c.at(i) * 8, out);
      }
      float yv[8], pw[8], g[8];
      if constexpr (POST) post_weight.get(c, i, pw);
      gate.get(c, i, g);
      if (read_y) {
        widen8(raw.y[i], yv);
        if (POST) {
#pragma unroll
          for (int e = 0; e < 8; ++e) yv[e] = fmaf(yv[e] - mean_y, ky, shift_y);
        }
        if (p.dgate) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float tu = tot[i][e] * (POST ? yv[e] * pw[e] : yv[e]);
            if constexpr (EXTRA) dg.kept[i][e] += tu;
            after[2] += tu;
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) tot[i][e] *= g[e] * token_gate;
      if constexpr (POST) {
        dpw.add(c, i, tot[i], yv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          tot[i][e] *= pw[e];
          after[0] += tot[i][e];
          after[1] = fmaf(tot[i][e], yv[e], after[1]);
        }
      }
    }
    if (POST || (p.dgate && p.gate_kind == DG_GATE_TOKEN)) team_sums<TEAM>(after, lds, turn);
    if (p.gate_kind == DG_GATE_TOKEN && p.dgate && c.lane == 0) p.dgate[t] = after[2];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!c.in(i)) continue;
      if constexpr (POST) {
        float yv[8];
        widen8(raw.y[i], yv);
        const float m = LAYER ? after[0] * inv_cols : 0.0f, mn = after[1] * inv_cols;
#pragma unroll
        for (int e = 0; e < 8; ++e) tot[i][e] = ky * fmaf(-fmaf(yv[e] - mean_y, ky, shift_y), mn, tot[i][e] - m);
      }
      store8<true>(p.dy + t * p.ld_dy + c.at(i) * 8, tot[i]);
    }
  }
  // The workgroup's row of partial sums; waves with rows of their own come together
  // in shared memory, in order.
  auto leave = [&](auto get, float* to) {
    if (!to) return;
    to += (int64_t)blockIdx.x * p.cols;
    if constexpr (kTeams > 1) {
      __shared__ float rows[kTeams][V * TEAM * 8];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float sum[8];
        get(i, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) rows[threadIdx.x / TEAM][c.at(i) * 8 + e] = sum[e];
      }
      __syncthreads();
      for (int col = threadIdx.x; col < p.cols; col += kBwdThreads<TEAM>) {
        float all = rows[0][col];
#pragma unroll
        for (int k = 1; k < kTeams; ++k) all += rows[k][col];
        to[col] = all;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!c.in(i)) continue;
        float sum[8];
        get(i, sum);
        float4* at = reinterpret_cast<float4*>(to + c.at(i) * 8);
        at[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        at[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      }
    }
  };
  const int64_t matrix = (int64_t)gridDim.x * p.cols;
  auto of = [&](const auto& sum) { return [&](int i, float (&v)[8]) { sum.get(c, i, v); }; };
  leave(of(dw), p.dweight ? p.parts : nullptr);
  if constexpr (EXTRA) leave(of(db), p.dbias ? p.parts + matrix : nullptr);
  if constexpr (POST) leave(of(dpw), p.dpost_weight ? p.parts + 2 * matrix : nullptr);
  if constexpr (EXTRA) leave(of(dg), p.dgate && p.gate_kind == DG_GATE_COLUMN ? p.parts + 3 * matrix : nullptr);
}

// Workgroup (x, y): 64 columns of matrix y, 16 threads wide (4 columns each) and 16
// rows tall; the rows' sums come together in shared memory.  Bound by latency: 256 rows
// of 7168 columns 4 us, of which 3.7 are the launch's.
__global__ __launch_bounds__(256) void column_sums_kernel(ColumnSums s) {
  __shared__ float4 rows[16][16];
  const float* from = s.from[blockIdx.y];
  const int at = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + at * 4;
  float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < s.cols) {
#pragma unroll 8
    for (int k = row; k < s.parts; k += 16) {
      const float4 v = *reinterpret_cast<const float4*>(from + (int64_t)k * s.cols + col);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
  }
  rows[row][at] = sum;
  __syncthreads();
  if (row == 0 && col < s.cols) {
#pragma unroll
    for (int k = 1; k < 16; ++k) {
      const float4 v = rows[k][at];
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    *reinterpret_cast<float4*>(s.to[blockIdx.y] + col) = sum;
  }
}

template <bool POW2, bool STREAMING, int TEAM, int V>
void go_norm(const NormParams& p, hipStream_t stream) {
  constexpr int kTeams = kNormThreads<TEAM> / TEAM;
  const int64_t need = ((int64_t)p.tokens + kTeams - 1) / kTeams;
  const unsigned grid = (unsigned)(need < (1 << 20) ? need : (1 << 20));
  if (p.layer) hipLaunchKernelGGL((norm_kernel<POW2, STREAMING, true, TEAM, V>), dim3(grid), dim3(kNormThreads<TEAM>), 0, stream, p);
  else hipLaunchKernelGGL((norm_kernel<POW2, STREAMING, false, TEAM, V>), dim3(grid), dim3(kNormThreads<TEAM>), 0, stream, p);
}

template <bool POW2, bool STREAMING>
void pick_norm(const NormParams& p, hipStream_t stream) {
  const int chunks = p.cols / 8;
  if (chunks <= 16) go_norm<POW2, STREAMING, 16, 1>(p, stream);
  else if (chunks <= 32) go_norm<POW2, STREAMING, 32, 1>(p, stream);
  else if (chunks <= 64) go_norm<POW2, STREAMING, 64, 1>(p, stream);
  else if (chunks <= 128) go_norm<POW2, STREAMING, 64, 2>(p, stream);
  else if (chunks <= 256) go_norm<POW2, STREAMING, 256, 1>(p, stream);
  else if (chunks <= 512) go_norm<POW2, STREAMING, 256, 2>(p, stream);
  else if (chunks <= 1024) go_norm<POW2, STREAMING, 512, 2>(p, stream);
  else go_norm<POW2, STREAMING, 1024, 2>(p, stream);
}

template <int TEAM, int V, bool POST, bool LAYER, bool EXTRA>
void go_norm_bwd(const NormBwdParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((norm_bwd_kernel<TEAM, V, POST, LAYER, EXTRA>), dim3(norm_bwd_parts(p.tokens, p.cols)),
                     dim3(kBwdThreads<TEAM>), 0, stream, p);
}

template <int TEAM, int V>
void pick_norm_bwd(const NormBwdParams& p, hipStream_t stream) {
  const bool extra = p.dbias || (p.dgate && p.gate_kind == DG_GATE_COLUMN);
  auto go = [&](auto post, auto layer) {
    constexpr bool kPost = decltype(post)::value, kLayer = decltype(layer)::value;
    if (extra) go_norm_bwd<TEAM, V, kPost, kLayer, true>(p, stream);
    else go_norm_bwd<TEAM, V, kPost, kLayer, false>(p, stream);
  };
  using std::false_type, std::true_type;
  if (p.post) p.layer ? go(true_type{}, true_type{}) : go(true_type{}, false_type{});
  else p.layer ? go(false_type{}, true_type{}) : go(false_type{}, false_type{});
}

// Rows that a workgroup of the gradient has at a time, and how many workgroups it
// takes to fill the card.
int teams_of(int cols) { return cols <= 128 ? 32 : cols <= 256 ? 16 : cols <= 1024 ? 8 : 1; }
int most_parts(int cols) { return cols <= 1024 ? 256 : cols <= 2048 ? 1024 : cols <= 4096 ? 512 : 256; }

}  // namespace

hipError_t launch_block_norm(const NormParams& p, bool pow2, hipStream_t stream) {
  const bool streaming = (int64_t)p.tokens * p.cols > (int64_t)8 << 20;
  if (pow2) streaming ? pick_norm<true, true>(p, stream) : pick_norm<true, false>(p, stream);
  else streaming ? pick_norm<false, true>(p, stream) : pick_norm<false, false>(p, stream);
  return hipGetLastError();
}

int norm_bwd_parts(int tokens, int cols) {
  const int64_t need = ((int64_t)tokens + teams_of(cols) - 1) / teams_of(cols);
  return need < most_parts(cols) ? (int)need : most_parts(cols);
}

hipError_t launch_block_norm_bwd(const NormBwdParams& p, hipStream_t stream) {
  const int chunks = p.cols / 8;
  if (p.tokens > 0) {
    if (chunks <= 16) pick_norm_bwd<16, 1>(p, stream);
    else if (chunks <= 32) pick_norm_bwd<32, 1>(p, stream);
    else if (chunks <= 64) pick_norm_bwd<64, 1>(p, stream);
    else if (chunks <= 128) pick_norm_bwd<64, 2>(p, stream);
    else if (chunks <= 256) pick_norm_bwd<256, 1>(p, stream);
    else if (chunks <= 512) pick_norm_bwd<512, 1>(p, stream);
    else if (chunks <= 1024) pick_norm_bwd<512, 2>(p, stream);
    else if (chunks <= 1536) pick_norm_bwd<512, 3>(p, stream);
    else pick_norm_bwd<512, 4>(p, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  ColumnSums s{};
  s.parts = norm_bwd_parts(p.tokens, p.cols), s.cols = p.cols;
  const int64_t matrix = (int64_t)s.parts * p.cols;
  float* column_gate = p.gate_kind == DG_GATE_COLUMN ? p.dgate : nullptr;
  float* const to[4] = {p.dweight, p.dbias, p.dpost_weight, column_gate};
  for (int k = 0; k < 4; ++k)
    if (to[k]) s.from[s.count] = p.parts + k * matrix, s.to[s.count++] = to[k];
  return s.count ? launch_column_sums(s, stream) : hipSuccess;
}

hipError_t launch_column_sums(const ColumnSums& c, hipStream_t stream) {
  hipLaunchKernelGGL(column_sums_kernel, dim3((c.cols + 63) / 64, c.count), dim3(256), 0, stream, c);
  return hipGetLastError();
}

}  // namespace dg
