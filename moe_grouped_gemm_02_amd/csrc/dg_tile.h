// 1x128 quantisation of float32 values, and the 128 x 128 tile that is
// quantised along its rows and, transposed, along its columns.
#pragma once

#include "dg_math.h"

namespace dg {

// e4m3_x4 without a cleared register to convert into: the two conversions write all
// four bytes, so whatever a's register holds beside them will do.
__device__ __forceinline__ uint32_t e4m3_of4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)__float_as_uint(a), false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Scale and its inverse for float32 values: s = amax / 448 (a product with one
// correction by its residual), kept normal (at least 2^-126) so that its
// reciprocal is finite; 0 for an all-zero tile.  Scale, inverse and product are
// each within about half an ulp, so |v| * inv stays below 448 * (1 + 2^-21),
// where the conversion still rounds to 448.
struct TileScale {
  float s, inv;
};
__device__ __forceinline__ TileScale tile_scale(float amax) {
  const float q = amax * (1.0f / 448.0f);
  const float s = fmaxf(fmaf(fmaf(-448.0f, q, amax), 1.0f / 448.0f, q), 0x1p-126f);
  return amax > 0.0f ? TileScale{s, reciprocal(s)} : TileScale{0.0f, 0.0f};
}

// Codes of four values: EXACT divides, by a correction with the quotient's residual
// (see encode_bf16_tile); otherwise the product with the inverse, within 2 ulp,
// stands for v / s.  Dividing costs nothing where memory is the bound and 150 ->
// 165 us in the gated unit's backward, where it changes one code in 10^6.
template <bool EXACT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float inv) {
  auto q = [&](float v) {
    const float p = v * inv;
    return EXACT ? fmaf(fmaf(-s, p, v), inv, p) : p;
  };
  return e4m3_of4(q(a), q(b), q(c), q(d));
}

// UE8M0 exponent of ue8m0_exponent() for any float32 amax, from its bits:
// amax = m 2^e with 448 = 1.75 * 2^8, so ceil(log2(amax / 448)) is e - 8, and
// one more where m > 1.75.
__device__ __forceinline__ uint32_t ue8m0_exponent_f32(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return (uint32_t)(e < 0 ? 0 : e);
}

// d silu / dv = sig (1 + v (1 - sig)) = sig n (1 + v + e^v) at v = code * scale.
// The sum crosses zero at v0 = -1.27846454..., where the roundings of v and e^v
// would be all that is left of it: within 1/16 of v0 it is u + e^v0 (e^u - 1)
// with u = v - v0 from the unrounded product, and the series of e^u to u^4 (the
// next term is below 2^-24 of the sum).
__device__ __forceinline__ float silu_slope(float code, float scale, float v, const Sigmoid& s) {
  constexpr float kRootHi = -1.27846455574035644531f, kRootLo = 1.29792827e-8f;  // v0 = hi + lo
  constexpr float kExpRoot = 0.27846454276107379511f;                            // e^v0 = -1 - v0
  const float u = fmaf(code, scale, -kRootHi) - kRootLo;
  float series = fmaf(u, kExpRoot / 24.0f, kExpRoot / 6.0f);
  series = fmaf(u, series, kExpRoot / 2.0f);
  series = fmaf(u, series, 1.0f + kExpRoot);
  const float near = u * series, far = (1.0f + __builtin_amdgcn_fmed3f(v, -150.0f, 80.0f)) + s.e;
  return s.sig * s.n * (fabsf(u) < 0.0625f ? near : far);
}

// Sixteen bf16 values of a lane; eight lanes own a tile of 128.
struct Lane16 {
  uint32_t w[8];
  __device__ __forceinline__ float at(int i) const {
    return (i & 1) ? __uint_as_float(w[i >> 1] & 0xFFFF0000u) : __uint_as_float(w[i >> 1] << 16);
  }
};
__device__ __forceinline__ Lane16 load16(const uint16_t* p) {
  const uint4 lo = *reinterpret_cast<const uint4*>(p), hi = *reinterpret_cast<const uint4*>(p + 8);
  return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// Maximum over the eight lanes of a tile, of values that are not negative.
__device__ __forceinline__ float max_of_tile(float v) {
  uint32_t u = __float_as_uint(v);
  u = umax(u, dpp<kXor1>(u));
  u = umax(u, dpp<kXor2>(u));
  u = umax(u, dpp<kHalfMirror>(u));
  return __uint_as_float(u);
}

template <typename Values>
__device__ __forceinline__ float amax16(const Values& at) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) m = fmaxf(m, fmaxf(fabsf(at(i)), fabsf(at(i + 1))));
  return max_of_tile(m);
}

// The same of a lane's bf16 values: their magnitudes are ordered like their bits,
// two of which are compared at once.
__device__ __forceinline__ float amax16(const Lane16& v) {
  typedef unsigned short v2u __attribute__((ext_vector_type(2)));
  v2u m = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2u, v.w[i] & 0x7FFF7FFFu));
  return max_of_tile(__uint_as_float(umax(m.x, m.y) << 16));
}

template <typename Values>
__device__ __forceinline__ uint4 encode16(const Values& at) {
  return make_uint4(e4m3_of4(at(0), at(1), at(2), at(3)), e4m3_of4(at(4), at(5), at(6), at(7)),
                    e4m3_of4(at(8), at(9), at(10), at(11)), e4m3_of4(at(12), at(13), at(14), at(15)));
}

// Codes and scale of a bf16 tile, those of the plain activation quantiser bit
// for bit: s = fp32(amax / 448), q = e4m3(fp32(x / s)).  Both quotients are a
// product with the rounded reciprocal and one correction by the exact residual,
// which is the rounded quotient itself (all s and |x| <= amax of normal bf16
// magnitude tried on the host, 1.03e9 pairs; quotients below 2^-12 may differ
// and have the code of zero).  The residual's order keeps the sign of a zero.
// That needs residuals that float32 holds: tiles with s below 2^-90 (an all-zero
// one among them) take the double-precision form.  (That form for all takes as long
// in the dispatch of 32768 x 7168, which waits for memory, but a quarter more
// vector instructions.)
__device__ __forceinline__ uint4 encode_bf16_tile(const Lane16& v, float& s) {
  const float amax = amax16(v);
  constexpr float kInv448 = 1.0f / 448.0f;
  const float s0 = amax * kInv448;
  s = fmaf(fmaf(-448.0f, s0, amax), kInv448, s0);
  if (__ballot(!(s >= 0x1p-90f))) {
    s = amax / 448.0f;
    const double rcp = tile_reciprocal(s);
    return encode16([&](int i) { return (float)((double)v.at(i) * rcp); });
  }
  float inv = reciprocal(s);
  inv = fmaf(fmaf(-s, inv, 1.0f), inv, inv);
  return encode16([&](int i) {
    const float x = v.at(i), q = x * inv;
    return fmaf(-fmaf(s, q, -x), inv, q);
  });
}
// The same with a power-of-two scale 2^(e - 127).
__device__ __forceinline__ uint4 encode_bf16_tile_pow2(const Lane16& v, uint32_t& e) {
  e = ue8m0_exponent_f32(amax16(v));
  const int up = 127 - (int)e;
  return encode16([&](int i) { return __builtin_ldexpf(v.at(i), up); });
}

// 128 x 128 tiles.  Thread t of the workgroup holds R rows, R (t / 16) on, and
// 8 columns, 8 (t % 16) on: a row of the tile is 16 lanes, a row of the
// hardware's row operations, and the R rows of a column are R bytes of the
// transposed codes.  R = 8 takes 256 threads, R = 4 512.
template <int R>
constexpr int kTileThreads = kBlockK * kBlockK / (8 * R);

// Shared memory of N tiles whose columns are quantised together.
template <int R, int N = 1>
struct TileLds {
  static constexpr int kGroups = kBlockK / R;
  static constexpr int kParts = kTileThreads<R> / kBlockK;  // threads that share a column's maximum
  // Maximum of each column over each group of R rows.  A thread writes 8 columns
  // as two vectors, each into a half of the row of its own, so that 8 lanes write
  // 128 consecutive bytes; the offsets of the halves and of every eighth group put
  // what 32 lanes then read, 32 / kParts columns of kParts groups, on 32 different
  // banks.
  static constexpr int kHalf = kBlockK / 2 + 16 / kParts, kRow = kHalf + kBlockK / 2;
  static __device__ __forceinline__ int partial_at(int group, int col) {
    return group * kRow + (group >> 3) * (32 / kParts) + ((col >> 2) & 1) * kHalf + (col >> 3) * 4 + (col & 3);
  }
  static __device__ __forceinline__ int inv_at(int col) {
    return ((col >> 2) & 1) * (kBlockK / 2) + (col >> 3) * 4 + (col & 3);
  }
  alignas(16) float partial[N][kGroups * kRow + 32];
  alignas(16) float inv[N][kBlockK], s[N][kBlockK];
  alignas(16) uint8_t codes[N][kBlockK * kBlockK];
};

// Where the code of row `row` and column `col` lies in TileLds::codes.  32 lanes
// write rows of columns 8 apart, 8 lanes read a column's 8 chunks of 16 bytes: the
// exclusive-ors spread the first over all banks (bit 6 of the column picks which
// half of a chunk holds its first 8 rows) and leave the second a permutation of
// 128 bytes.  (The gated unit's backward, 32768 x 2048: 150 us with no conflicts
// here or at the maxima, 153 with 2 and 4 lanes on a bank.)
__device__ __forceinline__ int codes_at(int col, int row) {
  return col * kBlockK + (((row >> 4) ^ ((col >> 3) & 7)) * 16) + ((row & 15) ^ ((col >> 6) * 8));
}

// Rows of the tile in use (0 <= index < end), the same in every wave: lane l looks
// at rows l and l + 64.
struct TileUse {
  uint64_t lo, hi;
  __device__ __forceinline__ bool any() const { return (lo | hi) != 0; }
  // The thread's R rows as bits.
  template <int R>
  __device__ __forceinline__ uint32_t of_thread() const {
    const int r0 = (threadIdx.x >> 4) * R;
    return (uint32_t)((r0 < 64 ? lo : hi) >> (r0 & 63)) & ((1u << R) - 1u);
  }
};
__device__ __forceinline__ TileUse tile_use(const int32_t* index, uint32_t end = 0x80000000u) {
  if (!index) return {~0ull, ~0ull};
  const int lane = threadIdx.x & 63;
  const uint32_t a = (uint32_t)index[lane], b = (uint32_t)index[lane + 64];
  return {__ballot(a < end), __ballot(b < end)};
}

// Tile of a workgroup, one of the first row_tiles x column_tiles.  Those
// that run one after another on one XCD (every eighth) take a contiguous eighth
// of the tiles, row tiles fastest: they write neighbouring pieces of the same
// columns through one L2 (requantising 32768 x 7168: 92 us against 98 in plain
// order, 118 and more in panels of rows; 83 with streaming stores).
struct TileAt {
  int row, col;
};
__device__ __forceinline__ TileAt tile_of_workgroup(int row_tiles, int column_tiles) {
  const int per = row_tiles * column_tiles / 8;
  int b = blockIdx.x;
  if (b < per * 8) b = (b % 8) * per + b / 8;
  return {b % row_tiles, b / row_tiles};
}

// R consecutive floats from a 16-byte boundary.
template <int R>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + i);
    v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
  }
}

// Scale and inverse of each of the thread's rows: lane i of the 16 (i < R)
// computes row i's, so that the rows' divisions are made once, not by all lanes;
// row i's inverse is then v of lane i.
template <int R>
__device__ __forceinline__ TileScale row_scale_of_lane(const float (&v)[R][8]) {
  const int i16 = threadIdx.x & 15;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float m = fmaxf(fabsf(v[i][0]), fabsf(v[i][1]));
#pragma unroll
    for (int c = 2; c < 8; c += 2) m = fmaxf(m, fmaxf(fabsf(v[i][c]), fabsf(v[i][c + 1])));
    uint32_t u = __float_as_uint(m);  // not negative: ordered like its bits
    u = umax(u, dpp<kXor1>(u));
    u = umax(u, dpp<kXor2>(u));
    u = umax(u, dpp<kHalfMirror>(u));
    u = umax(u, dpp<kRowMirror>(u));
    mine = i16 == i ? u : mine;
  }
  return tile_scale(__uint_as_float(mine));
}

// Row-wise codes of the thread's values: q points at the tile's first row and
// column (row stride ldq), sf at the scale of its first row.  Rows with their
// bit clear in `live` are not written.
template <bool EXACT, int R>
__device__ __forceinline__ void tile_rows(const float (&v)[R][8], uint8_t* q, int64_t ldq, float* sf, uint32_t live) {
  const int r0 = (threadIdx.x >> 4) * R, c0 = (threadIdx.x & 15) * 8, i16 = threadIdx.x & 15;
  const TileScale t = row_scale_of_lane<R>(v);
  if (i16 < R && ((live >> i16) & 1)) sf[r0 + i16] = t.s;
  q += (int64_t)r0 * ldq + c0;
  auto row = [&](auto index) {
    constexpr int i = decltype(index)::value;
    const float inv = dpp<kRowLane0 + i>(t.inv), s = EXACT ? dpp<kRowLane0 + i>(t.s) : 0.0f;
    const uint32_t lo = codes4<EXACT>(v[i][0], v[i][1], v[i][2], v[i][3], s, inv);
    const uint32_t hi = codes4<EXACT>(v[i][4], v[i][5], v[i][6], v[i][7], s, inv);
    if ((live >> i) & 1) store_streaming(q, make_uint2(lo, hi));
    q += ldq;
  };
  for_each_index<R>(row);
}

// Where a tile's transposed codes go: q its first column (as a row of the
// transposed matrix, row stride ldq) and first row, sf the scale of its first
// column.  q null: nowhere.
struct ColumnsTo {
  uint8_t* q;
  int64_t ldq;
  float* sf;
};

// Transposed codes of N tiles, one scale per column.  Every thread of the
// workgroup calls it; values of rows not in use must be zero.  Three barriers
// in all; a next call may follow at once, since each part of lds is written
// only behind a barrier that its last readers have passed.
template <bool EXACT, int R, int N>
__device__ __forceinline__ void tile_columns(const float (&v)[N][R][8], TileLds<R, N>& lds, const ColumnsTo (&to)[N]) {
  using Lds = TileLds<R, N>;
  constexpr int kParts = Lds::kParts;
  const int tid = threadIdx.x, group = tid >> 4, c0 = (tid & 15) * 8;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float amax[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      amax[c] = fmaxf(fabsf(v[n][0][c]), fabsf(v[n][1][c]));
#pragma unroll
      for (int i = 2; i < R; i += 2) amax[c] = fmaxf(amax[c], fmaxf(fabsf(v[n][i][c]), fabsf(v[n][i + 1][c])));
    }
    float* at = lds.partial[n] + Lds::partial_at(group, c0);
    *reinterpret_cast<float4*>(at) = make_float4(amax[0], amax[1], amax[2], amax[3]);
    *reinterpret_cast<float4*>(at + Lds::kHalf) = make_float4(amax[4], amax[5], amax[6], amax[7]);
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int col = tid / kParts, part = tid % kParts;
    uint32_t u = 0;  // maxima are not negative: ordered like their bits
#pragma unroll
    for (int i = 0; i < 8; ++i) u = umax(u, __float_as_uint(lds.partial[n][Lds::partial_at(part * 8 + i, col)]));
    u = umax(u, dpp<kXor1>(u));
    if (kParts == 4) u = umax(u, dpp<kXor2>(u));
    const TileScale t = tile_scale(__uint_as_float(u));
    if (part == 0) {
      lds.inv[n][Lds::inv_at(col)] = t.inv;
      if (EXACT) lds.s[n][Lds::inv_at(col)] = t.s;
      if (to[n].q) to[n].sf[col] = t.s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float inv[8], s[8];
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
      *reinterpret_cast<float4*>(inv + h) = *reinterpret_cast<const float4*>(lds.inv[n] + Lds::inv_at(c0 + h));
      if (EXACT) *reinterpret_cast<float4*>(s + h) = *reinterpret_cast<const float4*>(lds.s[n] + Lds::inv_at(c0 + h));
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint8_t* at = lds.codes[n] + codes_at(c0 + c, group * R);
      const uint32_t lo = codes4<EXACT>(v[n][0][c], v[n][1][c], v[n][2][c], v[n][3][c], s[c], inv[c]);
      if constexpr (R == 8) {
        const uint32_t hi = codes4<EXACT>(v[n][4][c], v[n][5][c], v[n][6][c], v[n][7][c], s[c], inv[c]);
        *reinterpret_cast<uint2*>(at) = make_uint2(lo, hi);
      } else {
        *reinterpret_cast<uint32_t*>(at) = lo;
      }
    }
  }
  __syncthreads();
  // 8 lanes write the 128 codes of a column.
  constexpr int kColumns = kTileThreads<R> / 8;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if (!to[n].q) continue;
#pragma unroll
    for (int i = 0; i < kBlockK / kColumns; ++i) {
      const int col = i * kColumns + (tid >> 3), row = (tid & 7) * 16;
      const bool swapped = i * kColumns >= 64;
      const uint4 w = *reinterpret_cast<const uint4*>(lds.codes[n] + (codes_at(col, row) & ~15));
      store_streaming(to[n].q + (int64_t)col * to[n].ldq + row,
                      swapped ? make_uint4(w.z, w.w, w.x, w.y) : w);
    }
  }
}

}  // namespace dg
