// 1x128 quantisation of float32 values, and the 128 x 128 tile that is
// quantised along its rows and, transposed, along its columns.
#pragma once

#include "dg_math.h"

namespace dg {

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
  const float near = u * series, far = (1.0f + fminf(v, 80.0f)) + s.e;
  return s.sig * s.n * (fabsf(u) < 0.0625f ? near : far);
}

// Tile kernels: 512 threads, thread t holds rows 4 (t / 16) .. + 3 and columns
// 8 (t % 16) .. + 7 of a 128 x 128 tile, so a row of the tile is 16 lanes and
// four rows of a column are the four bytes of a word of the transposed codes.
constexpr int kTileThreads = 512;

struct TileLds {
  float colmax[8][kBlockK];                 // a wave's maximum of each column
  uint32_t codes[kBlockK][kBlockK / 4 + 1];  // transposed codes, four rows a word
};

// Row-wise codes of the thread's 4 x 8 values: q points at the tile's first row
// and column (row stride ldq), sf at the scale of its first row.  Rows with
// their bit clear in `live` are not written.
__device__ __forceinline__ void tile_rows(const float (&v)[4][8], uint8_t* q, int64_t ldq, float* sf, uint32_t live) {
  const int r0 = (threadIdx.x >> 4) * 4, c0 = (threadIdx.x & 15) * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(v[i][c]));
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 16));
    const TileScale t = tile_scale(amax);
    if ((live >> i) & 1) {
      const uint32_t lo = e4m3_x4(v[i][0] * t.inv, v[i][1] * t.inv, v[i][2] * t.inv, v[i][3] * t.inv);
      const uint32_t hi = e4m3_x4(v[i][4] * t.inv, v[i][5] * t.inv, v[i][6] * t.inv, v[i][7] * t.inv);
      *reinterpret_cast<uint2*>(q + (int64_t)(r0 + i) * ldq + c0) = make_uint2(lo, hi);
      if (c0 == 0) sf[r0 + i] = t.s;
    }
  }
}

// Transposed codes of the tile, one scale per column: q points at the tile's
// first column (as a row of the transposed matrix, row stride ldq) and first
// row, sf at the scale of its first column.  Every thread of the workgroup
// calls it; values of rows not in use must be zero.
__device__ __forceinline__ void tile_columns(const float (&v)[4][8], TileLds& lds, uint8_t* q, int64_t ldq, float* sf) {
  const int tid = threadIdx.x, wave = tid >> 6;
  const int c0 = (tid & 15) * 8;
  float amax[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    amax[c] = fmaxf(fmaxf(fabsf(v[0][c]), fabsf(v[1][c])), fmaxf(fabsf(v[2][c]), fabsf(v[3][c])));
    amax[c] = fmaxf(amax[c], __shfl_xor(amax[c], 16, 64));
    amax[c] = fmaxf(amax[c], __shfl_xor(amax[c], 32, 64));
  }
  __syncthreads();  // the last use of lds is over
  if ((tid & 63) < 16) {
#pragma unroll
    for (int c = 0; c < 8; ++c) lds.colmax[wave][c0 + c] = amax[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float m = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, lds.colmax[w][c0 + c]);
    const TileScale t = tile_scale(m);
    lds.codes[c0 + c][tid >> 4] = e4m3_x4(v[0][c] * t.inv, v[1][c] * t.inv, v[2][c] * t.inv, v[3][c] * t.inv);
    if (tid < 16) sf[c0 + c] = t.s;
  }
  __syncthreads();
  // 8 lanes write the 128 codes of a column.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = i * 64 + (tid >> 3), w = (tid & 7) * 4;
    const uint32_t* p = &lds.codes[col][w];
    *reinterpret_cast<uint4*>(q + (int64_t)col * ldq + w * 4) = make_uint4(p[0], p[1], p[2], p[3]);
  }
}

}  // namespace dg
