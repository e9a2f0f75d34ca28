// Gradient of a product's epilogue for gfx950: what reaches the sum, as the codes
// that the input-gradient and the weight-gradient products take, and the bias'
// gradient.  16384 x 4096 with the GELU, 407 MB: 91.5 us, 4.5 TB/s; bound by the vector
// units and the memory together (the slope, two quotients and two roundings for each
// value).  Quotients from the hardware's reciprocal alone save 3 us, and codes next to a
// boundary then fall on its wrong side.

#include "dg_act.h"
#include "dg_block_internal.h"
#include "dg_tile.h"

namespace dg {
namespace {

// The first `rows` rows of a tile.
__device__ __forceinline__ TileUse first_rows(int rows) {
  return {rows >= 64 ? ~0ull : (1ull << rows) - 1, rows >= 128 ? ~0ull : rows > 64 ? (1ull << (rows - 64)) - 1 : 0ull};
}

// Workgroup: one 128 x 128 tile, 8 rows x 8 columns a thread: dd and z are read
// once for both code matrices and the columns' sums.
template <int ACT>
__global__ __launch_bounds__(kTileThreads<8>) void epilogue_bwd_kernel(EpilogueBwdParams p) {
  __shared__ TileLds<8> lds;
  __shared__ float sums[16][kBlockK];
  const int row_tiles = (p.rows + kBlockK - 1) / kBlockK;
  const TileAt tile = tile_of_workgroup(row_tiles, p.cols / kBlockK);
  const int64_t row0 = (int64_t)tile.row * kBlockK;
  const int col0 = tile.col * kBlockK;
  const int tid = threadIdx.x, r0 = (tid >> 4) * 8, c0 = (tid & 15) * 8;
  const int64_t left = p.rows - row0;
  const uint32_t live = first_rows(left < kBlockK ? (int)left : kBlockK).of_thread<8>();
  uint4 dd[8], z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = (live >> i) & 1;
    const int64_t row = row0 + r0 + i;
    dd[i] = z[i] = make_uint4(0, 0, 0, 0);
    if (in) dd[i] = load_streaming4(p.dd + row * p.ld_dd + col0 + c0);
    if (ACT != DG_ACT_NONE && in) z[i] = load_streaming4(p.pre + row * p.ld_pre + col0 + c0);
  }
  float vs[1][8][8];
  auto& v = vs[0];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a[4] = {dd[i].x, dd[i].y, dd[i].z, dd[i].w}, b[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      auto at = [&](const uint32_t* w) {
        return (c & 1) ? __uint_as_float(w[c >> 1] & 0xFFFF0000u) : __uint_as_float(w[c >> 1] << 16);
      };
      v[i][c] = ACT == DG_ACT_NONE ? at(a) : at(a) * act_slope<ACT>(at(b));
    }
  }
  if (p.dbias) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float sum = v[0][c];
#pragma unroll
      for (int i = 1; i < 8; ++i) sum += v[i][c];
      sums[tid >> 4][c0 + c] = sum;
    }
    __syncthreads();
    if (tid < kBlockK) {
      float sum = sums[0][tid];
#pragma unroll
      for (int k = 1; k < 16; ++k) sum += sums[k][tid];
      (row_tiles == 1 ? p.dbias : p.parts + (int64_t)tile.row * p.cols)[col0 + tid] = sum;
    }
  }
  tile_rows<true>(v, p.dq + row0 * p.cols + col0, p.cols, p.dsf + tile.col * p.ld_dsf + row0, live);
  if (!p.dqt) return;
  const int64_t wide = (int64_t)row_tiles * kBlockK;
  const ColumnsTo to[1] = {{p.dqt + (int64_t)col0 * wide + row0, wide, p.dsft + (int64_t)tile.row * p.ld_dsft + col0}};
  tile_columns<true>(vs, lds, to);
}

}  // namespace

hipError_t launch_epilogue_bwd(const EpilogueBwdParams& p, hipStream_t stream) {
  const int row_tiles = (int)(((int64_t)p.rows + kBlockK - 1) / kBlockK);
  if (p.rows > 0) {
    const dim3 grid((unsigned)(row_tiles * (p.cols / kBlockK))), block(kTileThreads<8>);
    switch (p.act) {
      case DG_ACT_RELU: hipLaunchKernelGGL(epilogue_bwd_kernel<DG_ACT_RELU>, grid, block, 0, stream, p); break;
      case DG_ACT_SILU: hipLaunchKernelGGL(epilogue_bwd_kernel<DG_ACT_SILU>, grid, block, 0, stream, p); break;
      case DG_ACT_GELU_TANH: hipLaunchKernelGGL(epilogue_bwd_kernel<DG_ACT_GELU_TANH>, grid, block, 0, stream, p); break;
      default: hipLaunchKernelGGL(epilogue_bwd_kernel<DG_ACT_NONE>, grid, block, 0, stream, p); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p.dbias || row_tiles == 1) return hipSuccess;
  ColumnSums s{};
  s.from[0] = p.parts, s.to[0] = p.dbias, s.count = 1, s.parts = row_tiles, s.cols = p.cols;
  return launch_column_sums(s, stream);
}

}  // namespace dg
