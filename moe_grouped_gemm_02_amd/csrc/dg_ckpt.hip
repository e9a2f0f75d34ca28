// The experts' gated unit and its 8-bit activation checkpoint for gfx950:
// quantised forward, backward from the checkpoint, and the operands of the
// weight-gradient GEMMs (tiles of 128 rows of a column, transposed).

#include "dg_device.h"
#include "dg_moe_internal.h"
#include "dg_tile.h"

namespace dg {
namespace {

// Sixteen bf16 values of a lane, widened.
struct Lane16 {
  uint32_t w[8];
  __device__ __forceinline__ float at(int i) const {
    return bf16_bits_to_f32((i & 1) ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
  }
};
__device__ __forceinline__ Lane16 load16(const uint16_t* p) {
  const uint4 lo = *reinterpret_cast<const uint4*>(p), hi = *reinterpret_cast<const uint4*>(p + 8);
  return {{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}};
}

// The 1x128 code of a bf16 tile whose 16 values a lane are in v, as the plain
// activation quantiser computes it.
__device__ __forceinline__ void store_bf16_tile(const Lane16& v, uint8_t* q, float* sf, int sub) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v.at(i)));
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 8));
  const float s = amax / 448.0f;
  const double rcp = tile_reciprocal(s);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    out[i] = e4m3_x4(quotient(v.w[2 * i] & 0xFFFFu, rcp), quotient(v.w[2 * i] >> 16, rcp),
                     quotient(v.w[2 * i + 1] & 0xFFFFu, rcp), quotient(v.w[2 * i + 1] >> 16, rcp));
  *reinterpret_cast<uint4*>(q) = make_uint4(out[0], out[1], out[2], out[3]);
  if (sub == 0) *sf = s;
}

constexpr int kTilesPerWave = 8;
constexpr int kRowWaves = 4;

// 8 lanes own one 128-value tile of a row's gate and the same tile of its up
// half; a wave owns 8 tiles, block (x, y) tiles [8 x, 8 x + 8) and four rows at a
// time.
template <bool POW2, bool CKPT>
__global__ __launch_bounds__(64 * kRowWaves) void swiglu_kernel(SwigluParams p) {
  const int tiles = p.inter / kBlockK;
  const int sub = threadIdx.x & 7;
  const int j = blockIdx.x * kTilesPerWave + ((threadIdx.x & 63) >> 3);
  if (j >= tiles) return;
  const int64_t total = (int64_t)p.groups * p.rows;
  for (int64_t gr = (int64_t)blockIdx.y * kRowWaves + (threadIdx.x >> 6); gr < total;
       gr += (int64_t)gridDim.y * kRowWaves) {
    const int64_t g = gr / p.rows, r = gr - g * p.rows;
    if (p.m_indices && p.m_indices[gr] < 0) continue;
    if (p.masked_m && r >= p.masked_m[g]) continue;
    const int col = j * kBlockK + sub * 16;
    const uint16_t* h = p.h + gr * p.ld_h + col;
    const Lane16 gate = load16(h), up = load16(h + p.inter);
    float a[16], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = gate.at(i);
      a[i] = v * sigmoid(v).sig * up.at(i);
      amax = fmaxf(amax, fabsf(a[i]));
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 8));
    uint32_t out[4];
    const int64_t sf_at = (g * tiles + j) * p.ld_sf + r;
    if constexpr (POW2) {
      const uint32_t e = ue8m0_exponent_f32(amax);
      const int up2 = 127 - (int)e;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = e4m3_x4(__builtin_ldexpf(a[4 * i], up2), __builtin_ldexpf(a[4 * i + 1], up2),
                         __builtin_ldexpf(a[4 * i + 2], up2), __builtin_ldexpf(a[4 * i + 3], up2));
      if (sub == 0) static_cast<uint8_t*>(p.sf)[sf_at] = (uint8_t)e;
    } else {
      const TileScale t = tile_scale(amax);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = e4m3_x4(a[4 * i] * t.inv, a[4 * i + 1] * t.inv, a[4 * i + 2] * t.inv, a[4 * i + 3] * t.inv);
      if (sub == 0) static_cast<float*>(p.sf)[sf_at] = t.s;
    }
    *reinterpret_cast<uint4*>(p.q + gr * p.inter + col) = make_uint4(out[0], out[1], out[2], out[3]);
    if constexpr (CKPT) {
      uint8_t* hq = p.hq + gr * 2 * p.inter + col;
      float* hsf = p.hsf + (g * 2 * tiles + j) * p.ld_hsf + r;
      store_bf16_tile(gate, hq, hsf, sub);
      store_bf16_tile(up, hq + p.inter, hsf + (int64_t)tiles * p.ld_hsf, sub);
    }
  }
}

// The thread's 8 codes of a row as numbers.
__device__ __forceinline__ void decode8(const uint8_t* q, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const uint2 w = *reinterpret_cast<const uint2*>(q);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int word = (int)(h ? w.y : w.x);
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(word, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
    v[4 * h] = a.x;
    v[4 * h + 1] = a.y;
    v[4 * h + 2] = b.x;
    v[4 * h + 3] = b.y;
  }
}

// Rows in use among the thread's R rows from row r on, as bits.
template <int R>
__device__ __forceinline__ uint32_t rows_in_use(const int32_t* m_indices, int64_t r) {
  uint32_t live = (1u << R) - 1u;
  if (m_indices) {
    live = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) live |= (m_indices[r + i] >= 0 ? 1u : 0u) << i;
  }
  return live;
}

// Workgroup (x, y): rows [128 x, 128 x + 128), gate and up tile y.
template <int R>
__global__ __launch_bounds__(kTileThreads<R>) void swiglu_bwd_kernel(SwigluBwdParams p) {
  __shared__ TileLds<R> lds;
  const int64_t row0 = (int64_t)blockIdx.x * kBlockK;
  const int tiles = p.inter / kBlockK, j = blockIdx.y, col0 = j * kBlockK;
  const int tid = threadIdx.x, r0 = (tid >> 4) * R, c0 = (tid & 15) * 8;
  const uint32_t live = rows_in_use<R>(p.m_indices, row0 + r0);
  if (!__syncthreads_or(live != 0)) return;
  float dg[R][8], du[R][8], act[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    float gate[8], up[8], da[8], gate_s = 0.0f, up_s = 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) gate[c] = up[c] = da[c] = 0.0f;
    if ((live >> i) & 1) {
      const int64_t r = row0 + r0 + i;
      const uint8_t* hq = p.hq + r * 2 * p.inter + col0 + c0;
      decode8(hq, gate);
      decode8(hq + p.inter, up);
      gate_s = p.hsf[j * p.ld_hsf + r];
      up_s = p.hsf[(tiles + j) * p.ld_hsf + r];
      const uint4 d = *reinterpret_cast<const uint4*>(p.dact + r * p.ld_dact + col0 + c0);
      const uint32_t b[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int c = 0; c < 8; ++c) da[c] = bf16_bits_to_f32((c & 1) ? b[c >> 1] >> 16 : b[c >> 1] & 0xFFFFu);
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float g = gate[c] * gate_s, u = up[c] * up_s;
      const Sigmoid sg = sigmoid(g);
      const float silu = g * sg.sig;
      act[i][c] = silu * u;
      du[i][c] = da[c] * silu;
      dg[i][c] = da[c] * u * silu_slope(gate[c], gate_s, g, sg);
    }
  }
  const int64_t ld = 2 * (int64_t)p.inter;
  tile_rows<R>(dg, p.dq + row0 * ld + col0, ld, p.dsf + j * p.ld_dsf + row0, live);
  tile_rows<R>(du, p.dq + row0 * ld + p.inter + col0, ld, p.dsf + (tiles + j) * p.ld_dsf + row0, live);
  float* dsft = p.dsft + (int64_t)blockIdx.x * p.ld_dsft + col0;
  tile_columns<R>(dg, lds, p.dqt + (int64_t)col0 * p.m_total + row0, p.m_total, dsft);
  tile_columns<R>(du, lds, p.dqt + (int64_t)(p.inter + col0) * p.m_total + row0, p.m_total, dsft + p.inter);
  if (p.aqt)
    tile_columns<R>(act, lds, p.aqt + (int64_t)col0 * p.m_total + row0, p.m_total,
                    p.asft + (int64_t)blockIdx.x * p.ld_asft + col0);
}

// Workgroup (x, y): rows [128 x, 128 x + 128), column tile y.
__global__ __launch_bounds__(kTileThreads<8>) void requant_t_kernel(RequantParams p) {
  __shared__ TileLds<8> lds;
  const int64_t row0 = (int64_t)blockIdx.x * kBlockK;
  const int col0 = blockIdx.y * kBlockK;
  const int tid = threadIdx.x, r0 = (tid >> 4) * 8, c0 = (tid & 15) * 8;
  const uint32_t live = rows_in_use<8>(p.m_indices, row0 + r0);
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + r0 + i;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[i][c] = 0.0f;
    if ((live >> i) & 1) {
      decode8(p.q + r * p.cols + col0 + c0, v[i]);
      const float s = p.sf[blockIdx.y * p.ld_sf + r];
#pragma unroll
      for (int c = 0; c < 8; ++c) v[i][c] *= s;
    }
  }
  if (!__syncthreads_or(live != 0)) return;
  tile_columns<8>(v, lds, p.qt + (int64_t)col0 * p.rows + row0, p.rows, p.sft + (int64_t)blockIdx.x * p.ld_sft + col0);
}

}  // namespace

hipError_t launch_swiglu_quant(const SwigluParams& p, bool pow2, hipStream_t stream) {
  const int gx = (p.inter / kBlockK + kTilesPerWave - 1) / kTilesPerWave;
  const int64_t total = (int64_t)p.groups * p.rows;
  int64_t gy = (16384 / kRowWaves + gx - 1) / gx;
  const int64_t need = (total + kRowWaves - 1) / kRowWaves;
  if (gy > need) gy = need;
  const dim3 grid(gx, (unsigned)(gy < 1 ? 1 : gy > 65535 ? 65535 : gy)), block(64 * kRowWaves);
  if (pow2) hipLaunchKernelGGL((swiglu_kernel<true, false>), grid, block, 0, stream, p);
  else if (p.hq) hipLaunchKernelGGL((swiglu_kernel<false, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((swiglu_kernel<false, false>), grid, block, 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(swiglu_bwd_kernel<4>, dim3(p.m_total / kBlockK, p.inter / kBlockK), dim3(kTileThreads<4>), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_requant_t(const RequantParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(requant_t_kernel, dim3(p.rows / kBlockK, p.cols / kBlockK), dim3(kTileThreads<8>), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
