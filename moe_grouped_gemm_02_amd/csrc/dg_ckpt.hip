// The experts' gated unit and its 8-bit activation checkpoint for gfx950:
// quantised forward, backward from the checkpoint, and the operands of the
// weight-gradient GEMMs (tiles of 128 rows of a column, transposed).

#include "dg_device.h"
#include "dg_moe_internal.h"
#include "dg_tile.h"

namespace dg {
namespace {

constexpr int kTilesPerWave = 8;
constexpr int kRowWaves = 4;

// 8 lanes own one 128-value tile of a row's gate and the same tile of its up
// half; a wave owns 8 tiles.  Block (x, y, g): tiles [8 x, 8 x + 8) of group g,
// row 4 y + its wave and every 4 gridDim.y rows on, up to the group's last row in
// use.  One read of h serves both the unit's output and the checkpoint, and
// nothing but codes and scales is written.  Bound by memory: 32768 rows x 2048
// read 0.26 GB and write 0.20 in 79 us (5.8 TB/s).  STREAMING: results larger than
// the L2s (79 us against 81.7 with plain stores).
template <bool POW2, bool CKPT, bool STREAMING>
__global__ __launch_bounds__(64 * kRowWaves) void swiglu_kernel(SwigluParams p) {
  const int tiles = p.inter / kBlockK;
  const int sub = threadIdx.x & 7;
  const int j = blockIdx.x * kTilesPerWave + ((threadIdx.x & 63) >> 3);
  if (j >= tiles) return;
  const int64_t g = blockIdx.z;
  const int rows = p.masked_m ? min(p.masked_m[g], p.rows) : p.rows;
  for (int64_t r = blockIdx.y * kRowWaves + (threadIdx.x >> 6); r < rows; r += gridDim.y * kRowWaves) {
    if (p.m_indices && p.m_indices[r] < 0) continue;
    const int64_t gr = g * p.rows + r;
    const int col = j * kBlockK + sub * 16;
    const uint16_t* h = p.h + gr * p.ld_h + col;
    const Lane16 gate = load16(h), up = load16(h + p.inter);
    float a[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float v = gate.at(i);
      a[i] = v * sigmoid(v).sig * up.at(i);
    }
    const float amax = amax16([&](int i) { return a[i]; });
    uint4 out;
    const int64_t sf_at = (g * tiles + j) * p.ld_sf + r;
    if constexpr (POW2) {
      const uint32_t e = ue8m0_exponent_f32(amax);
      const int up2 = 127 - (int)e;
      out = encode16([&](int i) { return __builtin_ldexpf(a[i], up2); });
      if (sub == 0) static_cast<uint8_t*>(p.sf)[sf_at] = (uint8_t)e;
    } else {
      const TileScale t = tile_scale(amax);
      out = encode16([&](int i) { return a[i] * t.inv; });
      if (sub == 0) static_cast<float*>(p.sf)[sf_at] = t.s;
    }
    store<STREAMING>(p.q + gr * p.inter + col, out);
    if constexpr (CKPT) {
      uint8_t* hq = p.hq + gr * 2 * p.inter + col;
      float* hsf = p.hsf + (g * 2 * tiles + j) * p.ld_hsf + r;
      float gs, us;
      store<STREAMING>(hq, encode_bf16_tile(gate, gs));
      store<STREAMING>(hq + p.inter, encode_bf16_tile(up, us));
      if (sub == 0) hsf[0] = gs, hsf[tiles * p.ld_hsf] = us;
    }
  }
}

// 8 codes as numbers.
__device__ __forceinline__ void decode8(uint2 w, float (&v)[8]) {
  typedef float v2f __attribute__((ext_vector_type(2)));
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

// What a thread reads of one tile: its 4 rows x 8 columns of gate and up codes
// and of dact, and the rows' scales.
struct SwigluBwdRaw {
  uint2 gate[4], up[4];
  uint4 da[4];
  float gate_s[4], up_s[4];
};

__device__ __forceinline__ void load_raw(const SwigluBwdParams& p, TileAt tile, SwigluBwdRaw& raw) {
  const int tiles = p.inter / kBlockK;
  const int64_t row = (int64_t)tile.row * kBlockK + (threadIdx.x >> 4) * 4;
  const int col = tile.col * kBlockK + (threadIdx.x & 15) * 8;
  const uint8_t* hq = p.hq + row * 2 * p.inter + col;
  const uint16_t* dact = p.dact + row * p.ld_dact + col;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    raw.gate[i] = load_streaming2(hq + (int64_t)i * 2 * p.inter);
    raw.up[i] = load_streaming2(hq + (int64_t)i * 2 * p.inter + p.inter);
    raw.da[i] = load_streaming4(dact + i * p.ld_dact);
  }
  load_floats<4>(p.hsf + tile.col * p.ld_hsf + row, raw.gate_s);
  load_floats<4>(p.hsf + (tiles + tile.col) * p.ld_hsf + row, raw.up_s);
}

// Workgroups walk over tiles of 128 rows x 128 gate columns and the same up
// columns, 32 workgroups of an XCD over its eighth of the tiles (row tiles
// fastest).  The checkpoint and dact are read once for all five code matrices.
// The three results of a tile stay in registers (96 of a thread) while their
// columns' maxima come together, so one workgroup fills a CU; the next tile is
// read while this one is quantised and written (158 us against 215 with a
// workgroup for each tile).  32768 rows x 2048 move 0.60 GB in 150 us (4.0 TB/s).
// Bound by vector instructions (53 for a pair of gate and up, busy 71 % of the
// time) and by what two waves on a SIMD leave open at the barriers: without any
// loads it takes 128 us, without stores 140.  Smaller tiles for two workgroups
// need more registers than there are (286 us).
constexpr int kBwdWorkgroups = 256;  // one for each CU

__global__ __launch_bounds__(kTileThreads<4>, 2) void swiglu_bwd_kernel(SwigluBwdParams p) {
  __shared__ TileLds<4, 3> lds;
  const int row_tiles = p.m_total / kBlockK, tiles = p.inter / kBlockK;
  const int all = row_tiles * tiles;
  // Workgroup b works on XCD b % 8.
  const int xcds = gridDim.x < 8 ? (int)gridDim.x : 8;
  const int xcd = blockIdx.x % xcds, mine = blockIdx.x / xcds, peers = ((int)gridDim.x - xcd + xcds - 1) / xcds;
  const int end = (int)((int64_t)all * (xcd + 1) / xcds);
  int t = (int)((int64_t)all * xcd / xcds) + mine;
  // The next tile of this workgroup with rows in use, from t on.
  auto seek = [&](TileUse& use) {
    for (; t < end; t += peers) {
      use = tile_use(p.m_indices ? p.m_indices + (int64_t)(t % row_tiles) * kBlockK : nullptr);
      if (use.any()) return;
    }
  };
  TileUse use;
  SwigluBwdRaw raw;
  seek(use);
  if (t < end) load_raw(p, {t % row_tiles, t / row_tiles}, raw);
  while (t < end) {
    const TileAt tile = {t % row_tiles, t / row_tiles};
    const uint32_t live = use.of_thread<4>();
    if (__ballot(live != 15u)) {  // rows not in use count as zeros, whatever they hold
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = (live >> i) & 1;
        raw.gate[i].x = in ? raw.gate[i].x : 0u, raw.gate[i].y = in ? raw.gate[i].y : 0u;
        raw.up[i].x = in ? raw.up[i].x : 0u, raw.up[i].y = in ? raw.up[i].y : 0u;
        raw.da[i].x = in ? raw.da[i].x : 0u, raw.da[i].y = in ? raw.da[i].y : 0u;
        raw.da[i].z = in ? raw.da[i].z : 0u, raw.da[i].w = in ? raw.da[i].w : 0u;
        raw.gate_s[i] = in ? raw.gate_s[i] : 0.0f, raw.up_s[i] = in ? raw.up_s[i] : 0.0f;
      }
    }
    float out[3][4][8];  // d gate, d up, and the unit's output
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float gate[8], up[8];
      decode8(raw.gate[i], gate);
      decode8(raw.up[i], up);
      const float gate_s = raw.gate_s[i], up_s = raw.up_s[i];
      const uint32_t b[4] = {raw.da[i].x, raw.da[i].y, raw.da[i].z, raw.da[i].w};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float da = bf16_bits_to_f32((c & 1) ? b[c >> 1] >> 16 : b[c >> 1] & 0xFFFFu);
        const float g = gate[c] * gate_s, u = up[c] * up_s;
        const Sigmoid sg = sigmoid(g);
        const float silu = g * sg.sig;
        out[0][i][c] = da * u * silu_slope(gate[c], gate_s, g, sg);
        out[1][i][c] = da * silu;
        out[2][i][c] = silu * u;
      }
    }
    t += peers;
    seek(use);
    if (t < end) load_raw(p, {t % row_tiles, t / row_tiles}, raw);
    const int64_t row0 = (int64_t)tile.row * kBlockK, ld = 2 * (int64_t)p.inter;
    const int col0 = tile.col * kBlockK;
    tile_rows<false>(out[0], p.dq + row0 * ld + col0, ld, p.dsf + tile.col * p.ld_dsf + row0, live);
    tile_rows<false>(out[1], p.dq + row0 * ld + p.inter + col0, ld, p.dsf + (tiles + tile.col) * p.ld_dsf + row0, live);
    uint8_t* dqt = p.dqt + (int64_t)col0 * p.m_total + row0;
    float* dsft = p.dsft + (int64_t)tile.row * p.ld_dsft + col0;
    const ColumnsTo to[3] = {
        {dqt, p.m_total, dsft},
        {dqt + (int64_t)p.inter * p.m_total, p.m_total, dsft + p.inter},
        {p.aqt ? p.aqt + (int64_t)col0 * p.m_total + row0 : nullptr, p.m_total, p.asft + (int64_t)tile.row * p.ld_asft + col0}};
    tile_columns<false>(out, lds, to);
  }
}

// Workgroup: one 128 x 128 tile, decoded, scaled and quantised again along its
// columns: read once, written once.  Bound by memory: 32768 x 7168 reads 0.23 GB
// and writes 0.23 in 83 us (5.6 TB/s).
__global__ __launch_bounds__(kTileThreads<8>) void requant_t_kernel(RequantParams p) {
  __shared__ TileLds<8> lds;
  const TileAt tile = tile_of_workgroup(p.rows / kBlockK, p.cols / kBlockK);
  const int64_t row0 = (int64_t)tile.row * kBlockK;
  const int col0 = tile.col * kBlockK;
  const int tid = threadIdx.x, r0 = (tid >> 4) * 8, c0 = (tid & 15) * 8;
  const TileUse use = tile_use(p.m_indices ? p.m_indices + row0 : nullptr);
  if (!use.any()) return;
  const uint32_t live = use.of_thread<8>();
  uint2 q[8];
  float s[8], vs[1][8][8];
  auto& v = vs[0];
  const uint8_t* from = p.q + (row0 + r0) * p.cols + col0 + c0;
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = load_streaming2(from + (int64_t)i * p.cols);
  load_floats<8>(p.sf + tile.col * p.ld_sf + row0 + r0, s);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool in = (live >> i) & 1;
    decode8(in ? q[i] : make_uint2(0, 0), v[i]);
    const float scale = in ? s[i] : 0.0f;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[i][c] *= scale;
  }
  const ColumnsTo to[1] = {{p.qt + (int64_t)col0 * p.rows + row0, p.rows, p.sft + (int64_t)tile.row * p.ld_sft + col0}};
  tile_columns<true>(vs, lds, to);
}

}  // namespace

hipError_t launch_swiglu_quant(const SwigluParams& p, bool pow2, hipStream_t stream) {
  const int gx = (p.inter / kBlockK + kTilesPerWave - 1) / kTilesPerWave;
  // Up to 16384 workgroups in all, most rows a wave of their own (32768 x 2048: 79
  // us, and 89.5 with 4096); each group its share of them.  A masked layout, whose
  // rows are mostly not in use when the batch is small, has fewer, since workgroups
  // that find nothing to do cost more than they bring: 1024 of a short one (32
  // groups of 128 rows x 2048, 4 % in use: 4.4 us against 6.3 with 4096; all in use:
  // a call in 8.8 against 8.5), 8192 of a tall one (32 groups of 1024 rows, 4 % in
  // use: a call in 7.6, and 10.2 with 16384; all in use: 44.3 and 42.9).
  const bool short_layout = (int64_t)p.groups * p.rows * p.inter <= (int64_t)16 << 20;
  const int64_t most = !p.masked_m ? 16384 : short_layout ? 1024 : 8192;
  const int64_t share = (most + (int64_t)gx * p.groups - 1) / ((int64_t)gx * p.groups);
  const int64_t need = ((int64_t)p.rows + kRowWaves - 1) / kRowWaves;
  const dim3 grid(gx, (unsigned)(need < share ? need : share), p.groups), block(64 * kRowWaves);
  const bool streaming = (int64_t)p.groups * p.rows * p.inter > (int64_t)32 << 20;
  auto go = [&](auto pow, auto ckpt, auto large) {
    hipLaunchKernelGGL((swiglu_kernel<decltype(pow)::value, decltype(ckpt)::value, decltype(large)::value>), grid, block,
                       0, stream, p);
  };
  using std::false_type, std::true_type;
  if (pow2) streaming ? go(true_type{}, false_type{}, true_type{}) : go(true_type{}, false_type{}, false_type{});
  else if (p.hq) streaming ? go(false_type{}, true_type{}, true_type{}) : go(false_type{}, true_type{}, false_type{});
  else streaming ? go(false_type{}, false_type{}, true_type{}) : go(false_type{}, false_type{}, false_type{});
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdParams& p, hipStream_t stream) {
  const int tiles = p.m_total / kBlockK * (p.inter / kBlockK);
  hipLaunchKernelGGL(swiglu_bwd_kernel, dim3(tiles < kBwdWorkgroups ? tiles : kBwdWorkgroups), dim3(kTileThreads<4>), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_requant_t(const RequantParams& p, hipStream_t stream) {
  const int tiles = p.rows / kBlockK * (p.cols / kBlockK);
  hipLaunchKernelGGL(requant_t_kernel, dim3(tiles), dim3(kTileThreads<8>), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
