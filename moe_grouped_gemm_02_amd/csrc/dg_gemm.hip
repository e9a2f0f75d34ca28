// Host side of the FP8 GEMMs: the choice of tile and work division, and the
// launch of the kernel instances (the kernel itself is in dg_gemm_kernel.h).

#include <stdlib.h>
#include <string.h>

#include <algorithm>

#include "dg_gemm_kernel.h"

namespace dg {

namespace {

struct Variant {
  int bm, bn, threads;
};
constexpr Variant kVariants[] = {
    {TileP256::BM, TileP256::BN, TileP256::kThreads},
    {TileP128::BM, TileP128::BN, TileP128::kThreads},
    {TileD128::BM, TileD128::BN, TileD128::kThreads},
    {TileD64::BM, TileD64::BN, TileD64::kThreads},
    {TileS64::BM, TileS64::BN, TileS64::kThreads},
    {TileW128::BM, TileW128::BN, TileW128::kThreads},
    {TileP128w8::BM, TileP128w8::BN, TileP128w8::kThreads},
    {TileS64w8::BM, TileS64w8::BN, TileS64w8::kThreads},
    {TileW128w16::BM, TileW128w16::BN, TileW128w16::kThreads},
    {TileV128::BM, TileV128::BN, TileV128::kThreads},
    {TileV128w8::BM, TileV128w8::BN, TileV128w8::kThreads},
    {TileP160::BM, TileP160::BN, TileP160::kThreads},
};
constexpr int kNumVariants = sizeof(kVariants) / sizeof(kVariants[0]);

template <class T, int LAYOUT, int SF>
hipError_t launch_one(const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  if constexpr (LAYOUT != kContiguous) {  // contiguous tiles may take two passes: data-parallel only
    if (s.stream_k) {
      hipLaunchKernelGGL((gemm_kernel<T, LAYOUT, true, SF>), dim3(grid), dim3(T::kThreads), 0, stream, p, s);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((gemm_kernel<T, LAYOUT, false, SF>), dim3(grid), dim3(T::kThreads), 0, stream, p, s);
  return hipGetLastError();
}

// Dense GEMM with MN-major operands (p.majors: kAMajorMN | kBMajorMN).
template <class T, int MAJ, int SF>
hipError_t launch_majors_one(const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  if (s.stream_k)
    hipLaunchKernelGGL((gemm_kernel<T, kDense, true, SF, MAJ>), dim3(grid), dim3(T::kThreads), 0, stream, p, s);
  else
    hipLaunchKernelGGL((gemm_kernel<T, kDense, false, SF, MAJ>), dim3(grid), dim3(T::kThreads), 0, stream, p, s);
  return hipGetLastError();
}

template <class T, int SF>
hipError_t launch_majors_sf(const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  switch (p.majors) {
    case kAMajorMN: return launch_majors_one<T, kAMajorMN, SF>(p, s, grid, stream);
    case kBMajorMN: return launch_majors_one<T, kBMajorMN, SF>(p, s, grid, stream);
    case kAMajorMN | kBMajorMN: return launch_majors_one<T, kAMajorMN | kBMajorMN, SF>(p, s, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

template <class T>
hipError_t launch_majors(const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  return p.sf_ue8m0 ? launch_majors_sf<T, kScaleUE8M0>(p, s, grid, stream)
                    : launch_majors_sf<T, kScaleF32>(p, s, grid, stream);
}

template <class T, int SF>
hipError_t launch_layout(int layout, const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  switch (layout) {
    case kDense: return launch_one<T, kDense, SF>(p, s, grid, stream);
    case kContiguous: return launch_one<T, kContiguous, SF>(p, s, grid, stream);
    default: return launch_one<T, kMasked, SF>(p, s, grid, stream);
  }
}

// K-grouped layout: data-parallel, row scales on B.
template <class T>
hipError_t launch_kgrouped(const GemmParams& p, const Schedule& s, int grid, hipStream_t stream) {
  hipLaunchKernelGGL((gemm_kernel<T, kKGrouped, false, kScaleRowB>), dim3(grid), dim3(T::kThreads), 0, stream, p, s);
  return hipGetLastError();
}

// Ceiling division of a >= 0 by b > 0 that cannot overflow.
int cdiv(int a, int b) { return a / b + (a % b != 0); }
int64_t cdiv64(int64_t a, int64_t b) { return a / b + (a % b != 0); }

constexpr int smallest_tile_dim(bool rows) {
  int v = 1 << 30;
  for (const Variant& t : kVariants) v = std::min(v, rows ? t.bm : t.bn);
  return v;
}

// Stream-K partial slots are addressed with 32-bit offsets: 2 * grid slots of
// at most 256 KB stay below 2^31 bytes with this cap.
constexpr int kMaxStreamKGrid = 1024;

int forced_variant() {
  // DG_FORCE_CONFIG="variant[:division[:k_rotate]]" overrides the heuristic
  // (sweeps and tests); division 0 = data-parallel, 1 = equal stream-K runs,
  // S >= 2 = S parts per tile.
  const char* e = getenv("DG_FORCE_CONFIG");
  if (!e || !*e) return -1;
  return atoi(e);
}

int forced_stream_k() {  // second field, -1 when absent
  const char* e = getenv("DG_FORCE_CONFIG");
  if (!e || !*e) return -1;
  const char* c = strchr(e, ':');
  return c ? std::max(0, atoi(c + 1)) : -1;
}

int forced_rotate() {  // third field: 0 or 1, -1 when absent
  const char* e = getenv("DG_FORCE_CONFIG");
  if (!e || !*e) return -1;
  const char* c = strchr(e, ':');
  if (!c) return -1;
  c = strchr(c + 1, ':');
  return c ? (atoi(c + 1) != 0) : -1;
}

}  // namespace

bool plannable(int layout, int m, int n, int groups) {
  if (m < 0 || n < 0 || groups < 1) return false;
  const int64_t gmul = (layout == kMasked || layout == kKGrouped) ? groups : 1;
  const int64_t tiles = cdiv64(m, smallest_tile_dim(true)) * cdiv64(n, smallest_tile_dim(false));  // < 2^50
  return tiles <= ((1LL << 31) - 1) / gmul;
}

bool variant_quantises_output(int variant) {
  return variant >= 0 && variant < kNumVariants && kVariants[variant].bn % 128 == 0;
}

GemmConfig choose_config(int layout, int m, int n, int k, int groups, int num_cus, int expected_m, bool qout,
                         bool narrow_ok) {
  // m: dense M, contiguous M_total, masked M_max.  The rules below come from
  // sweeps over tile variants on the benchmark shapes.  For the masked
  // layout a host hint of the typical valid rows per group replaces M_max in
  // the choice of tile (the launch itself still covers M_max rows per group,
  // skipping empty tiles on the device).
  const int nkb = k / kBlockK;
  const bool hinted = layout == kMasked && expected_m > 0 && expected_m < m;
  const int rows = hinted ? expected_m : m;
  const int gmul = (layout == kMasked || layout == kKGrouped) ? groups : 1;
  // Tile counts in 64 bits: with plannable() shapes every count fits an int,
  // but the products below (10 x tiles, tiles x parts) need not.
  auto tiles_of = [&](int bm, int bn) { return (int64_t)cdiv(rows, bm) * gmul * cdiv(n, bn); };
  int v;
  if (rows <= 128) {
    // Decode-sized M: the launch streams B once.  128x128 tiles (8 waves)
    // when they alone keep most CUs busy or K is long, else 64x64 tiles.
    const int64_t t128 = tiles_of(128, 128);
    v = (rows > 64 && (10 * t128 >= 7 * num_cus || nkb >= 64)) ? 6 : 4;
  } else if (tiles_of(256, 256) >= num_cus / 2) {
    v = 0;
    // Non-power-of-two BLOCK_N: when 256 x 256 tiles fill under 70% of the
    // CUs but one round of 256 x 160 tiles fills at least 80% of them, the
    // narrower tile runs data-parallel in one wave (measured 4096 x 2112 x
    // 7168: 103.4 us against 113.6 us for 256 x 256 tiles in equal
    // stream-K runs).  Not for the masked layout, whose tile count is only
    // a hint (4 x 1024 x 4096 x 7168 with about 512 valid rows per group:
    // 177 us with 256 x 160 tiles against 133 us with 256 x 256).
    const int64_t t256 = tiles_of(256, 256), t160 = tiles_of(256, 160);
    if (narrow_ok && !qout && (layout == kDense || layout == kContiguous) && 10 * t256 < 7 * (int64_t)num_cus && 5 * t160 >= 4 * (int64_t)num_cus && t160 <= num_cus) v = 11;
  } else {
    // Mid-size M (e.g. 1024 rows in all): 128-row tiles, 256 columns wide
    // unless 128 columns fill the CUs' last round better (measured on the
    // pages' all-valid masked rows: 1024x7168x2048 39.8 -> 31.1 us with
    // 128x256, 1024x4096x7168 58.5 -> 53.1 us with 128x128).
    auto fill = [&](int64_t t) { return (double)t / (double)(cdiv64(t, num_cus) * num_cus); };
    v = fill(tiles_of(128, 256)) >= fill(tiles_of(128, 128)) ? 5 : 6;
  }
  // A quantised output needs whole 128-column blocks per tile: the 64-wide
  // decode tiles give way to the 128x128 one.
  const bool widened = qout && kVariants[v].bn % 128 != 0;
  if (widened) v = 6;
  const int fv = forced_variant();
  if (fv >= 0 && fv < kNumVariants) v = fv;
  GemmConfig c{};
  c.variant = v;
  c.bm = kVariants[v].bm;
  c.bn = kVariants[v].bn;
  const int m_tiles = cdiv(m, c.bm) * gmul;
  const int n_tiles = cdiv(n, c.bn);
  c.tiles = m_tiles * n_tiles;
  // Work division.  Tiles that leave most CUs idle get their K ranges cut:
  // decode-sized tiles into S equal parts (one part per workgroup), larger
  // tiles with long K into equal runs of iterations over all CUs.  The
  // estimate uses the hinted rows for the masked layout.
  const int64_t est = tiles_of(c.bm, c.bn);
  int sk = 0;  // 0: data-parallel, 1: equal runs, S >= 2: S parts per tile
  if (layout != kContiguous && layout != kKGrouped && nkb >= 2 && 10 * est < 7 * num_cus) {
    // K parts for 128-row (or smaller) tiles up to 1024 rows in all; beyond
    // that, or when parts do not pay, equal runs for long K.
    if (c.bm <= 128 && rows <= 1024) {
      // Shorter parts for the 128x128 tiles that stand in for 64-wide ones
      // (quantised output): fewer tiles, so more parts (64x4096x7168 fused:
      // 27.5 -> 24.2 us with 8 parts instead of 3).
      const int min_slices = (c.bm * c.bn >= 128 * 128 && !widened) ? 16 : 8;
      int parts = (int)std::min<int64_t>(num_cus / std::max<int64_t>(est, 1), nkb / min_slices);
      // Two 64x64 workgroups share a CU: at least 4 parts where 2 x CUs hold
      // them (128x4096x7168: 20.4 -> 19.5 us with 4 parts on 512 workgroups
      // instead of 2 on 256; 64x7168x16384: 36.8 -> 33.8 us).
      if (v == 4 || v == 7)
        parts = std::max(parts, (int)std::min<int64_t>({4, 2 * num_cus / std::max<int64_t>(est, 1), nkb / min_slices}));
      if (c.bm * c.bn < 128 * 128) parts = std::min(parts, 6);  // 64x2112x7168: 6 parts 3% faster than 4
      // A fixup costs a few microseconds; short K ranges are not worth
      // cutting (64x7168x2048: 11.6 us in 2 parts, 10.2 us whole).
      if (nkb < 24) parts = 1;
      if (parts >= 2) sk = parts;
    }
    // Equal runs for long K - except the masked layout's 256 x 256 tiles,
    // whose valid count is only known on the device: there one data-parallel
    // round measured faster (4 x 1024 x 4096 x 7168 with 1841 valid rows, 160
    // valid tiles: 116.9 us against 132.5 us in equal runs).
    if (sk == 0 && rows > 128 && est * nkb >= 24LL * num_cus && !(layout == kMasked && c.bm == 256)) sk = 1;
  }
  const int fs = forced_stream_k();
  if (fs >= 0) sk = fs;
  if (layout == kContiguous || layout == kKGrouped || nkb < 2) sk = 0;
  if (sk >= 2) sk = std::min(sk, nkb);
  c.stream_k = sk > 0 ? 1 : 0;
  c.sk_split = sk >= 2 ? sk : 0;
  // Aligned parts: one workgroup per part, the grid a multiple of 8 so that
  // the XCD-contiguous numbering of runs spreads them evenly over the XCDs.
  // The 64x64 tiles take 72 KB of LDS, so two workgroups share a CU; with
  // more tiles than CUs a grid of two per CU gives each SIMD a second wave
  // (measured 64x32768x512: 11.0 -> 9.5 us, 64x24576x1536: 16.0 -> 14.5 us).
  // The same holds for their K parts.
  const int per_cu = (v == 4 || v == 7) ? 2 : 1;
  const int cap = std::min(num_cus * per_cu, kMaxStreamKGrid);
  const int64_t runs = c.sk_split ? (int64_t)c.tiles * c.sk_split : cap;
  const int64_t slots = c.sk_split ? runs : 2 * runs;
  c.grid = !c.stream_k ? std::max(1, std::min(c.tiles, num_cus * per_cu))
           : (int)std::min<int64_t>(cap, cdiv64(runs, 8) * 8);
  // Partial slots must stay 32-bit addressable, and every tile needs an
  // arrival counter in the workspace's fixed counter region.
  if (c.stream_k && (slots * c.bm * c.bn * 4 >= (1LL << 31) || c.tiles > kStreamKCounters)) {
    c.stream_k = c.sk_split = 0;
    c.grid = std::max(1, std::min(c.tiles, num_cus));
  }
  c.sk_slots = c.stream_k ? (int)slots : 0;
  c.group_m = 8;
  // Rotated K walks for the decode-sized tiles when the weight rows are a
  // multiple of 16 KiB apart (see the kernel's K walk).  The 256x256 tile
  // keeps every tile on the same slice: its operands are shared through L2
  // by the tiles of a raster group, and rotation would spread that working
  // set over many slices.
  c.k_rotate = (c.bm * c.bn < 256 * 256 && k % 16384 == 0) ? 1 : 0;
  const int fr = forced_rotate();
  if (fr >= 0) c.k_rotate = fr;
  return c;
}

size_t workspace_bytes_for(const GemmConfig& cfg, int layout, int m, int n, int groups) {
  (void)layout; (void)m; (void)n; (void)groups;
  if (!cfg.stream_k) return 0;
  // The fixed counter region, then the fp32 partial tiles.
  return kStreamKCounterBytes + (size_t)cfg.sk_slots * cfg.bm * cfg.bn * sizeof(float);
}

Schedule schedule_of(int layout, const GemmParams& p, const GemmConfig& cfg) {
  Schedule s{};
  s.n_tiles = cdiv(p.n, cfg.bn);
  s.m_tiles = layout == kKGrouped ? cdiv(p.m, cfg.bm) : cfg.tiles / s.n_tiles;  // K-grouped: per group
  s.tiles = cfg.tiles;
  s.stream_k = cfg.stream_k;
  s.sk_split = cfg.sk_split;
  s.sk_slots = cfg.sk_slots;
  s.group_m = cfg.group_m;
  s.k_rotate = cfg.k_rotate;
  return s;
}

hipError_t launch_gemm(int layout, const GemmParams& p0, const GemmConfig& cfg,
                       hipStream_t stream) {
  GemmParams p = p0;
  const Schedule s = schedule_of(layout, p, cfg);
  if (cfg.stream_k) p.counters = reinterpret_cast<int*>(p.workspace);
  if (layout == kKGrouped) {
    switch (cfg.variant) {
      case 0: return launch_kgrouped<TileP256>(p, s, cfg.grid, stream);
      case 4: return launch_kgrouped<TileS64>(p, s, cfg.grid, stream);
      case 5: return launch_kgrouped<TileW128>(p, s, cfg.grid, stream);
      case 6: return launch_kgrouped<TileP128w8>(p, s, cfg.grid, stream);
      default: return hipErrorInvalidValue;
    }
  }
  if (p.majors) {  // MN-major operands: dense layout, the dense heuristic's tiles
    if (layout != kDense) return hipErrorInvalidValue;
    switch (cfg.variant) {
      case 0: return launch_majors<TileP256>(p, s, cfg.grid, stream);
      case 4: return launch_majors<TileS64>(p, s, cfg.grid, stream);
      case 5: return launch_majors<TileW128>(p, s, cfg.grid, stream);
      case 6: return launch_majors<TileP128w8>(p, s, cfg.grid, stream);
      default: return hipErrorInvalidValue;
    }
  }
  if (p.sf_ue8m0) {  // UE8M0 instances: the tiles the heuristic picks
    switch (cfg.variant) {
      case 0: return launch_layout<TileP256, kScaleUE8M0>(layout, p, s, cfg.grid, stream);
      case 1: return launch_layout<TileP128, kScaleUE8M0>(layout, p, s, cfg.grid, stream);
      case 4: return launch_layout<TileS64, kScaleUE8M0>(layout, p, s, cfg.grid, stream);
      case 6: return launch_layout<TileP128w8, kScaleUE8M0>(layout, p, s, cfg.grid, stream);
      case 5: return launch_layout<TileW128, kScaleUE8M0>(layout, p, s, cfg.grid, stream);
      default: return hipErrorInvalidValue;
    }
  }
  switch (cfg.variant) {
    case 0: return launch_layout<TileP256, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 1: return launch_layout<TileP128, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 2: return launch_layout<TileD128, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 3: return launch_layout<TileD64, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 4: return launch_layout<TileS64, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 5: return launch_layout<TileW128, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 6: return launch_layout<TileP128w8, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 7: return launch_layout<TileS64w8, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 8: return launch_layout<TileW128w16, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 9: return launch_layout<TileV128, kScaleF32>(layout, p, s, cfg.grid, stream);
    case 10: return launch_layout<TileV128w8, kScaleF32>(layout, p, s, cfg.grid, stream);
    default: return launch_layout<TileP160, kScaleF32>(layout, p, s, cfg.grid, stream);
  }
}

}  // namespace dg
