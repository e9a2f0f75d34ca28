// Exchange between token rows and expert rows for gfx950: the row plan (a
// stable counting sort of the routed entries by expert), the dispatch into
// quantised expert rows, the weighted combine and its gradient.

#include "dg_device.h"
#include "dg_moe_internal.h"
#include "dg_tile.h"

namespace dg {
namespace {

// ------------------------------------------------------------------- plan --

// A stable counting sort.  Blocks of 1024 entries count their experts (one
// launch) and place their entries (another): the rank of an entry is the count
// of its expert in the blocks before, in the waves before, and in the lanes
// before, which a ballot for each bit of the expert's number tells.  The counts of
// the blocks before are added up by each block, or, where there are many, by a
// launch in between.  Up to 4096
// entries one workgroup does it all in one launch (1024 entries of 32 experts:
// 4.7 us, against 1.3 + 4.7 in two launches).  Both are a chain of reads and
// barriers, not a stream: 131072 entries of 4 experts take 3.0 + 4.8 us for 2 MB.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kOnePlanEntries = 4096;
constexpr int kOnePlanRows = 1 << 15;  // what one workgroup can fill in about as long as it sorts

int plan_blocks(int64_t entries) {
  const int64_t b = (entries + kPlanThreads - 1) / kPlanThreads;
  return (int)(b > 0 ? b : 1);
}

// Local expert of an entry, or -1.
__device__ __forceinline__ int local_of(int64_t i, const PlanParams& p) {
  const int id = i < p.entries ? p.ids[i] : -1;
  const int64_t g = (int64_t)id - p.first;
  return id >= 0 && g >= 0 && g < p.groups ? (int)g : -1;
}

// Lanes of the wave with the same local expert as this one (any, if it has none).
__device__ __forceinline__ uint64_t same_expert(int g, int groups) {
  uint64_t same = __ballot(g >= 0);
  for (int bit = 1; bit < groups; bit <<= 1) {
    const uint64_t ones = __ballot(g & bit);
    same &= (g & bit) ? ones : ~ones;
  }
  return same;
}

// Counts the experts of each block's 1024 entries.
__global__ __launch_bounds__(kPlanThreads) void plan_count_kernel(PlanParams p) {
  __shared__ int count[kMaxLocalExperts];
  const int tid = threadIdx.x;
  const int g = local_of((int64_t)blockIdx.x * kPlanThreads + tid, p);
  if (tid < p.groups) count[tid] = 0;
  const uint64_t same = same_expert(g, p.groups);
  __syncthreads();
  if (g >= 0 && __ffsll((unsigned long long)same) - 1 == (tid & 63)) atomicAdd(&count[g], __popcll(same));
  __syncthreads();
  if (tid < p.groups) p.hist[(int64_t)blockIdx.x * p.groups + tid] = count[tid];
}

// Replaces each block's counts by their sums over the blocks before and puts the
// groups' totals behind the last block's.  Workgroup: 2^shift groups, whose
// columns of counts are cut into as many parts as there are threads for.
constexpr int kScanShift = 4;

__global__ __launch_bounds__(kPlanThreads) void plan_scan_kernel(PlanParams p, int shift) {
  __shared__ int sums[kPlanThreads];
  const int tid = threadIdx.x, part = tid >> shift, parts = kPlanThreads >> shift;
  const int col = (blockIdx.x << shift) + (tid & ((1 << shift) - 1));
  const int per = (p.blocks + parts - 1) / parts;
  const int lo = min(part * per, p.blocks), hi = min(lo + per, p.blocks);
  const bool in = col < p.groups;
  int32_t* const hist = p.hist + (in ? col : 0);
  // Eight counts at a time, so that their reads are in flight together.
  auto read8 = [&](int b, int (&c)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) c[u] = in && b + u < hi ? hist[(int64_t)(b + u) * p.groups] : 0;
  };
  int sum = 0, c[8];
  for (int b = lo; b < hi; b += 8) {
    read8(b, c);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum += c[u];
  }
  sums[tid] = sum;
  __syncthreads();
  for (int off = 1 << shift; off < kPlanThreads; off <<= 1) {
    const int other = tid >= off ? sums[tid - off] : 0;
    __syncthreads();
    sums[tid] += other;
    __syncthreads();
  }
  int before = sums[tid] - sum;
  if (!in) return;
  for (int b = lo; b < hi; b += 8) {
    read8(b, c);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (b + u < hi) hist[(int64_t)(b + u) * p.groups] = before;
      before += c[u];
    }
  }
  if (part == parts - 1) hist[(int64_t)p.blocks * p.groups] = before;
}

// Places the entries and fills the index arrays of the layout's rows.  ONE: one
// workgroup, which counts the entries itself; otherwise block b places entries
// [1024 b, 1024 b + 1024) with the counts of all blocks or their sums (blocks past
// the last entry help with the rows alone).
template <bool ONE>
__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanParams p) {
  __shared__ int start[kMaxLocalExperts + 1];  // first row of each group
  __shared__ int count[kMaxLocalExperts];      // entries of each group
  __shared__ int base[kMaxLocalExperts];       // of them, those placed before
  __shared__ uint16_t per_wave[kPlanWaves][kMaxLocalExperts];
  __shared__ uint32_t totals[kPlanWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first_chunk = ONE ? 0 : blockIdx.x, chunks = ONE ? (p.entries + kPlanThreads - 1) / kPlanThreads : blockIdx.x + 1;
  int g = local_of((int64_t)first_chunk * kPlanThreads + tid, p);
  if (tid < p.groups) count[tid] = base[tid] = 0;
  __syncthreads();
  if constexpr (ONE) {
    if (g >= 0) atomicAdd(&count[g], 1);
    for (int c = 1; c < chunks; ++c) {
      const int e = local_of((int64_t)c * kPlanThreads + tid, p);
      if (e >= 0) atomicAdd(&count[e], 1);
    }
  } else {
    if (p.scanned) {
      if (tid < p.groups) {
        count[tid] = p.hist[(int64_t)p.blocks * p.groups + tid];
        if (blockIdx.x < p.blocks) base[tid] = p.hist[(int64_t)blockIdx.x * p.groups + tid];
      }
    } else {
      const int before = blockIdx.x * p.groups, all = p.blocks * p.groups;
      for (int i = tid; i < all; i += kPlanThreads) {
        const int v = p.hist[i], e = i % p.groups;
        atomicAdd(&count[e], v);
        if (i < before) atomicAdd(&base[e], v);
      }
    }
  }
  __syncthreads();
  // Starts of the groups: exclusive sums of their sizes.
  {
    uint32_t size = 0;
    if (tid < p.groups) size = p.masked ? p.m_max : ((uint32_t)count[tid] + kBlockK - 1) / kBlockK * kBlockK;
    uint32_t sum = size;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t other = __shfl_up(sum, off, 64);
      if (lane >= off) sum += other;
    }
    if (lane == 63) totals[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += totals[w];
    const uint32_t limit = (uint32_t)p.layout_rows;
    if (tid < p.groups) {
      start[tid] = (int)umin(sum - size, limit);
      if (tid == p.groups - 1) start[p.groups] = (int)umin(sum, limit);
    }
    __syncthreads();
  }

  for (int c = first_chunk; c < chunks; ++c) {
    const int64_t i = (int64_t)c * kPlanThreads + tid;
    if (c != first_chunk) g = local_of(i, p);
    for (int k = tid; k < kPlanWaves * p.groups; k += kPlanThreads) per_wave[k / p.groups][k % p.groups] = 0;
    const uint64_t same = same_expert(g, p.groups);
    const int ahead = __popcll(same & ((1ull << lane) - 1ull));
    __syncthreads();
    if (g >= 0 && ahead == 0) per_wave[wave][g] = (uint16_t)__popcll(same);
    __syncthreads();
    if (i < p.entries) {
      int row = -1;
      if (g >= 0) {
        int rank = base[g] + ahead;
#pragma unroll
        for (int w = 0; w < kPlanWaves; ++w) rank += w < wave ? per_wave[w][g] : 0;
        const int64_t at = (int64_t)start[g] + rank;
        if (at < (p.masked ? (int64_t)start[g] + p.m_max : p.layout_rows)) {
          row = (int)at;
          p.src[row] = (int)i;
        }
      }
      p.rows[i] = row;
    }
    if (ONE && c + 1 < chunks) {
      __syncthreads();
      if (tid < p.groups)
        for (int w = 0; w < kPlanWaves; ++w) base[tid] += per_wave[w][tid];
      __syncthreads();
    }
  }

  for (int64_t r = (int64_t)blockIdx.x * kPlanThreads + tid; r < p.layout_rows; r += (int64_t)gridDim.x * kPlanThreads) {
    int lo = 0;  // the last group that starts at or before row r
    if (p.masked) {
      lo = (int)divided((uint32_t)r, p.by_m_max);
    } else {
      int hi = p.groups;
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= r) lo = mid;
        else hi = mid;
      }
    }
    const bool used = r - start[lo] < count[lo];
    if (!used) p.src[r] = -1;
    if (p.m_indices) p.m_indices[r] = used ? lo : -1;
  }
  if (blockIdx.x == 0) {
    if (p.k_offsets)
      for (int e = tid; e <= p.groups; e += kPlanThreads) p.k_offsets[e] = start[e];
    if (p.masked_m && tid < p.groups) p.masked_m[tid] = count[tid] < p.m_max ? count[tid] : p.m_max;
  }
}

// --------------------------------------------------------------- dispatch --

// Row-wise gather and quantise, the mapping of the plain activation
// quantiser: 8 lanes own a 128-value tile, a wave owns 8 tiles of a row and
// ROWS rows at a time, so that their gathered loads are in flight together; which
// rows and tokens is the same for the whole wave and kept in scalar registers.
// A token's rows are in different groups, far apart in the walk, so each row of
// the result is a read and a quantisation of its own: 32768 rows x 7168 of 16384
// tokens read 0.45 GB, twice what the tokens hold, and write 0.23 in 107 us (6.3
// TB/s); the more of a token's choices are in the layout, the more is read again.
// Rows walked in token order measured the same (124 us against 125 at the time), 16
// lanes a tile lost (135 and more).
constexpr int kTilesPerWave = 8;
constexpr int kRowWaves = 4;

template <bool POW2, int ROWS>
__global__ __launch_bounds__(64 * kRowWaves) void dispatch_kernel(DispatchParams p) {
  const int tiles_per_row = p.cols / kBlockK;
  const uint32_t total_rows = (uint32_t)p.groups * (uint32_t)p.rows, entries = (uint32_t)(p.tokens * p.topk);
  const int lane = threadIdx.x & 63, sub = lane & 7;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = blockIdx.x * kTilesPerWave + (lane >> 3);
  const bool in = j < tiles_per_row;
  const int col = j * kBlockK + sub * 16;
  const uint32_t step = gridDim.y * kRowWaves * ROWS;
  for (uint32_t r0 = (blockIdx.y * kRowWaves + wave) * ROWS; r0 < total_rows; r0 += step) {
    uint32_t entry = ~0u;
    if (lane < ROWS && r0 + lane < total_rows) entry = (uint32_t)p.src[r0 + lane];
    const uint64_t rows = __ballot(entry < entries);
    if (rows == 0) continue;
    Lane16 x[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const uint32_t token = divided(lane_value(entry, u), p.by_topk);
      if (in && ((rows >> u) & 1)) x[u] = load16(p.x + (int64_t)token * p.ld_x + col);
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      if (!in || !((rows >> u) & 1)) continue;
      const uint32_t row = r0 + u, g = divided(row, p.by_rows), r = row - g * (uint32_t)p.rows;
      const int64_t sf_at = ((int64_t)g * tiles_per_row + j) * p.ld_sf + r;
      uint4* to = reinterpret_cast<uint4*>(p.q + (int64_t)row * p.cols + col);
      if constexpr (POW2) {
        uint32_t e;
        const uint4 q = encode_bf16_tile_pow2(x[u], e);
        store<ROWS == 4>(to, q);
        if (sub == 0) static_cast<uint8_t*>(p.sf)[sf_at] = (uint8_t)e;
      } else {
        float s;
        const uint4 q = encode_bf16_tile(x[u], s);
        store<ROWS == 4>(to, q);
        if (sub == 0) static_cast<float*>(p.sf)[sf_at] = s;
      }
    }
  }
}

// ---------------------------------------------------------------- combine --

// Workgroup (x, y, z): 2048 columns, 8 a thread, of token x (past those of a smaller
// z): one pass over the rows, sums in float32 registers, the only rounding at the
// end.  Bound by the reads: 32110 rows x 7168 into 4096 tokens in 95 us, 0.46 GB
// read and 0.06 written (5.5 TB/s).
constexpr int kCombineThreads = 256;

__global__ __launch_bounds__(kCombineThreads) void combine_kernel(CombineParams p) {
  const int64_t t = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  if (t >= p.tokens) return;
  const int col = (blockIdx.y * kCombineThreads + threadIdx.x) * 8;
  if (col >= p.cols) return;
  float acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.0f;
  for (int j = 0; j < p.topk; ++j) {
    const int r = p.rows[t * p.topk + j];
    if (r < 0 || r >= p.total_rows) continue;
    const float w = p.weights ? p.weights[t * p.topk + j] : 1.0f;
    const uint4 v = load_streaming4(p.d + (int64_t)r * p.ld_d + col);
    const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      acc[2 * c] = fmaf(w, bf16_bits_to_f32(b[c] & 0xFFFFu), acc[2 * c]);
      acc[2 * c + 1] = fmaf(w, bf16_bits_to_f32(b[c] >> 16), acc[2 * c + 1]);
    }
  }
  auto bf = [](float f) { return f == f ? f32_to_bf16_rne(f) : 0x7FC0u; };
  uint32_t o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = bf(acc[2 * c]) | (bf(acc[2 * c + 1]) << 16);
  *reinterpret_cast<uint4*>(p.y + t * p.ld_y + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

// 8 columns of dy and d multiplied and added to a sum.
__device__ __forceinline__ float add_dot8(uint4 a, uint4 b, float sum) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    sum = fmaf(bf16_bits_to_f32(x[c] & 0xFFFFu), bf16_bits_to_f32(y[c] & 0xFFFFu), sum);
    sum = fmaf(bf16_bits_to_f32(x[c] >> 16), bf16_bits_to_f32(y[c] >> 16), sum);
  }
  return sum;
}

// The weight's gradient of entry e by one wave.
__device__ __forceinline__ void dweight_of_entry(const CombineBwdParams& p, int e) {
  const int lane = threadIdx.x & 63;
  const int row = p.rows[e];
  float sum = 0.0f;
  if (row >= 0 && row < p.m_total && p.src[row] == e) {
    const uint16_t* dy = p.dy + (int64_t)divided((uint32_t)e, p.by_topk) * p.ld_dy;
    const uint16_t* d = p.d + (int64_t)row * p.ld_d;
    for (int c = lane * 8; c < p.cols; c += 64 * 8)
      sum = add_dot8(*reinterpret_cast<const uint4*>(dy + c), *reinterpret_cast<const uint4*>(d + c), sum);
  }
  sum = wave_sum(sum);
  if (lane == 0) p.dweights[e] = sum;
}

// Workgroup: one 128 x 128 tile of the expert rows.  dy and d are read once for
// all three results: the products go from registers to row codes and, through
// shared memory, to column codes; the rows' dot products over this tile's columns
// go to the workspace, summed in a fixed order by the next kernel (an atomic sum
// would differ from run to run).  Bound by memory: 32768 rows x 7168 move 0.74 GB
// in and 0.47 out in 215 to 260 us (5.6 to 4.6 TB/s), by where the five matrices
// lie; tiles in row order, in panels, or sorted by token change nothing or lose.
//
// APART: workgroups past the tiles sum the weights' gradient of four entries each,
// reading their rows again, and no second kernel is needed.
template <bool APART>
__global__ __launch_bounds__(kTileThreads<8>) void combine_bwd_kernel(CombineBwdParams p) {
  __shared__ TileLds<8> lds;
  const int row_tiles = p.m_total / kBlockK, column_tiles = p.cols / kBlockK;
  if constexpr (APART) {
    const int past = (int)blockIdx.x - row_tiles * column_tiles;
    if (past >= 0) {
      const int e = past * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      if (e < p.tokens * p.topk) dweight_of_entry(p, e);
      return;
    }
  }
  const TileAt tile = tile_of_workgroup(row_tiles, column_tiles);
  const int64_t row0 = (int64_t)tile.row * kBlockK;
  const int col0 = tile.col * kBlockK;
  const int tid = threadIdx.x, r0 = (tid >> 4) * 8, i16 = tid & 15, c0 = i16 * 8;
  const uint32_t entries = (uint32_t)(p.tokens * p.topk);
  const TileUse use = tile_use(p.src + row0, entries);
  if (!use.any()) return;
  float vs[1][8][8], w[8];
  auto& v = vs[0];
  uint32_t live = 0;
  uint4 a[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = row0 + r0 + i;
    const uint32_t e = (uint32_t)p.src[r];
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    w[i] = 0.0f;
    if (e < entries) {
      live |= 1u << i;
      a[i] = *reinterpret_cast<const uint4*>(p.dy + (int64_t)(divided(e, p.by_topk)) * p.ld_dy + col0 + c0);
      if (!APART) b[i] = load_streaming4(p.d + r * p.ld_d + col0 + c0);
      w[i] = p.weights[e];
    }
  }
  float mine = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[i][2 * c] = w[i] * bf16_bits_to_f32(x[c] & 0xFFFFu);
      v[i][2 * c + 1] = w[i] * bf16_bits_to_f32(x[c] >> 16);
    }
    if constexpr (!APART) {
      const float dot = row_sum(add_dot8(a[i], b[i], 0.0f));
      mine = i16 == i ? dot : mine;
    }
  }
  if (!APART && i16 < 8 && ((live >> i16) & 1)) p.dots[tile.col * (int64_t)p.m_total + row0 + r0 + i16] = mine;
  tile_rows<true>(v, p.dq + row0 * p.cols + col0, p.cols, p.dsf + tile.col * p.ld_dsf + row0, live);
  if (!p.dqt) return;
  const ColumnsTo to[1] = {{p.dqt + (int64_t)col0 * p.m_total + row0, p.m_total, p.dsft + (int64_t)tile.row * p.ld_dsft + col0}};
  tile_columns<true>(vs, lds, to);
}

// Workgroup x: the dot products of rows [64 x, 64 x + 64), each wave every fourth
// tile's, added into the rows' entries; and zeros for those of entries
// [256 x, 256 x + 256) that no row is of.  (32768 rows x 56 tiles: 5.9 us.)
__global__ __launch_bounds__(256) void combine_dweights_kernel(CombineBwdParams p) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t entries = (int64_t)p.tokens * p.topk;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = (int64_t)blockIdx.x * 64 + lane;
  if (i < entries) {
    const int at = p.rows[i];
    if (at < 0 || at >= p.m_total || p.src[at] != i) p.dweights[i] = 0.0f;
  }
  float sum = 0.0f;
  int e = -1;
  if (r < p.m_total) {
    e = p.src[r];
    if (e >= entries || (e >= 0 && p.rows[e] != r)) e = -1;
  }
  if (e >= 0) {
#pragma unroll 4
    for (int j = wave; j < p.cols / kBlockK; j += 4) sum += p.dots[j * (int64_t)p.m_total + r];
  }
  part[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && e >= 0) p.dweights[e] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
}

}  // namespace

size_t plan_workspace_bytes(int64_t entries, int groups) {
  return ((size_t)plan_blocks(entries) + 1) * groups * sizeof(int32_t);
}

hipError_t launch_plan(const PlanParams& params, hipStream_t stream) {
  PlanParams p = params;
  p.blocks = plan_blocks(p.entries);
  const dim3 block(kPlanThreads);
  if (p.entries <= kOnePlanEntries && p.layout_rows <= kOnePlanRows) {
    hipLaunchKernelGGL(plan_place_kernel<true>, dim3(1), block, 0, stream, p);
  } else {
    const int for_rows = (int)(((int64_t)p.layout_rows + 4 * kPlanThreads - 1) / (4 * kPlanThreads));
    const int most = for_rows < 256 ? for_rows : 256;
    // Few counts are added up by every block again, many by a launch of their own,
    // which costs 2 to 3 us (131072 entries of 4 groups: 9.6 us against 11.9; of 128:
    // 14.3 and 14.0, of 1024: 49.5 and 18.0; 1M of 4: 19.4 both, of 256: 159 and 30.3)
    // and keeps the work in proportion to the entries.
    p.scanned = (int64_t)p.blocks * (p.groups > 16 ? p.groups : 16) >= 16384;
    hipLaunchKernelGGL(plan_count_kernel, dim3(p.blocks), block, 0, stream, p);
    if (p.scanned) {
      int shift = 0;
      while (shift < kScanShift && 1 << shift < p.groups) ++shift;
      const int columns = (p.groups + (1 << shift) - 1) >> shift;
      hipLaunchKernelGGL(plan_scan_kernel, dim3(columns), block, 0, stream, p, shift);
    }
    hipLaunchKernelGGL(plan_place_kernel<false>, dim3(p.blocks > most ? p.blocks : most), block, 0, stream, p);
  }
  return hipGetLastError();
}

hipError_t launch_dispatch(const DispatchParams& p, bool pow2, hipStream_t stream) {
  const int gx = (p.cols / kBlockK + kTilesPerWave - 1) / kTilesPerWave;
  const int64_t total = (int64_t)p.groups * p.rows;
  // Tall layouts are streams, which four rows of a wave at a time and streaming
  // stores suit, whatever their width (32768 x 7168: 103 us, 116 with plain stores
  // and 127 with those row by row; 16384 x 1024: 8.2, 10.4 and 9.8; only very narrow
  // ones lose, 16384 x 128: 7.9, 7.9 and 6.9), and few rows in use go both ways (32
  // groups of 1024 rows, 3 % in use: 12.0 us against 10.1 row by row; 64 groups, 6 %:
  // 15.5 and 24.1).  Short ones wait for their reads, which more waves share (128
  // tokens in 32 groups of 128 rows: 4.8 us, and 5.7 by four; 8192 rows: a call in
  // 21.9 and 22.8).
  const int rows = total >= 16384 ? 4 : 1;
  // Tall: most waves make one trip (107 us, 114 with up to four trips).  Short: up
  // to two (8192 rows: a call in 23.6, 24.3 with one).
  int64_t gy = ((rows == 4 ? 65536 : 16384) / kRowWaves + gx - 1) / gx;
  const int64_t need = (total + kRowWaves * rows - 1) / (kRowWaves * rows);
  if (gy > need) gy = need;
  const dim3 grid(gx, (unsigned)(gy < 1 ? 1 : gy)), block(64 * kRowWaves);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, p); };
  if (pow2) {
    if (rows == 4) go(dispatch_kernel<true, 4>);
    else go(dispatch_kernel<true, 1>);
  } else {
    if (rows == 4) go(dispatch_kernel<false, 4>);
    else go(dispatch_kernel<false, 1>);
  }
  return hipGetLastError();
}

hipError_t launch_combine(const CombineParams& p, hipStream_t stream) {
  const GridXY by_token = spread(p.tokens);
  const dim3 grid(by_token.x, (p.cols / 8 + kCombineThreads - 1) / kCombineThreads, by_token.y);
  hipLaunchKernelGGL(combine_kernel, grid, dim3(kCombineThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineBwdParams& p, hipStream_t stream) {
  const int tiles = p.m_total / kBlockK * (p.cols / kBlockK);
  const int64_t entries = (int64_t)p.tokens * p.topk;
  const dim3 block(kTileThreads<8>);
  // Up to 20M values the second kernel costs more than reading twice (768 rows x
  // 7168 of 128 tokens: a call in 8.6 us, and 13.2 with it; 4608 x 4096: 20.2 and
  // 24.8; 4608 x 7168: 42.9 and 39.1), and up to 32768 entries the waves for those
  // without a row cost less too (1 of 16 with a row, x 2048: 11.5 and 13.8; of
  // 131072 entries, x 512: 21.0 and 12.6).
  if (entries <= 32768 && (int64_t)p.m_total * p.cols <= (int64_t)20 << 20) {
    const dim3 grid((unsigned)(tiles + (entries + 3) / 4));
    hipLaunchKernelGGL(combine_bwd_kernel<true>, grid, block, 0, stream, p);
    return hipGetLastError();
  }
  if (tiles > 0) hipLaunchKernelGGL(combine_bwd_kernel<false>, dim3(tiles), block, 0, stream, p);
  const int64_t by_entry = (entries + 255) / 256, by_row = (p.m_total + 63) / 64;
  hipLaunchKernelGGL(combine_dweights_kernel, dim3((unsigned)(by_entry > by_row ? by_entry : by_row)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dg
