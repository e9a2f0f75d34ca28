// The dense FP8 GEMM with bias, activation and residual in its epilogue: the
// kernel of dg_gemm_kernel.h in the tiles that the dense heuristic picks, with
// the sums changed where they are rounded (apply_epilogue).  A sum that lies in
// partial tiles (stream-K) meets the epilogue once, in the workgroup that joins
// them.

#include "dg_gemm_kernel.h"

namespace dg {

namespace {

template <class T, int SF>
hipError_t launch_one(const GemmParams& p, const GemmEpilogue& e, const Schedule& s, int grid, hipStream_t stream) {
  if (s.stream_k)
    hipLaunchKernelGGL((gemm_kernel<T, kDense, true, SF, 0, GemmEpilogue>), dim3(grid), dim3(T::kThreads), 0, stream, p, s, e);
  else
    hipLaunchKernelGGL((gemm_kernel<T, kDense, false, SF, 0, GemmEpilogue>), dim3(grid), dim3(T::kThreads), 0, stream, p, s, e);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_epilogue(const GemmParams& p0, const GemmEpilogue& e, const GemmConfig& cfg, hipStream_t stream) {
  GemmParams p = p0;
  const Schedule s = schedule_of(kDense, p, cfg);
  if (cfg.stream_k) p.counters = reinterpret_cast<int*>(p.workspace);
  if (p.sf_ue8m0) {
    switch (cfg.variant) {
      case 0: return launch_one<TileP256, kScaleUE8M0>(p, e, s, cfg.grid, stream);
      case 4: return launch_one<TileS64, kScaleUE8M0>(p, e, s, cfg.grid, stream);
      case 5: return launch_one<TileW128, kScaleUE8M0>(p, e, s, cfg.grid, stream);
      case 6: return launch_one<TileP128w8, kScaleUE8M0>(p, e, s, cfg.grid, stream);
      default: return hipErrorInvalidValue;
    }
  }
  switch (cfg.variant) {
    case 0: return launch_one<TileP256, kScaleF32>(p, e, s, cfg.grid, stream);
    case 4: return launch_one<TileS64, kScaleF32>(p, e, s, cfg.grid, stream);
    case 5: return launch_one<TileW128, kScaleF32>(p, e, s, cfg.grid, stream);
    case 6: return launch_one<TileP128w8, kScaleF32>(p, e, s, cfg.grid, stream);
    case 11: return launch_one<TileP160, kScaleF32>(p, e, s, cfg.grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dg
