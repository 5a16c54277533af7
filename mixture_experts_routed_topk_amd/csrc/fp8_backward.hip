// e4m3 products with block scales, the two gradients (gfx950).  fp8_tile.h has the tiles.
//
// dx = dz w reads the weights along their rows, as they are stored, and applies their block scales; dw = dz^T x reads
// both operands along their rows.  dz's and x's scales are powers of two, so dw's MFMAs apply all scales
// themselves, and dx's too with UE8M0 weights.
#include "dense_tile.h"
#include "fp8_tile.h"

namespace moe {
namespace {

template <bool FOLD>
hipError_t launch_dx_tiles(const Fp8Job& p, int tile, int y, hipStream_t s) {
  if (tile == 256) hipLaunchKernelGGL((fp8_rows_tile_kernel<true, kGrad, 2, FOLD>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  else hipLaunchKernelGGL((fp8_rows_tile_kernel<true, kGrad, 1, FOLD>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  return hipGetLastError();
}
hipError_t launch_dw_tiles(const Fp8Job& p, int tile, int y, hipStream_t s) {
  if (tile == 256) hipLaunchKernelGGL((fp8_dw_kernel<2>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  else hipLaunchKernelGGL((fp8_dw_kernel<1>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  return hipGetLastError();
}

// A gradient over one matrix: tiles, and the splits' sum
template <typename F>
hipError_t run_gradient(const Fp8Gemm& g, void* ws, hipStream_t s, F&& tiles) {
  const Plan plan = plan_fp8(g.g.M, g.g.e.N, g.g.K, 0);
  Job job{};
  job.g = g.g;
  job.splits = plan.splits;
  job.slices = plan.slices;
  job.crows = g.g.e.N;
  job.mt = (int)((g.g.M + plan.tile - 1) / plan.tile);
  job.nt = (job.crows + 255) / 256;
  if (plan.splits > 1) {
    job.part = static_cast<float*>(ws);
    job.ldpart = g.g.e.N;
  }
  hipError_t err = tiles(fp8_job(g, job), plan.tile, plan.splits);
  if (err != hipSuccess || plan.splits == 1) return err;
  const int64_t pieces = g.g.M * (g.g.e.N / 8);
  hipLaunchKernelGGL((dense_join_kernel<uint16_t, false>), dim3((unsigned)((pieces + 255) / 256)), dim3(256), 0, s, job);
  return hipGetLastError();
}

}  // namespace

size_t fp8_dx_workspace(int64_t T, int64_t K, int64_t cols, int E) {
  return T == 0 || E ? 0 : forward_part(plan_fp8(T, K, cols, 0), T, K, 0, 1);
}
size_t fp8_dw_workspace(int64_t T, int64_t K, int64_t cols, int E) {
  return T == 0 || E ? 0 : forward_part(plan_fp8(cols, K, T, 0), cols, K, 0, 1);
}

hipError_t launch_fp8_dx(const Fp8Gemm& g, void* ws, hipStream_t s) {
  const bool fold = !g.cs.bytes;
  if (!g.E)
    return run_gradient(g, ws, s, [&](const Fp8Job& p, int tile, int y) {
      return fold ? launch_dx_tiles<true>(p, tile, y, s) : launch_dx_tiles<false>(p, tile, y, s);
    });
  Job job{};
  job.g = g.g;
  job.splits = 1;
  job.slices = (int)(g.g.K / 128);
  job.crows = g.g.e.N;
  job.mt = (int)max_row_tiles(g.g.M, g.E, g.runs.height);
  job.nt = (job.crows + 255) / 256;
  const Fp8Job p = fp8_job(g, job);
  return fold ? launch_dx_tiles<true>(p, g.runs.height, 1, s) : launch_dx_tiles<false>(p, g.runs.height, 1, s);
}

hipError_t launch_fp8_dw(const Fp8Gemm& g, void* ws, hipStream_t s) {
  if (!g.E) return run_gradient(g, ws, s, [&](const Fp8Job& p, int tile, int y) { return launch_dw_tiles(p, tile, y, s); });
  Job job{};
  job.g = g.g;
  job.splits = 1;
  job.crows = g.g.e.N;
  const int tile = g.g.M % 256 == 0 || g.g.M > 1024 ? 256 : 128;
  job.mt = (int)((g.g.M + tile - 1) / tile);
  job.nt = (job.crows + 255) / 256;
  return launch_dw_tiles(fp8_job(g, job), tile, g.E, s);
}

}  // namespace moe
