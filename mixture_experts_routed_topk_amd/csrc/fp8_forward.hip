// e4m3 products with block scales, forward (gfx950): the choice of tiles and the launches.  fp8_tile.h has the tiles.
#include "dense_tile.h"
#include "fp8_tile.h"

namespace moe {
namespace {

template <int EPI>
hipError_t launch_tiles(const Fp8Job& p, int tile, int y, hipStream_t s) {
  if (tile == 256) hipLaunchKernelGGL((fp8_rows_tile_kernel<false, EPI, 2, true>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  else hipLaunchKernelGGL((fp8_rows_tile_kernel<false, EPI, 1, true>), fp8_grid(p.j, y), dim3(512), 0, s, p);
  return hipGetLastError();
}

// Sums that are stored as they are take the gradients' plain store
bool plain(const DenseEpi& e) { return !e.bias && !e.res && !e.pre && e.act == kActNone; }

}  // namespace

int fp8_grouped_height(int64_t T, int E) { return T >= (int64_t)192 * E ? 256 : 128; }

size_t fp8_gemm_workspace(const Fp8Gemm& g) {
  if (g.g.M == 0 || g.E || fp8_rows_take(g.g.M, g.g.K)) return 0;
  return forward_part(plan_fp8(g.g.M, g.g.e.N, g.g.K, g.g.gated), g.g.M, g.g.e.N, g.g.gated, 1);
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, hipStream_t s) {
  if (g.E) {
    const int height = g.runs.height;
    Job job{};
    job.g = g.g;
    job.splits = 1;
    job.slices = (int)(g.g.K / 128);
    job.crows = g.g.gated ? 2 * g.g.e.N : g.g.e.N;
    job.mt = (int)max_row_tiles(g.g.M, g.E, height);
    job.nt = (job.crows + 255) / 256;
    const Fp8Job p = fp8_job(g, job);
    return g.g.gated ? launch_tiles<kGated>(p, height, 1, s) : launch_tiles<kGrad>(p, height, 1, s);
  }
  if (fp8_rows_take(g.g.M, g.g.K)) return launch_fp8_rows(g, s);
  const Plan plan = plan_fp8(g.g.M, g.g.e.N, g.g.K, g.g.gated);
  return run_forward<uint16_t>(g.g, plan, 256, ws, s, [&](const Job& job, int epi) {
    const Fp8Job p = fp8_job(g, job);
    if (epi == kPartial) return launch_tiles<kPartial>(p, plan.tile, job.splits, s);
    if (epi == kGated) return launch_tiles<kGated>(p, plan.tile, 1, s);
    return plain(g.g.e) ? launch_tiles<kGrad>(p, plan.tile, 1, s) : launch_tiles<kLinear>(p, plan.tile, 1, s);
  });
}

}  // namespace moe
