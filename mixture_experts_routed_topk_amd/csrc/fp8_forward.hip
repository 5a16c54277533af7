// e4m3 products with block scales, forward (gfx950): the choice of tiles and the launches.  fp8_tile.h has the tiles.
#include "dense_tile.h"
#include "fp8_tile.h"

namespace moe {
namespace {

template <int EPI>
hipError_t launch_tiles(const Fp8Job& p, int tile, hipStream_t s) {
  const dim3 grid = fp8_grid((int64_t)p.j.mt * p.j.nt * p.j.splits);
  if (tile == 256) hipLaunchKernelGGL((fp8_forward_kernel<EPI, 2>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((fp8_forward_kernel<EPI, 1>), grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

// Sums that are stored as they are take the gradients' plain store
bool plain(const DenseEpi& e) { return !e.bias && !e.res && !e.pre && e.act == kActNone; }

}  // namespace

// The height whose rounds of tiles take less, with half a tile of every run empty.  Over 90 products of 8 to 64 runs of 32 to 512 rows on
// average this takes 0.9% longer than the better height (28% at most, where the uneven runs fill one round more or less);
// 256 rows from 192 a run on would take 2.9% longer, from 400 on 1.4%.
int fp8_grouped_height(int64_t T, int E, int64_t K, int64_t cols) {
  double best = 1e30;
  int rows = 0;
  for (const TileCost& t : kTilesFp8) {
    const double tiles = fmax((double)T / t.rows + 0.5 * E, (double)(T < E ? T : E)) * ((cols + 255) / 256);
    const double us = ceil(tiles / 256) * ((K / 128) * t.alone + t.fixed);
    if (us < best) best = us, rows = t.rows;
  }
  return rows;
}

size_t fp8_gemm_workspace(const Fp8Gemm& g) {
  if (g.g.M == 0 || g.E || g.few) return 0;
  return forward_part(plan_fp8(g.g.M, g.g.e.N, g.g.K, g.g.gated), g.g.M, g.g.e.N, g.g.gated, 1);
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, hipStream_t s) {
  if (g.few) return launch_fp8_rows(g, s);
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
    return g.g.gated ? launch_tiles<kGated>(p, height, s) : launch_tiles<kGrad>(p, height, s);
  }
  const Plan plan = plan_fp8(g.g.M, g.g.e.N, g.g.K, g.g.gated);
  return run_forward<uint16_t>(g.g, plan, 256, ws, s, [&](const Job& job, int epi) {
    const Fp8Job p = fp8_job(g, job);
    if (epi == kPartial) return launch_tiles<kPartial>(p, plan.tile, s);
    if (epi == kGated) return launch_tiles<kGated>(p, plan.tile, s);
    return plain(g.g.e) ? launch_tiles<kGrad>(p, plan.tile, s) : launch_tiles<kLinear>(p, plan.tile, s);
  });
}

}  // namespace moe
