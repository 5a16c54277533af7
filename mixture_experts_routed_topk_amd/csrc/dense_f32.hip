// float32 matrix products of the dense operators (gfx950): the float32 layers, used for checking.
//
// The same tiles as in bf16 (dense_tile.h) with the float32 MFMA, which multiplies at a sixteenth of the bf16
// rate: a slice of a tile takes 1 to 2 us of its CU, and what counts is that the tiles fill the
// CUs evenly, so tiles go down to 32 rows and contractions are split.
#include "dense_tile.h"

namespace moe {
namespace {

template <int EPI>
void launch_tiles(const Job& job, int tile, hipStream_t s) {
  const dim3 grid = tile_grid(job);
  if (tile == 128) hipLaunchKernelGGL((dense_128_kernel<float, 128, false, false, EPI>), grid, dim3(256), 0, s, job);
  else if (tile == 64) hipLaunchKernelGGL((dense_128_kernel<float, 64, false, false, EPI>), grid, dim3(256), 0, s, job);
  else hipLaunchKernelGGL((dense_128_kernel<float, 32, false, false, EPI>), grid, dim3(256), 0, s, job);
}

// dx in tiles of TA rows and dw in tiles of 128 (as dense_pair_kernel in dense_bf16.hip)
template <int TA>
__global__ __launch_bounds__(256, 2) void dense_pair_f32_kernel(Job dx, Job dw, int n_first, int dw_first) {
  __shared__ __attribute__((aligned(1024))) char lds[lds_128<128>()];
  const bool first = (int)blockIdx.x < n_first;
  const int b = first ? blockIdx.x : blockIdx.x - n_first;
  if (first == (dw_first != 0)) {
    const int n = (dw.mt * dw.nt + 7) / 8 * 8;
    tile_128<float, 128, true, true, kGrad>(dw, b % n, b / n, lds);
  } else {
    const int n = (dx.mt * dx.nt + 7) / 8 * 8;
    tile_128<float, TA, false, true, kGrad>(dx, b % n, b / n, lds);
  }
}

}  // namespace

size_t dense_gemm_f32_workspace(int64_t M, int64_t N, int64_t K, int gated, int vec) {
  return forward_part(plan_f32(M, N, K, gated), M, N, gated, vec);
}

hipError_t launch_dense_gemm_f32(const DenseGemm& g, void* ws, hipStream_t s) {
  const Plan p = plan_f32(g.M, g.e.N, g.K, g.gated);
  return run_forward<float>(g, p, 128, ws, s, [&](const Job& job, int epi) {
    if (epi == kPartial) launch_tiles<kPartial>(job, p.tile, s);
    else if (epi == kGated) launch_tiles<kGated>(job, p.tile, s);
    else launch_tiles<kLinear>(job, p.tile, s);
    return hipGetLastError();
  });
}

size_t dense_gradients_f32_workspace(int64_t rows, int64_t N, int64_t cols) {
  return gradients_part<float>(kPairsF32, kPairTilesF32, kJoinF32, rows, N, cols, false);
}

hipError_t launch_dense_gradients_f32(const DenseGemm* dx, const DenseGemm* dw, void* ws, hipStream_t s) {
  return run_gradients<float>(kPairsF32, kPairTilesF32, kJoinF32, dx, dw, false, ws, s,
                              [&](int pair, dim3 grid, const Job& x, const Job& w, int n_first, int dw_first) {
    if (pair == 0) hipLaunchKernelGGL(dense_pair_f32_kernel<128>, grid, dim3(256), 0, s, x, w, n_first, dw_first);
    else if (pair == 1) hipLaunchKernelGGL(dense_pair_f32_kernel<64>, grid, dim3(256), 0, s, x, w, n_first, dw_first);
    else hipLaunchKernelGGL(dense_pair_f32_kernel<32>, grid, dim3(256), 0, s, x, w, n_first, dw_first);
    return hipGetLastError();
  });
}

}  // namespace moe
