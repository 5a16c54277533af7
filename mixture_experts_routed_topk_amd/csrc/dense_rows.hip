// Forward products of the dense operators on few rows (decode steps) in bf16 (gfx950).
//
// With few rows the product is one pass over the weights: its time is their bytes over the
// memory rate, and below a few megabytes the latency of one load and one reduction.  A
// workgroup takes 16 weight rows (gated: 8 gate rows and the matching 8 up rows) and its NW
// waves split the contraction, each a contiguous run of 32-element steps, so that all of the
// weights are in flight at once from as many waves as there are.  Weights and activations
// go from memory straight into the MFMA's registers (16 bytes a lane); the weights sit on
// the MFMA's row side, so a lane ends with four consecutive columns of one output row.  The waves' float32
// sums meet in LDS and are added in wave order, in the same launch: no workspace, no second
// kernel.
#include "dense_device.h"

namespace moe {
namespace {

// U steps of this wave from k on, all their loads before the first product.  TAIL: pieces from
// `end` on are zero (loaded from the row's start and replaced, so that no load hangs on a branch).
template <int MT, int U, bool TAIL>
__device__ __forceinline__ void steps(const uint16_t* const (&rp)[MT], const uint16_t* cp, int k, int end, f32x4 (&acc)[MT]) {
  bf16x8 c[U], r[U][MT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = !TAIL || k + 32 * u < end ? k + 32 * u : 0;
    c[u] = *reinterpret_cast<const bf16x8*>(cp + at);
#pragma unroll
    for (int i = 0; i < MT; ++i) r[u][i] = *reinterpret_cast<const bf16x8*>(rp[i] + at);
  }
  __builtin_amdgcn_sched_barrier(0);   // (or the compiler starts multiplying with half the loads issued)
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (TAIL && k + 32 * u >= end) {
      c[u] = bf16x8{};
#pragma unroll
      for (int i = 0; i < MT; ++i) r[u][i] = bf16x8{};
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = mfma_16x16x32_bf16(c[u], r[u][i], acc[i]);
  }
}

template <int MT, bool GATED, int NW>
__global__ __launch_bounds__(NW * 64) void dense_rows_kernel(DenseGemm g) {
  constexpr int U = MT == 1 ? 8 : 4;
  constexpr int COLS = GATED ? 8 : 16;
  __shared__ f32x4 red[MT][NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int grp = lane >> 4, i16 = lane & 15;
  const int n0 = blockIdx.x * COLS, N = g.e.N;
  const int per = (int)(((g.K + 31) / 32 + NW - 1) / NW);   // steps of a wave
  const int k0 = wave * per * 32 + grp * 8;
  const int end = min((int)g.K, (wave + 1) * per * 32);     // (whole 16-byte pieces: K is a multiple of 8)

  // rows past the matrix repeat its last one and are not stored
  const int64_t crow = min(n0 + i16 % COLS, N - 1) + (GATED ? (int64_t)(i16 / COLS) * N : 0);
  const uint16_t* cp = static_cast<const uint16_t*>(g.c) + crow * g.ldc;
  const uint16_t* rp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    rp[i] = static_cast<const uint16_t*>(g.r) + min((int64_t)(i * 16 + i16), g.M - 1) * g.ldr;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{};
  const int full = max(0, (end - wave * per * 32) / 32);    // steps inside K
  int s = 0;
  for (; s + U <= full; s += U) steps<MT, U, false>(rp, cp, k0 + 32 * s, end, acc);
  if (per - s > U / 2) steps<MT, U, true>(rp, cp, k0 + 32 * s, end, acc);
  else if (per - s > U / 4) steps<MT, U / 2, true>(rp, cp, k0 + 32 * s, end, acc);
  else if (per > s) steps<MT, U / 4, true>(rp, cp, k0 + 32 * s, end, acc);

#pragma unroll
  for (int i = 0; i < MT; ++i) red[i][wave][lane] = acc[i];
  __syncthreads();
  // a thread finishes one element (little code: a kernel this short waits for its own instructions)
  for (int t = threadIdx.x; t < MT * 16 * COLS; t += NW * 64) {
    const int i = t / (16 * COLS), q = t / COLS % 16, c = t % COLS;
    const int64_t m = i * 16 + q;
    if (m >= g.M || n0 + c >= N) continue;
    float z = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      z += red[i][w][(c >> 2) * 16 + q][c & 3];
      if (GATED) u += red[i][w][(2 + (c >> 2)) * 16 + q][c & 3];
    }
    epi_store1<uint16_t, GATED>(g.e, m, n0 + c, z, u);
  }
}

template <int MT, int NW>
void launch_rows(const DenseGemm& g, hipStream_t s) {
  const dim3 grid((unsigned)(g.gated ? (g.e.N + 7) / 8 : (g.e.N + 15) / 16));
  if (g.gated) hipLaunchKernelGGL((dense_rows_kernel<MT, true, NW>), grid, dim3(NW * 64), 0, s, g);
  else hipLaunchKernelGGL((dense_rows_kernel<MT, false, NW>), grid, dim3(NW * 64), 0, s, g);
}
template <int MT>
void launch_waves(const DenseGemm& g, hipStream_t s) {
  // more waves share a longer contraction
  if (g.K > 4096) launch_rows<MT, 16>(g, s);
  else launch_rows<MT, 8>(g, s);
}

}  // namespace

// Beside the tile kernels (dense_bf16.hip; both replayed from a graph): one row of K = 2048, N = 7168
// 7.0 against 8.7 us, gated N = 5632 10.7 against 14.0; 16 rows of K = 2048, N = 2048 5.9 against 8.9; 32
// rows 7.8 against 9.5.  Each workgroup reads all rows of r, so with rows x K above 65536 the
// tiles win (16 rows of K = 7168, N = 2048: 16.9 against 14.1 us).
bool dense_rows_take(int64_t M, int64_t K) { return M <= 32 && M * K <= 65536; }

hipError_t launch_dense_rows(const DenseGemm& g, hipStream_t s) {
  if (g.M <= 16) launch_waves<1>(g, s);
  else launch_waves<2>(g, s);
  return hipGetLastError();
}

}  // namespace moe
