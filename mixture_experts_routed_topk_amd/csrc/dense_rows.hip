// Forward products of the dense operators on few rows (decode steps), bf16 and float32 (gfx950).
//
// With few rows the product is one pass over the weights: its time is their bytes over the
// memory rate, and below a few megabytes the latency of one load and one reduction.  A
// workgroup takes 16 weight rows (gated: 8 gate rows and the matching 8 up rows) and its NW
// waves split the contraction, each a contiguous run of 64-byte steps, so that all of the
// weights are in flight at once from as many waves as there are.  Weights and activations
// go from memory straight into the MFMA's registers (16 bytes a lane); the weights sit on
// the MFMA's row side, so a lane ends with four consecutive columns of one output row.  The waves' float32
// sums meet in LDS and are added in wave order, in the same launch: no workspace, no second
// kernel.
#include "dense_tile.h"

namespace moe {
namespace {

// U steps of this wave from k on, all their loads before the first product.  TAIL: pieces from
// `end` on are zero (loaded from the row's start and replaced, so that no load hangs on a branch).
template <typename T, int MT, int U, bool TAIL>
__device__ __forceinline__ void steps(const T* const (&rp)[MT], const T* cp, int k, int end, f32x4 (&acc)[MT]) {
  constexpr int KSTEP = 64 / sizeof(T);   // k of a step: 16 bytes a lane
  Frag<T> c[U], r[U][MT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = !TAIL || k + KSTEP * u < end ? k + KSTEP * u : 0;
    c[u] = *reinterpret_cast<const Frag<T>*>(cp + at);
#pragma unroll
    for (int i = 0; i < MT; ++i) r[u][i] = *reinterpret_cast<const Frag<T>*>(rp[i] + at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (TAIL && k + KSTEP * u >= end) {
      c[u] = Frag<T>{};
#pragma unroll
      for (int i = 0; i < MT; ++i) r[u][i] = Frag<T>{};
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = multiply_add(c[u], r[u][i], acc[i]);
  }
}

template <typename T, int MT, bool GATED, int NW>
__global__ __launch_bounds__(NW * 64) void dense_rows_kernel(DenseGemm g) {
  constexpr int U = MT == 1 ? 8 : 4;
  constexpr int KSTEP = 64 / sizeof(T);
  constexpr int COLS = GATED ? 8 : 16;
  __shared__ f32x4 red[MT][NW][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int grp = lane >> 4, i16 = lane & 15;
  const int n0 = blockIdx.x * COLS, N = g.e.N;
  const int per = (int)(((g.K + KSTEP - 1) / KSTEP + NW - 1) / NW);   // steps of a wave
  const int k0 = wave * per * KSTEP + grp * (KSTEP / 4);
  const int end = min((int)g.K, (wave + 1) * per * KSTEP);     // (whole 16-byte pieces: K is a multiple of 8)

  // rows past the matrix repeat its last one and are not stored
  const int64_t crow = min(n0 + i16 % COLS, N - 1) + (GATED ? (int64_t)(i16 / COLS) * N : 0);
  const T* cp = static_cast<const T*>(g.c) + crow * g.ldc;
  const T* rp[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    rp[i] = static_cast<const T*>(g.r) + min((int64_t)(i * 16 + i16), g.M - 1) * g.ldr;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{};
  const int full = max(0, (end - wave * per * KSTEP) / KSTEP);    // steps inside K
  int s = 0;
  for (; s + U <= full; s += U) steps<T, MT, U, false>(rp, cp, k0 + KSTEP * s, end, acc);
  if (per - s > U / 2) steps<T, MT, U, true>(rp, cp, k0 + KSTEP * s, end, acc);
  else if (per - s > U / 4) steps<T, MT, U / 2, true>(rp, cp, k0 + KSTEP * s, end, acc);
  else if (per > s) steps<T, MT, U / 4, true>(rp, cp, k0 + KSTEP * s, end, acc);

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
    epi_store1<T, GATED>(g.e, m, n0 + c, z, u);
  }
}

template <typename T, int MT, int NW>
void launch_rows(const DenseGemm& g, hipStream_t s) {
  const dim3 grid((unsigned)(g.gated ? (g.e.N + 7) / 8 : (g.e.N + 15) / 16));
  if (g.gated) hipLaunchKernelGGL((dense_rows_kernel<T, MT, true, NW>), grid, dim3(NW * 64), 0, s, g);
  else hipLaunchKernelGGL((dense_rows_kernel<T, MT, false, NW>), grid, dim3(NW * 64), 0, s, g);
}
template <typename T, int MT>
void launch_waves(const DenseGemm& g, hipStream_t s) {
  // more waves share a longer contraction
  if (g.K * (int64_t)sizeof(T) > 8192) launch_rows<T, MT, 16>(g, s);
  else launch_rows<T, MT, 8>(g, s);
}
template <typename T>
void launch_type(const DenseGemm& g, hipStream_t s) {
  if (g.M <= 16) launch_waves<T, 1>(g, s);
  else launch_waves<T, 2>(g, s);
}

}  // namespace

// Beside the tile kernels (both replayed from a graph): one row of K = 2048, N = 7168
// 7.0 against 8.7 us, gated N = 5632 10.2 against 14.0; 16 rows of K = 2048, N = 2048 5.9 against 8.9; 32
// rows 7.8 against 9.5.  Each workgroup reads all rows of r, so with more than 128 KB of them
// the tiles win (16 bf16 rows of K = 7168, N = 2048: 16.9 against 14.1 us).
bool dense_rows_take(int64_t M, int64_t K, bool f32) { return M <= 32 && M * K * (f32 ? 4 : 2) <= 131072; }

hipError_t launch_dense_rows(const DenseGemm& g, bool f32, hipStream_t s) {
  if (f32) launch_type<float>(g, s);
  else launch_type<uint16_t>(g, s);
  return hipGetLastError();
}

}  // namespace moe
