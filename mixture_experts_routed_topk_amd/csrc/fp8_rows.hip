// e4m3 products with block scales on few rows (decode steps), forward (gfx950).
//
// One pass over the weights, as in dense_rows.hip: a workgroup takes 16 weight rows (gated: 8 gate rows and the matching
// 8 up rows), its waves share the contraction in contiguous runs of 128-k slices, and codes go from memory
// straight into the MFMA's registers, 32 bytes a lane.  A slice's result is folded in times the row's and the
// block's scale.  The waves' float32 sums meet in LDS and are added in wave order.
#include "dense_device.h"
#include "fp8_internal.h"

namespace moe {
namespace {

// U slices from kt on, all their loads before the first product; slices from `end` on are not counted (they repeat the
// last one, times zero)
template <int MT, int U, bool UE8>
__device__ __forceinline__ void slices(const uint8_t* const (&rp)[MT], const uint8_t* cp, const float* const (&sp)[MT],
                                       const void* bp, int kt, int end, f32x4 (&acc)[MT]) {
  i32x4 c[U][2], r[U][MT][2];
  float sr[U][MT], sb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = min(kt + u, end - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) c[u][h] = *reinterpret_cast<const i32x4*>(cp + (int64_t)at * 128 + h * 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) r[u][i][h] = *reinterpret_cast<const i32x4*>(rp[i] + (int64_t)at * 128 + h * 16);
      sr[u][i] = sp[i][at];
    }
    if constexpr (UE8) {
      const uint32_t b = static_cast<const uint8_t*>(bp)[at];
      sb[u] = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
    } else {
      sb[u] = static_cast<const float*>(bp)[at];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const i32x8 cv = __builtin_shufflevector(c[u][0], c[u][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const i32x8 rv = __builtin_shufflevector(r[u][i][0], r[u][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
      const f32x4 p = mfma_16x16x128_e4m3(cv, rv, f32x4{});
      const float s = sr[u][i] * sb[u];
      if (kt + u < end) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(p[q], s, acc[i][q]);
      }
    }
  }
}

template <int MT, bool GATED, int NW, bool UE8>
__global__ __launch_bounds__(NW * 64) void fp8_rows_kernel(Fp8Gemm p) {
  constexpr int U = MT == 2 && NW == 16 ? 2 : 4;     // (what fits in the registers of so many waves)
  constexpr int COLS = GATED ? 8 : 16;
  __shared__ f32x4 red[MT][NW][64];
  const DenseGemm& g = p.g;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int grp = lane >> 4, i16 = lane & 15;
  const int n0 = blockIdx.x * COLS, N = g.e.N;
  const int KT = (int)(g.K / 128);
  const int per = (KT + NW - 1) / NW;
  const int first = wave * per, end = min(KT, first + per);

  const int64_t crow = n0 + i16 % COLS + (GATED ? (int64_t)(i16 / COLS) * N : 0);
  const uint8_t* cp = static_cast<const uint8_t*>(g.c) + crow * g.ldc + grp * 32;
  // the block of this lane's result columns 4 grp .. 4 grp + 3 (gated: lane groups 2 and 3 hold the up rows)
  const int64_t block = (n0 >> 7) + (GATED ? (int64_t)(grp >> 1) * (N >> 7) : 0);
  const void* bp = static_cast<const char*>(p.cs.p) + block * p.cs.row * (UE8 ? 1 : 4);
  const uint8_t* rp[MT];
  const float* sp[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {       // rows past the matrix repeat its last one and are not stored
    const int64_t m = min((int64_t)(i * 16 + i16), g.M - 1);
    rp[i] = static_cast<const uint8_t*>(g.r) + m * g.ldr + grp * 32;
    sp[i] = static_cast<const float*>(p.rs.p) + m * p.rs.row;
    acc[i] = f32x4{};
  }
  for (int kt = first; kt < end; kt += U) {
    if (end - kt > U / 2) slices<MT, U, UE8>(rp, cp, sp, bp, kt, end, acc);
    else slices<MT, U / 2, UE8>(rp, cp, sp, bp, kt, end, acc);
  }

#pragma unroll
  for (int i = 0; i < MT; ++i) red[i][wave][lane] = acc[i];
  __syncthreads();
  for (int t = threadIdx.x; t < MT * 16 * COLS; t += NW * 64) {
    const int i = t / (16 * COLS), q = t / COLS % 16, c = t % COLS;
    const int64_t m = i * 16 + q;
    if (m >= g.M) continue;
    float z = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      z += red[i][w][(c >> 2) * 16 + q][c & 3];
      if (GATED) u += red[i][w][(2 + (c >> 2)) * 16 + q][c & 3];
    }
    epi_store1<uint16_t, GATED>(g.e, m, n0 + c, z, u);
  }
}

template <int MT, int NW, bool UE8>
void launch_rows(const Fp8Gemm& g, hipStream_t s) {
  const dim3 grid((unsigned)(g.g.gated ? g.g.e.N / 8 : g.g.e.N / 16));
  if (g.g.gated) hipLaunchKernelGGL((fp8_rows_kernel<MT, true, NW, UE8>), grid, dim3(NW * 64), 0, s, g);
  else hipLaunchKernelGGL((fp8_rows_kernel<MT, false, NW, UE8>), grid, dim3(NW * 64), 0, s, g);
}
template <int MT, bool UE8>
void launch_waves(const Fp8Gemm& g, hipStream_t s) {
  if (g.g.K > 4096) launch_rows<MT, 16, UE8>(g, s);
  else launch_rows<MT, 8, UE8>(g, s);
}
template <bool UE8>
void launch_heights(const Fp8Gemm& g, hipStream_t s) {
  if (g.g.M <= 16) launch_waves<1, UE8>(g, s);
  else launch_waves<2, UE8>(g, s);
}

}  // namespace

bool fp8_rows_take(int64_t M, int64_t K) { return M <= 32 && M * K <= 131072; }

hipError_t launch_fp8_rows(const Fp8Gemm& g, hipStream_t s) {
  if (g.cs.bytes) launch_heights<true>(g, s);
  else launch_heights<false>(g, s);
  return hipGetLastError();
}

}  // namespace moe
