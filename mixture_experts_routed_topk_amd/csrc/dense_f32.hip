// Matrix products of the dense operators in float32 (gfx950): the float32 layers, used for
// checking.
//
// out[m][n] = epilogue(sum_k r[m][k] c[n][k]) with each operand stored along k or along its
// rows (DenseGemm), any pitch and alignment.  A workgroup of four waves computes a 64 x 64
// tile (gated: 64 gate and the matching 64 up columns) with the float32 MFMA, K in slices of
// 16 through LDS; a wave's tile is 32 x 32.  The second operand sits on the MFMA's row side
// with its rows permuted so that a lane's two fragments hold eight consecutive columns of one output row
// (the row pieces epi_store writes).  Elements past the matrices are zero in LDS.
#include "dense_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int TM = 64, TN = 64, KS = 16;
constexpr int PITCH = TM + 4;   // LDS row pitch: k rows start 4 banks apart

// This thread's four elements of the [64 rows][16 k] slice at (row0, k0)
template <typename T>
__device__ __forceinline__ void load_slice(const void* p, int64_t ld, bool kmajor, int64_t row0, int64_t rows, int64_t k0,
                                           int64_t K, float v[4]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = kmajor ? row0 + (t & 15) * 4 + i : row0 + (t >> 2);
    const int64_t k = kmajor ? k0 + (t >> 4) : k0 + (t & 3) * 4 + i;
    v[i] = row < rows && k < K ? Piece<T>::get(p, kmajor ? k * ld + row : row * ld + k) : 0.f;
  }
}
__device__ __forceinline__ void put_slice(float (*lds)[PITCH], bool kmajor, const float v[4]) {
  const int t = threadIdx.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kmajor) lds[t >> 4][(t & 15) * 4 + i] = v[i];
    else lds[(t & 3) * 4 + i][t >> 2] = v[i];
  }
}

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void dense_f32_kernel(DenseGemm g) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ float R[KS][PITCH], C[NB][KS][PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave >> 1, wn = wave & 1, grp = lane >> 4, r16 = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.x * TM;
  const int n0 = blockIdx.y * TN;
  const int N = g.e.N;
  f32x4 acc[NB][2][2] = {};
  for (int64_t k0 = 0; k0 < g.K; k0 += KS) {
    float vr[4], vc[NB][4];
    load_slice<T>(g.r, g.ldr, g.r_kmajor, m0, g.M, k0, g.K, vr);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // the up projection's rows follow the N gate rows
      const char* c = static_cast<const char*>(g.c) + (int64_t)b * N * g.ldc * (int64_t)sizeof(T);
      load_slice<T>(c, g.ldc, g.c_kmajor, n0, N, k0, g.K, vc[b]);
    }
    __syncthreads();   // the previous slice has been read
    put_slice(R, g.r_kmajor, vr);
#pragma unroll
    for (int b = 0; b < NB; ++b) put_slice(C[b], g.c_kmajor, vc[b]);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KS; k += 4) {
      float fr[2], fc[NB][2];
#pragma unroll
      for (int i = 0; i < 2; ++i) fr[i] = R[k + grp][wm * 32 + i * 16 + r16];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) fc[b][j] = C[b][k + grp][wn * 32 + 8 * (r16 >> 2) + 4 * j + (r16 & 3)];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[b][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fc[b][j], fr[i], acc[b][i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm * 32 + i * 16 + r16;
    if (m >= g.M) continue;
    float z[8], u[8];
#pragma unroll
    for (int v = 0; v < 8; ++v) {
      z[v] = acc[0][i][v >> 2][v & 3];
      u[v] = acc[NB - 1][i][v >> 2][v & 3];
    }
    epi_store<T, GATED>(g.e, m, n0 + wn * 32 + 8 * grp, z, u);
  }
}

template <typename T>
hipError_t launch(const DenseGemm& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.M + TM - 1) / TM), (unsigned)((g.e.N + TN - 1) / TN));
  if (g.gated) hipLaunchKernelGGL((dense_f32_kernel<T, true>), grid, dim3(kThreads), 0, s, g);
  else hipLaunchKernelGGL((dense_f32_kernel<T, false>), grid, dim3(kThreads), 0, s, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dense_gemm_f32(const DenseGemm& g, hipStream_t s) { return launch<float>(g, s); }

}  // namespace moe
