// Matrix products of the dense operators in float32 (gfx950): the float32 layers, used for
// checking.
//
// out[m][n] = epilogue(sum_k r[m][k] c[n][k]) with each operand stored along k or along its
// rows (DenseGemm).  A workgroup computes a 64 x 64 tile (gated: 64 gate and the matching 64 up columns)
// with the float32 MFMA.  Its G groups of four waves (2 x 2, a wave 32 x 32 of the tile) take
// every G-th slice of the contraction and their sums are added in group order through LDS at the end, so
// that two waves share a SIMD where there are fewer tiles than CUs: 333 x 1408 x 2048 (192 tiles)
// 46.4 us with one group and 37.6 with two.  (The MFMAs of one tile take 19 us on its CU: the rest
// is one wave's reads and stores that the other does not cover.)
//
// A slice goes memory -> registers -> LDS, loaded two rounds ahead of its use and stored one
// ahead, two LDS buffers per group, one barrier per round.  Operands keep their storage
// order in LDS: rows of KS k (+4) or k rows of 64 (+16), which spreads a fragment's 16 rows and
// 4 k over all 64 banks.  The second operand sits on the MFMA's row side; its rows are permuted on
// their way into LDS so that a lane's two fragments hold eight consecutive columns of one output row
// (the pieces epi_store writes): fragment j, row q is column 8 (q / 4) + 4 j + q % 4.
#include "dense_device.h"

namespace moe {
namespace {

constexpr int TM = 64, TN = 64;
template <int KS>
constexpr int buf_floats() { return TM * (KS + 4) > KS * (TM + 16) ? TM * (KS + 4) : KS * (TM + 16); }

// LDS row of tile column n: 32 (n / 32) + 16 j + q
__device__ __forceinline__ int permuted(int n) { return (n & 35) | ((n & 24) >> 1) | ((n & 4) << 2); }

// This thread's pieces of four elements of a [64 rows][KS k] slice, one of 256 threads
template <bool KM, bool PERM, int KS>
struct Slice {
  static constexpr int NP = KS / 16;                  // pieces a thread
  static constexpr int KP = KS + 4, RP = TM + 16;     // LDS pitches: [row][k], [k][row]
  f32x4 v[NP];
  static __device__ __forceinline__ int row_of(int t, int q) { return KM ? (t & 15) * 4 : t / (KS / 4) + (1024 / KS) * q; }
  static __device__ __forceinline__ int k_of(int t, int q) { return KM ? (t >> 4) + 16 * q : t % (KS / 4) * 4; }
  // next[q] is where piece q of the slice comes from, row_ok whether its row exists; pieces past the
  // rows or past the `left` k that the contraction still has are zero (and read from `base`)
  __device__ __forceinline__ void load(int t, const float* base, const float* (&next)[NP], const bool (&row_ok)[NP],
                                       int64_t step, int left) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const bool in = row_ok[q] && k_of(t, q) < left;
      const f32x4 got = *reinterpret_cast<const f32x4*>(in ? next[q] : base);
      v[q] = in ? got : f32x4{};
      next[q] += step;
    }
  }
  static __device__ __forceinline__ void start(int t, const float* base, int64_t ld, int64_t row0, int64_t rows, int k,
                                               const float* (&next)[NP], bool (&row_ok)[NP]) {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int64_t row = row0 + row_of(t, q);
      row_ok[q] = row < rows;
      next[q] = base + (KM ? (int64_t)(k + k_of(t, q)) * ld + row : row * ld + k + k_of(t, q));
    }
  }
  __device__ __forceinline__ void put(int t, float* lds) const {
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int row = PERM ? permuted(row_of(t, q)) : row_of(t, q);
      *reinterpret_cast<f32x4*>(lds + (KM ? k_of(t, q) * RP + row : row * KP + k_of(t, q))) = v[q];
    }
  }
  static __device__ __forceinline__ float at(const float* lds, int row, int k) { return lds[KM ? k * RP + row : row * KP + k]; }
};

template <bool RK, bool CK, bool GATED, int G, int KS>
__global__ __launch_bounds__(G * 256) void dense_f32_kernel(DenseGemm g) {
  constexpr int NB = GATED ? 2 : 1;
  constexpr int BUF = buf_floats<KS>();
  static_assert((G - 1) * 4 * NB * 4 * 256 <= G * 2 * (1 + NB) * BUF, "the groups' sums fit the operand buffers");
  __shared__ __attribute__((aligned(16))) float lds[G][2][1 + NB][BUF];
  const int group = threadIdx.x >> 8, t = threadIdx.x & 255;
  const int lane = t & 63, wave = t >> 6;
  const int wm = wave >> 1, wn = wave & 1, grp = lane >> 4, r16 = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.x * TM;
  const int n0 = blockIdx.y * TN;
  const int N = g.e.N;
  const float* r = static_cast<const float*>(g.r);
  const float* c = static_cast<const float*>(g.c);
  using SR = Slice<RK, false, KS>;
  using SC = Slice<CK, true, KS>;
  SR sr[2];
  SC sc[2][NB];
  const float *rnext[SR::NP], *cnext[NB][SC::NP];
  bool rok[SR::NP], cok[SC::NP];
  SR::start(t, r, g.ldr, m0, g.M, group * KS, rnext, rok);
#pragma unroll
  for (int b = 0; b < NB; ++b)     // (the up projection's rows follow the N gate rows)
    SC::start(t, c + (int64_t)b * N * g.ldc, g.ldc, n0, N, group * KS, cnext[b], cok);
  const int64_t rstep = (int64_t)G * KS * (RK ? g.ldr : 1), cstep = (int64_t)G * KS * (CK ? g.ldc : 1);
  auto load = [&](int set, int64_t round) __attribute__((always_inline)) {   // called for rounds 0, 1, 2, ... in turn
    const int left = (int)max(int64_t(0), min((int64_t)KS, g.K - (round * G + group) * KS));
    sr[set].load(t, r, rnext, rok, rstep, left);
#pragma unroll
    for (int b = 0; b < NB; ++b) sc[set][b].load(t, c, cnext[b], cok, cstep, left);
  };
  auto put = [&](int set) __attribute__((always_inline)) {
    sr[set].put(t, lds[group][set][0]);
#pragma unroll
    for (int b = 0; b < NB; ++b) sc[set][b].put(t, lds[group][set][1 + b]);
  };
  f32x4 acc[NB][2][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[b][i][j] = f32x4{};
  auto multiply = [&](int set) __attribute__((always_inline)) {
    float fr[KS / 4][2], fc[KS / 4][NB][2];
#pragma unroll
    for (int k = 0; k < KS / 4; ++k) {
#pragma unroll
      for (int i = 0; i < 2; ++i) fr[k][i] = SR::at(lds[group][set][0], wm * 32 + i * 16 + r16, 4 * k + grp);
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) fc[k][b][j] = SC::at(lds[group][set][1 + b], wn * 32 + j * 16 + r16, 4 * k + grp);
    }
    __builtin_amdgcn_sched_barrier(0);   // loads and fragment reads before the products
#pragma unroll
    for (int k = 0; k < KS / 4; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[b][i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fc[k][b][j], fr[k][i], acc[b][i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // round n is in LDS buffer `set`, round n + 1 in the other register set: round n + 2 is loaded (past
  // the end: zeros) while n is multiplied, then n + 1 is stored
  auto step = [&](int set, int64_t n) __attribute__((always_inline)) {
    __syncthreads();     // the stores of round n are done, and so are the reads of the other buffer
    load(set, n + 2);
    multiply(set);
    put(set ^ 1);
  };
  const int64_t rounds = (g.K + G * KS - 1) / (G * KS);
  load(0, 0);
  load(1, 1);
  put(0);
  for (int64_t n = 0; n < rounds; n += 2) {
    step(0, n);
    step(1, n + 1);      // (past the end: zeros)
  }
  if constexpr (G > 1) {
    __syncthreads();     // the operand buffers are free
    f32x4* sums = reinterpret_cast<f32x4*>(&lds[0][0][0][0]);
    if (group > 0) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) sums[(((group - 1) * 4 * NB + (b * 2 + i) * 2 + j) * 256) + t] = acc[b][i][j];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int o = 0; o < G - 1; ++o)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[b][i][j] += sums[((o * 4 * NB + (b * 2 + i) * 2 + j) * 256) + t];
  }
  const int n = n0 + wn * 32 + 8 * grp;
  const EpiBias<float, GATED> bias(g.e, n);
  EpiRes res[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) res[i] = epi_res<float>(g.e, m0 + wm * 32 + i * 16 + r16, g.M, n);
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
    epi_store<float, GATED>(g.e, m, n, z, u, bias, res[i]);
  }
}

template <bool RK, bool CK, bool GATED>
void launch(const DenseGemm& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.M + TM - 1) / TM), (unsigned)((g.e.N + TN - 1) / TN));
  // short contractions (64 x 64 x 2048: 4.5 against 5.8 us) keep one group
  if (g.K < 256) hipLaunchKernelGGL((dense_f32_kernel<RK, CK, GATED, 1, 32>), grid, dim3(256), 0, s, g);
  else hipLaunchKernelGGL((dense_f32_kernel<RK, CK, GATED, 2, 32>), grid, dim3(512), 0, s, g);
}

}  // namespace

hipError_t launch_dense_gemm_f32(const DenseGemm& g, hipStream_t s) {
  if (g.gated) launch<false, false, true>(g, s);
  else if (!g.c_kmajor) launch<false, false, false>(g, s);
  else if (!g.r_kmajor) launch<false, true, false>(g, s);
  else launch<true, true, false>(g, s);
  return hipGetLastError();
}

}  // namespace moe
