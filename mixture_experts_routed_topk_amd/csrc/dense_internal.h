// Launch interfaces of the dense operators around the routed experts: RMS norm, linear
// and gated projections, forward and backward (dense_api.hip checks the arguments).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// ---------------------------------------------------------------------------- RMS norm
struct NormArgs {
  int64_t T;
  int H;
  float eps;
  int64_t ldx, ldr, ldh, ldy;   // row pitches in elements (backward: of dx, dh, h, dy)
  const void* x;
  const void* res;              // residual (backward: dh), may be null
  const void* weight;
  void* y;                      // may be null
  void* h;                      // x + residual (forward, when there is a residual)
  float* rstd;
  uint8_t* q;                   // e4m3 codes [T][H], may be null
  float* q_scale;               // [T][H/128]
  // backward
  const void* dy;
  const void* hin;
  const float* rstd_in;
  void* dx;
  void* dweight;
  float* part;                  // [norm_backward_parts(T, H)][H]
};
hipError_t launch_rms_norm(const NormArgs& a, bool f32, hipStream_t s);
int64_t norm_backward_parts(int64_t T, int H);
hipError_t launch_rms_norm_backward(const NormArgs& a, bool f32, hipStream_t s);

// ---------------------------------------------------------------------------- matrix products
enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActRelu = 3 };

// What becomes of a product's element z = sum_k r[m][k] c[n][k]:
//   z += bias[n]; pre[m][n] = z; out[m][n] = act(z) + res[m][n], or, gated,
//   out[m][n] = act(z_gate) * z_up with the gate in rows [0, I) and the up projection in
//   rows [I, 2I) of the second operand (pre holds both, [m][2I]).
struct DenseEpi {
  void* out;
  int64_t ldo;
  int out_f32;                  // out and res are float32 (else the operands' type)
  const void* bias;             // operands' type, may be null
  const void* res;              // may be null
  int64_t ldr;
  void* pre;                    // operands' type, may be null
  int64_t ldp;
  int act;
  int N;                        // output columns (gated: I)
  int vec;                      // rows of out, res and pre may be accessed in 16-byte pieces
};

// Whether bf16 operands' results are activations kept in float32
__host__ __device__ inline bool wide_act(const DenseEpi& e) { return e.out_f32 && (e.act == kActSilu || e.act == kActGelu); }

// out[M][N] from r (M rows) and c (N rows, gated 2N): element (m, k) of r is r[m * ldr + k],
// or r[k * ldr + m] with r_kmajor; c likewise.  Rows start on 16 bytes, and their last 16-byte
// piece may be read whole: past K it holds zeros, past the rows of a k-major operand anything.
struct DenseGemm {
  const void* r;
  int64_t ldr;
  int r_kmajor;
  const void* c;
  int64_t ldc;
  int c_kmajor;
  int64_t M;
  int64_t K;
  int gated;
  DenseEpi e;
};
// Forward products (both operands stored along k).  Bytes of scratch: the partial sums of a split
// contraction, and of an output that cannot be stored in 16-byte pieces (vec == 0: a second
// kernel stores it by the element).
size_t dense_gemm_workspace(int64_t M, int64_t N, int64_t K, int gated, bool f32, int vec);
hipError_t launch_dense_gemm(const DenseGemm& g, void* ws, bool f32, hipStream_t s);

// The gradients dx [T][N] = dz w (c stored along its rows) and dw [cols][N] = dz^T x (both stored along
// their rows), dz [T][cols]; either may be null.  Outputs in the operands' type, no epilogue.
// two_parts (bf16): dz and x are 2 T rows, dz's second T what rounding took from its first and x's the
// first again with zeros for what is not finite; so dw is over all of dz as it is, and a row of dx is the sum of two of
// dx's 2 T, or the first of them where that is not finite.
size_t dense_gradients_workspace(int64_t rows, int64_t N, int64_t cols, bool f32, bool two_parts);
hipError_t launch_dense_gradients(const DenseGemm* dx, const DenseGemm* dw, void* ws, bool f32, bool two_parts, hipStream_t s);

// The same in float32 (dense_f32.hip)
size_t dense_gemm_f32_workspace(int64_t M, int64_t N, int64_t K, int gated, int vec);
hipError_t launch_dense_gemm_f32(const DenseGemm& g, void* ws, hipStream_t s);
size_t dense_gradients_f32_workspace(int64_t rows, int64_t N, int64_t cols);
hipError_t launch_dense_gradients_f32(const DenseGemm* dx, const DenseGemm* dw, void* ws, hipStream_t s);

// forward products of few rows
bool dense_rows_take(int64_t M, int64_t K, bool f32);
hipError_t launch_dense_rows(const DenseGemm& g, bool f32, hipStream_t s);

// ---------------------------------------------------------------------------- backward
// dz = dy * act'(pre) (gated: [da * up * act'(gate), da * act(gate)]) in the operands' type,
// [T][ldz] with zeros in columns [cols, ldz), and its column sums.
struct DzArgs {
  int64_t T;
  int N;                        // columns of dy (gated: I; dz has 2I)
  int gated;
  int act;
  const void* dy;
  int64_t ldy;
  int dy_f32;                   // dy is float32 (else the operands' type)
  const void* pre;
  int64_t ldp;
  void* dz;                     // may be null: column sums only
  int64_t ldz;
  const void* x;                // with x2: dz is written in two parts (row t and row T + t), and x
  int64_t ldx;                  // [T][K] to both halves of x2 [2T][K], in the second with zeros for infinities and NaN
  void* x2;
  int K;
  float* part;                  // [dz_parts(T)][cols], null without dbias
  void* dbias;                  // operands' type
};
int64_t dz_parts(int64_t T);
hipError_t launch_dz(const DzArgs& a, bool f32, hipStream_t s);

// out[j] = sum_i part[i][j] in the order of i, rounded to bf16 (or float32 with f32)
hipError_t launch_column_sum(const float* part, int64_t rows, int64_t cols, void* out, bool f32, hipStream_t s);
// zeros (T = 0: gradients of parameters)
hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t s);

}  // namespace moe
