// Launch interfaces of the e4m3 products with block scales, their gradients and the quantisers
// in front of them (fp8_api.hip checks the arguments).
#pragma once

#include "dense_internal.h"

namespace moe {

constexpr int kFp8Group = 128;        // elements that share a scale, and k of a slice

// ---------------------------------------------------------------------------- runs of rows
// Where each expert's rows are, and the rows cut into tiles that do not cross experts.  Made on the
// device from offsets [E + 1], whose values are taken into [0, T] and made non-decreasing, so that no table leads outside.
struct RowTile {
  int32_t expert;
  int32_t start, end;   // the expert's rows
  int32_t first, count; // its tiles
  int32_t pad[3];
};
struct Runs {
  int32_t* group;       // [E + 1]: 128-row tiles before the expert's
  int32_t* order;       // [E]: the experts with rows, then those without
  int32_t* count;       // [3]: tiles, 128-row tiles, experts with rows
  RowTile* tiles;       // of `height` rows
  RowTile* groups;      // of 128 rows; the same as tiles with height == 128
  int height;
};
// At most this many tiles
inline int64_t max_row_tiles(int64_t T, int E, int height) { return T / height + (T < E ? T : E); }
size_t runs_bytes(int64_t T, int E, int height);
Runs runs_at(void* ws, int64_t T, int E, int height);
hipError_t launch_runs(const Runs& r, const int32_t* offsets, int64_t T, int E, hipStream_t s);

// ---------------------------------------------------------------------------- quantisers
// What the backward products read.  dz = dy * act'(pre) (gated: [da * up * act'(gate), da * act(gate)]), [T][cols], in
// groups of 128 columns (zr, for dx) and of 128 rows of its expert (zc, for dw), x in groups of 128 rows (xc).  zc and xc are
// stored by 128-row tiles, each with its own 128 rows (zeros past the run's end), so that dw contracts over whole ones.
// Scales are powers of two: bytes (UE8M0), or float32 for zr with zr_f32.
struct GroupsArgs {
  int64_t T;
  int N;                        // columns of dy (gated: I; dz has 2 I)
  int gated;
  int act;
  const void* dy;               // bf16
  int64_t ldy;
  const void* pre;              // bf16, null without an activation
  int64_t ldp;
  uint8_t* zr;                  // [T][cols], null without dx
  void* zr_scale;               // [T][cols / 128]
  int zr_f32;
  uint8_t* zc;                  // [128-row tiles][128][cols], null without dw
  uint8_t* zc_scale;            // [128-row tiles][cols]
  const void* x;                // bf16
  int64_t ldx;
  int K;
  uint8_t* xc;                  // [128-row tiles][128][K], null without dw
  uint8_t* xc_scale;            // [128-row tiles][K]
  float* part;                  // [128-row tiles][cols] sums of dz, null without dbias
  const RowTile* tiles;         // null: one run of T rows
  const int32_t* count;
  int64_t max_tiles;
};
hipError_t launch_groups(const GroupsArgs& a, hipStream_t s);

// e4m3 codes of `count` matrices [N][K] with one scale per 128 x 128 block
hipError_t launch_blocks(const void* w, bool f32, int count, int N, int K, bool ue8m0, uint8_t* q, void* scale, hipStream_t s);

// ---------------------------------------------------------------------------- products
// out[M][N] from e4m3 codes r (M rows) and c (N rows, gated 2 N), stored as in DenseGemm; element sizes and pitches of r and c
// are bytes.  An operand's scale of row i and slice kt (128 k) is entry i * row + kt * slice of its scales; c's
// row counts in blocks of 128 rows when c_blocks.  Entries are float32, or bytes (2^(b - 127)).
struct Fp8Scales {
  const void* p;
  int64_t row, slice;
  int bytes;
};
struct Fp8Gemm {
  DenseGemm g;                  // epilogue in bf16; g.M: all rows
  Fp8Scales rs, cs;
  int c_blocks;
  // runs of rows, each with its own c (forward and dx) or its own output (dw: contractions over the runs)
  int E;                        // 0: none
  int64_t c_expert;             // bytes from an expert's c to the next one's
  int64_t cs_expert;            // entries
  const int32_t* offsets;       // few rows: the runs themselves, without tables
  Runs runs;
  int few;                      // forward: the kernel of few rows takes it (fp8_rows_take)
};
// Rows of the tiles that a product by runs takes: forward, K x cols weights an expert, and dx
int fp8_grouped_height(int64_t T, int E, int64_t K, int64_t cols);
int fp8_dx_height(int64_t T, int E, int64_t cols, bool ue8m0);
size_t fp8_gemm_workspace(const Fp8Gemm& g);
hipError_t launch_fp8_gemm(const Fp8Gemm& g, void* ws, hipStream_t s);
// dx: r (codes [T][cols]) along k, c along its rows; dw: both along their rows, g.K: rows of all 128-row tiles.  Either may be null.
size_t fp8_gradients_workspace(int64_t T, int64_t N, int64_t cols, int E);
hipError_t launch_fp8_gradients(const Fp8Gemm* dx, const Fp8Gemm* dw, void* ws, hipStream_t s);

// forward products of few rows, M in all (E: over the runs)
bool fp8_rows_take(int64_t M, int64_t K, int E, bool gated);
hipError_t launch_fp8_rows(const Fp8Gemm& g, hipStream_t s);

}  // namespace moe
