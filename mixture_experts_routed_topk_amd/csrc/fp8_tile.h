// Tiles of the e4m3 products with scales for blocks and groups of 128 (gfx950).
//
// out[m][n] = epilogue(sum_kt sr(m, kt) sc(n, kt) sum_{k in slice kt} r[m][k] c[n][k]), r and c e4m3 codes,
// a slice 128 k, sums in float32.  One 16x16x128 block-scaled MFMA multiplies a slice of a fragment pair; inside it
// a slice's products meet with an error of at most 2^-10 of the largest one (1.4e-5 of a
// typical sum), and adding to its accumulator rounds once in float32.
//   FOLD : scales are float32 (any weights'): each MFMA starts from zero and its result is added times sr * sc, an FMA
//          an element.  sc is one value per slice and 128 columns (a weight block's).
//   else : scales are powers of two, bytes by row: the MFMA applies both (a lane passes the bytes of its two
//          operand rows) and accumulates itself, so no vector work is left.
//
// Operands reach LDS by DMA as 128-byte rows, in either storage order (as in dense_tile.h, for bytes):
//   along k    : a row's 128 k, its eight 16-byte chunks XOR-permuted by the row; a lane's 32 k are two of them
//   along rows : a k's 128 rows, chunks XOR-permuted by k; a lane's 32 k are four transposing reads
//                (ds_read_b64_tr_b8: 16 lanes read eight k of 16 rows, and each gets one row's eight k), so that
//                gradients need no transposed copies of the weights
// c sits on the MFMA's row side: a lane ends with four consecutive columns per fragment, and two exchanges between lane
// groups make them eight.
//
// Eight waves in a 2 x 4 grid; a wave's columns are 32 of each half of the tile's 256 (gated: 32 gate and the
// matching 32 up columns).
//   NH = 2, 256 rows, two slices in LDS.  A slice is four phases of a quadrant (64 rows x 32 columns, eight
//   MFMAs); as a phase uses its row fragments for the last time it reads the next phase's into their place:
//     phase   multiplies   half way                                               then reads
//     0       R0 x C0      wait for C1, R1(kt); barrier; DMA of R0, scales, C0(kt+2)   C1(kt)
//     1       R0 x C1                                                             R1(kt)
//     2       R1 x C0      wait for R0, C0(kt+1); barrier; DMA of C1, R1(kt+2)
//     3       R1 x C1                                                             R0, C0(kt+1)
//   Each DMA has a slice and a half to land, and a barrier comes when the reads before it have long ended.
//   NH = 1, 128 rows, three slices in LDS: phases 0 and 1 alone, one barrier and one wait per slice.
#pragma once

#include <type_traits>

#include "dense_tile.h"
#include "fp8_internal.h"

namespace moe {
namespace {

typedef int i32x2v __attribute__((ext_vector_type(2)));

// 16 rows of a 128-row region from row r0 (a multiple of 16), 128 k: lane group g has k 16 g .. 16 g + 15 and 64 + 16 g .. (for
// rows along k its chunks g and 4 + g, whose reads meet no bank twice; with chunks 2 g and 2 g + 1 half of them do)
template <bool KM>
struct Frag8 {
  uint32_t off[2];
  int f;
  __device__ __forceinline__ Frag8(int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!KM) {
#pragma unroll
      for (int h = 0; h < 2; ++h) off[h] = (uint32_t)(i * 128 + (((4 * h + g) ^ (i >> 1)) << 4));
    } else {
      off[0] = (uint32_t)((16 * g + (i >> 1)) * 128 + (i & 1) * 8);
      f = (i >> 1) ^ (g & 1);
    }
  }
  __device__ __forceinline__ i32x8 load(const char* region, int r0) const {
    if constexpr (!KM) {
      const i32x4 a = *reinterpret_cast<const i32x4*>(region + r0 * 128 + off[0]);
      const i32x4 b = *reinterpret_cast<const i32x4*>(region + r0 * 128 + off[1]);
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      typedef __attribute__((address_space(3))) i32x2v lds2;
      const uint32_t p = lds_addr(region) + off[0] + (uint32_t)(((r0 >> 4) ^ f) << 4);
      i32x8 v;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const i32x2v a = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds2*)(p + (t >> 1) * 8192 + (t & 1) * 1024));
        v[2 * t] = a[0];
        v[2 * t + 1] = a[1];
      }
      return v;
    }
  }
};

// This lane's DMA sources for the two instructions of a wave in a region (rows: tile rows of the region, clamped)
template <bool KM>
struct Stream8 {
  uint32_t off[2];
  static __device__ __forceinline__ int chunk_k(int ins, int lane) {
    if constexpr (KM) return ins * 8 + (lane >> 3);
    return ((lane & 7) ^ (((ins * 8 + (lane >> 3)) >> 1) & 7)) * 16;
  }
  static __device__ __forceinline__ int chunk_row(int ins, int lane) {
    if constexpr (!KM) return ins * 8 + (lane >> 3);
    const int k = chunk_k(ins, lane);
    return ((lane & 7) ^ ((k & 7) ^ ((k >> 4) & 1))) * 16;
  }
  template <typename F>
  __device__ __forceinline__ void init(int first, int lane, int64_t ld, F&& row_of) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t row = row_of(chunk_row(first + q, lane));
      off[q] = (uint32_t)(KM ? chunk_k(first + q, lane) * ld + row : row * ld + chunk_k(first + q, lane));
    }
  }
};

struct Fp8Job {
  Job j;
  Fp8Scales rs, cs;
  int c_blocks;
  int E;
  int64_t c_expert, cs_expert;
  Runs runs;
};

// 2^(b - 127); 255 is NaN
__device__ __forceinline__ float ue8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// Two fragments' four columns per lane into eight consecutive ones: lane group g holds columns 4 g .. 4 g + 3 of
// both, and gets 8 g .. 8 g + 7 of the 32
__device__ __forceinline__ void eight_columns(f32x4& a, f32x4& b) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[q]), __float_as_uint(b[q]), false, false);
    const auto y = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
    a[q] = __uint_as_float(y[0]);
    b[q] = __uint_as_float(y[1]);
  }
}

constexpr int kMaxSlices = 512;         // K <= 65536

template <int NH>
struct Ring {
  static constexpr int SLICES = NH == 2 ? 2 : 3;
  static constexpr int STAGE = (NH + 2) * REGION;                 // R0 [R1] C0 C1
  static constexpr int SCALES = (128 * NH + 256) * 4;             // a dword per row of r and, for the MFMA, of c
  static constexpr int TABLE = SLICES * STAGE + 3 * SCALES;       // FOLD: c's block scales, [2 halves][kMaxSlices]
  static constexpr int BYTES = TABLE + 2 * kMaxSlices * 4;
};

// One tile: rows m0 .. of which `rows` exist (tile rows past them repeat the last), columns from tile column nt,
// KT slices from slice kt0 on; c and its scales from expert e.
template <bool RK, bool CK, int EPI, int NH, bool FOLD>
__device__ __forceinline__ void tile_fp8(const Fp8Job& p, const Job& job, int64_t m0, int64_t rows, int nt, int e, int64_t kt0,
                                         int KT, int split, char* lds) {
  using Rg = Ring<NH>;
  const DenseGemm& g = job.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, g4 = lane >> 4;
  const int n0 = nt * (EPI == kGated ? 128 : 256);
  const int64_t k0 = kt0 * 128;
  // tile column -> row of c
  auto c_row = [&](int col) __attribute__((always_inline)) -> int64_t {
    if constexpr (EPI == kGated) return min(n0 + (col & 127), g.e.N - 1) + (int64_t)(col >> 7) * g.e.N;
    return min((int64_t)(n0 + col), (int64_t)job.crows - 1);
  };

  const char* rbase = static_cast<const char*>(g.r) + (RK ? k0 * g.ldr + m0 : m0 * g.ldr + k0);
  const char* cbase = static_cast<const char*>(g.c) + e * p.c_expert + (CK ? k0 * g.ldc + n0 : n0 * g.ldc + k0);
  const int64_t rstep = RK ? 128 * g.ldr : 128, cstep = CK ? 128 * g.ldc : 128;
  // gated: the second column half is the up projection's rows, N rows on (more than 32-bit offsets reach)
  const char* const chalf[2] = {cbase, cbase + (EPI == kGated ? (int64_t)g.e.N * g.ldc : 0)};
  Stream8<RK> sr[NH];
  Stream8<CK> sc[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h < NH)
      sr[h].init(wave * 2, lane, g.ldr, [&](int row) -> int64_t { return min((int64_t)(h * 128 + row), rows - (RK ? 16 : 1)); });
    sc[h].init(wave * 2, lane, g.ldc, [&](int row) -> int64_t {
      if constexpr (EPI == kGated) return min(row, g.e.N - 1 - n0);
      return min((int64_t)(h * 128 + row), (int64_t)job.crows - n0 - (CK ? 16 : 1));
    });
  }
  // Scales by row, a dword each (64 a wave): FOLD: r's, by waves 0 .. 2 NH - 1 (the others bring the same again); else waves
  // 0 .. 3 bring r's and 4 .. 7 c's
  const bool r_wave = FOLD || wave < 4;
  const int s_row = r_wave ? (wave % (2 * NH)) * 64 + lane : (wave - 4) * 64 + lane;
  const Fp8Scales& sp = r_wave ? p.rs : p.cs;
  constexpr int S_SIZE = FOLD ? 4 : 1;
  const int64_t s_at = r_wave ? (m0 + min((int64_t)s_row, rows - 1)) * sp.row
                              : e * p.cs_expert + (p.c_blocks ? c_row(s_row) >> 7 : c_row(s_row)) * sp.row;
  // (a wave's first lane gives the base, so that a lane's offset fits in 32 bits)
  const int64_t s_first = ((int64_t)__builtin_amdgcn_readfirstlane((int)(s_at >> 32)) << 32) |
                          (uint32_t)__builtin_amdgcn_readfirstlane((int)s_at);
  const char* sbase = static_cast<const char*>(sp.p) + (s_first + kt0 * sp.slice) * S_SIZE;
  const uint32_t s_off = (uint32_t)((s_at - s_first) * S_SIZE);
  const uint32_t s_lds = (uint32_t)(Rg::SLICES * Rg::STAGE + (r_wave ? (wave % (2 * NH)) * 256 : NH * 512 + (wave - 4) * 256));
  const int64_t s_step = sp.slice * S_SIZE;
  const uint32_t lds0 = lds_addr(lds);
  const char* const table = lds + Rg::TABLE;      // FOLD: c's block scales of this tile, [2 halves][kMaxSlices] dwords
  auto issue_table = [&]() __attribute__((always_inline)) {
    for (int i0 = wave * 64; i0 < 2 * kMaxSlices; i0 += 512) {
      const int h = i0 / kMaxSlices;
      if (i0 - h * kMaxSlices >= KT) continue;
      const int kt = min(i0 - h * kMaxSlices + lane, KT - 1);
      const int64_t first = e * p.cs_expert + (c_row(h * 128) >> 7) * p.cs.row + kt0 * p.cs.slice;
      const uint32_t dst = lds0 + (uint32_t)(Rg::TABLE + i0 * 4);
      if (p.cs.bytes) dma_lds_u8(static_cast<const uint8_t*>(p.cs.p) + first, (uint32_t)(kt * p.cs.slice), dst);
      else dma_lds_x1(static_cast<const float*>(p.cs.p) + first, (uint32_t)(kt * p.cs.slice * 4), dst);
    }
  };
  // Where slice kt is in the ring
  auto stage = [&](int kt) __attribute__((always_inline)) -> int { return (NH == 2 ? (kt & 1) : kt % 3) * Rg::STAGE; };
  auto issue_r = [&](int h, int kt, int q) __attribute__((always_inline)) {
    dma_lds_x4(rbase + kt * rstep, sr[h].off[q], lds0 + (uint32_t)(stage(kt) + h * REGION + wave * 2048 + q * 1024));
  };
  auto issue_c = [&](int h, int kt, int q) __attribute__((always_inline)) {
    dma_lds_x4(chalf[h] + kt * cstep, sc[h].off[q], lds0 + (uint32_t)(stage(kt) + (NH + h) * REGION + wave * 2048 + q * 1024));
  };
  auto issue_s = [&](int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + s_lds + (uint32_t)(kt % 3 * Rg::SCALES);
    if constexpr (FOLD) dma_lds_x1(sbase + kt * s_step, s_off, dst);
    else dma_lds_u8(sbase + kt * s_step, s_off, dst);
  };
  // a slice's DMA number n: R0, scales, C0 (0 .. 4), C1 (5, 6), R1 (7, 8; of 256 rows)
  auto issue_n = [&](int kt, int n) __attribute__((always_inline)) {
    if (n < 2) issue_r(0, kt, n);
    else if (n == 2) issue_s(kt);
    else if (n < 5) issue_c(0, kt, n - 3);
    else if (n < 7) issue_c(1, kt, n - 5);
    else if constexpr (NH == 2) issue_r(1, kt, n - 7);
  };
  auto issue_slice = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < 5 + 2 * NH; ++n) issue_n(kt, n);
  };

  const Frag8<RK> fr(lane);
  const Frag8<CK> fc(lane);
  f32x4 acc[NH][2][4][2];
#pragma unroll
  for (int a = 0; a < NH; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[a][b][i][j] = f32x4{};
  i32x8 r[4], c[2][2];
  const char* const scales = lds + Rg::SLICES * Rg::STAGE;
  uint32_t rsc[4], csc[2][2];           // FOLD: a half's columns have one scale, csc[h][0]
  auto read_r = [&](int i, int h, int kt) __attribute__((always_inline)) {
    r[i] = fr.load(lds + stage(kt) + h * REGION, wm * 64 + i * 16);
    rsc[i] = *reinterpret_cast<const uint32_t*>(scales + (kt % 3) * Rg::SCALES + (h * 128 + wm * 64 + i * 16 + l16) * 4);
  };
  auto read_c = [&](int h, int kt) __attribute__((always_inline)) {
    const char* s = scales + (kt % 3) * Rg::SCALES + NH * 512 + (h * 128 + wn * 32) * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[h][j] = fc.load(lds + stage(kt) + (NH + h) * REGION, wn * 32 + j * 16);
      if (!FOLD) csc[h][j] = *reinterpret_cast<const uint32_t*>(s + (j * 16 + l16) * 4);
    }
    if (FOLD) csc[h][0] = *reinterpret_cast<const uint32_t*>(table + (h * kMaxSlices + min(kt, kMaxSlices - 1)) * 4);
  };
  // A phase's products; after(i) reads into fragment i's place.  FOLD: a result is folded in three products after its own, when the
  // MFMA has long written it (so a phase's last three in the next one: `before` is the accumulator of the phase before)
  f32x4 pr[4];
  float prs[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) pr[q] = f32x4{}, prs[q] = 0.f;
  auto fold = [&](f32x4& a, int at, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = fmaf(pr[at][q], prs[i], a[q]);
  };
  auto multiply = [&](f32x4 (&a)[4][2], f32x4 (&before)[4][2], int h, auto&& after) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    const float sb = FOLD && p.cs.bytes ? ue8m0_value(csc[h][0]) : __uint_as_float(csc[h][0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (FOLD) {
          const int n = 2 * i + j, old = (n + 5) & 7;
          pr[n & 3] = mfma_16x16x128_e4m3(c[h][j], r[i], f32x4{});
          fold(n < 3 ? before[old >> 1][old & 1] : a[old >> 1][old & 1], old & 3, old >> 1);
          if (j == 1) prs[i] = __uint_as_float(rsc[i]) * sb;
        } else {
          a[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(c[h][j], r[i], a[i][j], 0, 0, 0, (int)csc[h][j], 0, (int)rsc[i]);
        }
      }
      after(i);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto nothing = [](int) __attribute__((always_inline)) {};

  // The loop's body without branches, for slices behind which one is issued or none: across a branch the compiler
  // moves products behind the DMAs and keeps all their operands in registers
  auto body = [&](auto more, int kt) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;
    // published: `younger` DMAs of this wave may be in flight, every read so far is done; then for the workgroup
    auto meet = [&](auto younger) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (MORE) wait_vmcnt<decltype(younger)::value>();
      else wait_vmcnt<0>();
      wait_lds();
      barrier();
    };
    // DMA n of the slice ahead.  They go out one at a time between products: eight waves' bursts behind a barrier would hold
    // up every wave's next product until the addresses of all are taken
    auto ahead = [&](int n) __attribute__((always_inline)) {
      if constexpr (MORE) issue_n(kt + (NH == 2 ? 2 : 3), n);
    };
    if constexpr (NH == 2) {
      multiply(acc[0][0], acc[1][1], 0, [&](int i) __attribute__((always_inline)) {
        if (i == 0) return;
        if (i == 1) {
          meet(std::integral_constant<int, 9>{});     // C1, R1(kt) are here; younger: kt + 1
          read_c(1, kt);
        }
        ahead(i - 1);
        __builtin_amdgcn_sched_barrier(0);
      });
      multiply(acc[0][1], acc[0][0], 1, [&](int i) __attribute__((always_inline)) {
        read_r(i, 1, kt);
        if (i & 1) ahead(3 + i / 2);
      });
      multiply(acc[1][0], acc[0][1], 0, [&](int i) __attribute__((always_inline)) {
        if (i == 1) meet(std::integral_constant<int, 9>{});   // R0, C0(kt + 1); younger: C1, R1(kt + 1) and R0, scales, C0(kt + 2)
        if (i & 1) ahead(5 + i / 2);
        __builtin_amdgcn_sched_barrier(0);
      });
      read_c(0, kt + 1);                              // (behind the last slice: what the ring holds, not used)
      multiply(acc[1][1], acc[1][0], 1, [&](int i) __attribute__((always_inline)) {
        read_r(i, 0, kt + 1);
        if (i & 1) ahead(7 + i / 2);
      });
    } else {
      read_c(1, kt);
      multiply(acc[0][0], acc[0][1], 0, nothing);
      multiply(acc[0][1], acc[0][0], 1, [&](int i) __attribute__((always_inline)) {
        if (i == 0) return;
        if (i == 1) {
          meet(std::integral_constant<int, 7>{});     // slice kt + 1; younger: kt + 2
          read_c(0, kt + 1);
          read_r(0, 0, kt + 1);
        }
        read_r(i, 0, kt + 1);
#pragma unroll
        for (int n = 0; n < 7; ++n)
          if (n / 3 == i - 1 || (n == 6 && i == 3)) ahead(n);
      });
    }
  };
  constexpr int AHEAD = NH == 2 ? 2 : 3;
  if (KT > 0) {
    if constexpr (FOLD) issue_table();
    issue_slice(0);
    if (KT > 1) issue_slice(1);
    if (NH == 1 && KT > 2) issue_slice(2);
    if (KT >= AHEAD) wait_vmcnt<NH == 2 ? 13 : 14>();
    else wait_vmcnt<0>();
    barrier();                             // slice 0 has landed (of 256 rows, R0 and C0)
#pragma unroll
    for (int i = 0; i < 4; ++i) read_r(i, 0, 0);
    read_c(0, 0);
    int kt = 0;
    for (; kt + AHEAD < KT; ++kt) body(std::true_type{}, kt);
    for (; kt < KT; ++kt) body(std::false_type{}, kt);
    if constexpr (FOLD) {
#pragma unroll
      for (int n = 5; n < 8; ++n) fold(acc[NH - 1][1][n >> 1][n & 1], n & 3, n >> 1);
    }
  }

#pragma unroll
  for (int a = 0; a < NH; ++a) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) eight_columns(acc[a][b][i][0], acc[a][b][i][1]);
    const int64_t m = m0 + a * 128 + wm * 64 + l16;
    const int col = n0 + wn * 32 + 8 * g4;
    if constexpr (EPI == kGated) {
      store_rows<uint16_t, EPI>(job, split, m, col, acc[a][0], acc[a][1]);
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) store_rows<uint16_t, EPI>(job, split, m, col + b * 128, acc[a][b], acc[a][b]);
    }
  }
}

// Forward and dx: rows in tiles, over one matrix (splits along blockIdx.y) or by runs of rows
template <bool CK, int EPI, int NH, bool FOLD>
__global__ __launch_bounds__(512, 1) void fp8_rows_tile_kernel(Fp8Job p) {
  __shared__ __attribute__((aligned(1024))) char lds[Ring<NH>::BYTES];
  Job job = p.j;
  if (p.E) job.mt = p.runs.count[0];
  int mt, nt;
  if (!tile_of(job, blockIdx.x, mt, nt)) return;
  int64_t m0 = (int64_t)mt * 128 * NH, rows = job.g.M - m0;
  int e = 0;
  if (p.E) {
    const RowTile t = p.runs.tiles[mt];
    m0 = t.row0;
    rows = t.rows;
    e = t.expert;
    job.g.M = m0 + rows;
  }
  const int64_t kt0 = (int64_t)blockIdx.y * job.slices;
  const int KT = (int)min((int64_t)job.slices, job.g.K / 128 - kt0);
  tile_fp8<false, CK, EPI, NH, FOLD>(p, job, m0, rows, nt, e, kt0, KT, blockIdx.y, lds);
}

// dw: contractions over the rows in tiles of 128 (a run's last filled up with zeros): all of them (splits along
// blockIdx.y) or each run's (run blockIdx.y)
template <int NH>
__global__ __launch_bounds__(512, 1) void fp8_dw_kernel(Fp8Job p) {
  __shared__ __attribute__((aligned(1024))) char lds[Ring<NH>::BYTES];
  Job job = p.j;
  int mt, nt;
  if (!tile_of(job, blockIdx.x, mt, nt)) return;
  const int64_t m0 = (int64_t)mt * 128 * NH;
  int64_t kt0;
  int KT, split = 0;
  if (p.E) {
    const int e = blockIdx.y;
    kt0 = p.runs.group[e];
    KT = (int)(p.runs.group[e + 1] - kt0);
    job.g.e.out = static_cast<uint16_t*>(job.g.e.out) + (int64_t)e * job.g.M * job.g.e.N;
  } else {
    split = blockIdx.y;
    kt0 = (int64_t)split * job.slices;
    KT = (int)min((int64_t)job.slices, job.g.K / 128 - kt0);
  }
  tile_fp8<true, true, kGrad, NH, false>(p, job, m0, job.g.M - m0, nt, 0, kt0, KT, split, lds);
}

inline Fp8Job fp8_job(const Fp8Gemm& g, const Job& job) {
  Fp8Job p{};
  p.j = job;
  p.rs = g.rs;
  p.cs = g.cs;
  p.c_blocks = g.c_blocks;
  p.E = g.E;
  p.c_expert = g.c_expert;
  p.cs_expert = g.cs_expert;
  p.runs = g.runs;
  return p;
}
inline dim3 fp8_grid(const Job& job, int y) {
  return dim3((unsigned)(((int64_t)job.mt * job.nt + 7) / 8 * 8), (unsigned)y);
}

// Costs of a tile, as in dense_plan.h, in slices of 128 k
constexpr TileCost kTilesFp8[] = {{256, 256, 1, 1.25, 1.25, 7.0}, {128, 256, 1, 0.8, 0.8, 4.0}};
constexpr JoinCost kJoinFp8 = {2.8, 3.36e6};

inline Plan plan_fp8(int64_t M, int64_t N, int64_t K, int gated) {
  return plan_forward<uint8_t>(kTilesFp8, kJoinFp8, M, N, K, gated);
}

}  // namespace
}  // namespace moe
