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
// groups make them eight; plain bf16 results are turned into rows in LDS instead (Patch).
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
// One workgroup a CU takes one tile after another, and the DMAs run on: the next tile's first slices arrive during a
// tile's last ones and its stores.  (A workgroup per tile: 2.6 us of first DMAs and 1.8 us between workgroups beside 1.8 us a slice.)
//
// A slice of 256 x 256 x 128 is 2048 cycles of MFMAs on each SIMD.  Measured: 2670 with the MFMA's own scales, 3500 to 3600
// with FOLD, 4130 for dw, whose short contractions lie between bursts of stores.  The clock falls to 1.4 to 1.9 GHz under
// these kernels (it depends on the codes): with three quarters of the FMAs left out a slice takes as long, in fewer
// cycles.  8192 x 8192 x 8192 of random codes: 526 to 530 us (2.08 PFLOP/s) with powers of two as weights' scales in either format (the
// forward folds both), 535 with other float32 ones.  16384 rows of 32 runs, 2048 -> 7168: 325 us (1.48 PFLOP/s, 0.74 GB).  Gated,
// 8192 x 7168 -> 2 x 2048 with saved projections: 240 us (2.0).  dx and dw of 16384 rows of 32 runs, 7168 <- 2 x 2048: 1200 us (1.6, beside 2.1 GB of results).
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

// Where instruction `ins` (1 KB) of a 128-row region takes lane `lane`'s 16 bytes from: tile row and k (along rows: first row of the
// chunk and its k)
template <bool KM>
struct Chunk8 {
  static __device__ __forceinline__ int k(int ins, int lane) {
    if constexpr (KM) return ins * 8 + (lane >> 3);
    return ((lane & 7) ^ (((ins * 8 + (lane >> 3)) >> 1) & 7)) * 16;
  }
  static __device__ __forceinline__ int row(int ins, int lane) {
    if constexpr (!KM) return ins * 8 + (lane >> 3);
    const int kk = k(ins, lane);
    return ((lane & 7) ^ ((kk & 7) ^ ((kk >> 4) & 1))) * 16;
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
constexpr int kMaxDxSlices = 1024;      // of dx, which contracts over up to 2 x 65536 columns

// This lane's number, formed anew (from a zero that the compiler does not know to be one): what follows from it is computed
// where it is used, once a tile, and not kept in registers through the loop
__device__ __forceinline__ int lane_again() {
  int zero = 0;
  asm volatile("" : "+v"(zero));
  return (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, (uint32_t)zero));
}

// The kernel's argument number J, read from memory again: what a tile needs once does not occupy scalar registers in the loop.
// (Kernels take one or two of these and nothing in front of them.)
template <int J>
__device__ __forceinline__ const Fp8Job& argument() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return ((const Fp8Job*)p)[J];
}

// The values are formed here: products that only later code reads would be moved there, behind branches, and their
// operands kept in registers until then.  (No instruction: nothing is read.)
__device__ __forceinline__ void formed(f32x4 (&a)[4][2]) {
  asm volatile("" : "+v"(a[0][0]), "+v"(a[0][1]), "+v"(a[1][0]), "+v"(a[1][1]), "+v"(a[2][0]), "+v"(a[2][1]), "+v"(a[3][0]), "+v"(a[3][1]));
}

template <int NH, bool FOLD>
struct Ring {
  static constexpr int SLICES = NH == 2 ? 2 : 3;                  // in LDS, and how far the DMAs are ahead
  static constexpr int STAGE = (NH + 2) * REGION;                 // R0 [R1] C0 C1
  static constexpr int SCALES = (128 * NH + 256) * 4;             // a dword per row of r and, for the MFMA, of c
  static constexpr int TABLE = SLICES * STAGE + 3 * SCALES;       // FOLD: c's block scales of NT tiles, [2 halves][slices]
  static constexpr int BYTES = 160 * 1024;
  // 1 KB a wave through which results turn into rows (Patch); 128-row tiles leave no room for it beside the longest tables
  static constexpr bool PATCHED = NH == 2 || !FOLD;
  static constexpr int PATCH = BYTES - (PATCHED ? 8 * 1024 : 0);
  static constexpr int TABLES = PATCH - TABLE;
  // Slices of the longest contraction whose block scales TABLES holds for two tiles: the next one's arrive while a tile's last slices
  // still read theirs
  static constexpr int LONGEST = TABLES / 4 / 4 / 64 * 64;
};
static_assert(Ring<1, true>::LONGEST >= kMaxSlices && Ring<2, true>::LONGEST >= kMaxDxSlices, "two tiles' block scales");
constexpr int kLongestShortTile = Ring<1, true>::LONGEST;      // 704: longer contractions with float32 block scales take 256-row tiles

// 16 x 32 bf16 results of a wave, turned in LDS: lane l has row l & 15, columns 4 (l >> 4) and 16 further on, and gets row l >> 2, eight columns from
// 8 (l & 3) on.  Four neighbouring lanes then store 64 bytes of a row, where the results as they are formed would go out in
// pieces of 8 or, exchanged between lane groups, 16.  A row's four 16-byte pieces are XOR-permuted by row / 4 (no bank conflicts).  LDS executes
// a wave's accesses in order, so that nothing waits but the store.
struct Patch {
  char *to, *to16;
  const char* from;
  __device__ __forceinline__ Patch(char* patch, int lane) {
    const uint32_t at = (lane & 15) * 64 + ((((lane >> 5) ^ (lane >> 2)) & 3) << 4) + (lane >> 4 & 1) * 8;
    to = patch + at;
    to16 = patch + (at ^ 32);
    from = patch + (lane >> 2) * 64 + (((lane ^ (lane >> 4)) & 3) << 4);
  }
  __device__ __forceinline__ i32x4 turn(const f32x4 (&z)[2]) const {
    *reinterpret_cast<i32x2v*>(to) = i32x2v{(int)pack_bf16x2(z[0][0], z[0][1]), (int)pack_bf16x2(z[0][2], z[0][3])};
    *reinterpret_cast<i32x2v*>(to16) = i32x2v{(int)pack_bf16x2(z[1][0], z[1][1]), (int)pack_bf16x2(z[1][2], z[1][3])};
    __builtin_amdgcn_wave_barrier();
    const i32x4 v = *reinterpret_cast<const i32x4*>(from);
    __builtin_amdgcn_wave_barrier();
    return v;
  }
};
// What the table kernel wrote: read through the scalar cache (a vector load would have the compiler wait for every DMA in flight)
__device__ __forceinline__ int table_entry(const void* table, int64_t i) {
  typedef const __attribute__((address_space(4))) int32_t* Table;
  return ((Table)(uintptr_t)table)[i];
}

// A tile of the product: rows m0 .. of which `rows` exist (tile rows past them repeat the last), columns from tile column
// nt, KT slices from kt0 on; c, its scales and dw's output from expert e
struct Tile {
  int64_t m0;
  int rows, nt, e, split;
  int kt0, KT;
};
// Forward and dx: row tiles of one matrix (with splits of the contraction) or of runs of rows
struct RowTiles {
  static __device__ __forceinline__ int count(const Fp8Job& p) {
    return (p.E ? table_entry(p.runs.count, 0) : p.j.mt * p.j.splits) * p.j.nt;
  }
  template <int NH>
  static __device__ __forceinline__ Tile at(const Fp8Job& p, int t) {
    Tile x{};
    Job j = p.j;
    if (p.E) {
      // an expert's tiles follow one another: entry t / nt of the list is one of its row tiles
      const int64_t at = (int64_t)(t / j.nt) * (sizeof(RowTile) / 4);
      x.e = table_entry(p.runs.tiles, at);
      const int start = table_entry(p.runs.tiles, at + 1), end = table_entry(p.runs.tiles, at + 2);
      j.mt = table_entry(p.runs.tiles, at + 4);
      int mt;
      tile_at(j, t - table_entry(p.runs.tiles, at + 3) * j.nt, mt, x.nt);
      x.m0 = start + mt * 128 * NH;
      x.rows = min(128 * NH, end - (int)x.m0);
      x.KT = j.slices;
    } else {
      const int per = j.mt * j.nt;
      x.split = t / per;
      int mt;
      tile_at(j, t - x.split * per, mt, x.nt);
      x.m0 = (int64_t)mt * 128 * NH;
      x.rows = (int)min((int64_t)128 * NH, j.g.M - x.m0);
      x.kt0 = x.split * j.slices;
      x.KT = min(j.slices, (int)(j.g.K / 128) - x.kt0);
    }
    return x;
  }
};
// dw: contractions over 128-row tiles, all of them (with splits) or each run's
struct DwTiles {
  static __device__ __forceinline__ int count(const Fp8Job& p) { return (p.E ? table_entry(p.runs.count, 2) : p.j.splits) * p.j.mt * p.j.nt; }
  template <int NH>
  static __device__ __forceinline__ Tile at(const Fp8Job& p, int t) {
    Tile x{};
    const int per = p.j.mt * p.j.nt, part = t / per;
    int mt;
    tile_at(p.j, t - part * per, mt, x.nt);
    x.m0 = (int64_t)mt * 128 * NH;
    x.rows = (int)min((int64_t)128 * NH, p.j.g.M - x.m0);
    if (p.E) {
      x.e = table_entry(p.runs.order, part);
      x.kt0 = table_entry(p.runs.group, x.e);
      x.KT = table_entry(p.runs.group, x.e + 1) - x.kt0;
    } else {
      x.split = part;
      x.kt0 = part * p.j.slices;
      x.KT = min(p.j.slices, (int)(p.j.g.K / 128) - x.kt0);
    }
    return x;
  }
};

// Which tiles of a job a workgroup takes: each by itself would go round all G workgroups.  Where another job's last round
// leaves `heavy` of them with a tile more, the others take `extra` tiles of this one first; the last rounds then
// begin at the less loaded ones.
struct Share {
  int G, heavy, early, at;      // early: tiles that go to the others first; at: this workgroup's place in the full rounds
  __device__ __forceinline__ Share(int q, int workgroups, int heavy_, int extra, bool others_first) {
    G = workgroups;
    heavy = heavy_;
    early = heavy ? extra * (G - heavy) : 0;
    at = !others_first ? q : q < heavy ? q + G - heavy : q - heavy;
  }
  __device__ __forceinline__ int first(int q) const { return q >= heavy && early > 0 ? q - heavy : early + at; }
  __device__ __forceinline__ int next(int t) const {
    if (t >= early) return t + G;
    t += G - heavy;
    return t < early ? t : early + at;
  }
};

// Workgroups go to the eight XCDs in turn: each XCD takes a run of neighbouring tiles of every round, so that the 32 that run
// on it together are 8 x 4 and share their operands in its L2
__device__ __forceinline__ int place_in_round() { return (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3); }

// This workgroup's tiles of job J
template <typename TILES, int J, bool RK, bool CK, int EPI, int NH, bool FOLD>
__device__ __forceinline__ void run_tiles(const Fp8Job& p, char* lds, const Share& share) {
  using Rg = Ring<NH, FOLD>;
  constexpr int AHEAD = Rg::SLICES;
  constexpr int DMAS = 5 + 2 * NH;             // of a wave and slice
  const DenseGemm& g = p.j.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15;
  const int total = TILES::count(p);
  const int first = share.first(place_in_round());
  if (first >= total) return;
  const uint32_t lds0 = lds_addr(lds);
  barrier();                                   // (a job before may still be read)

  // ------------------------------------------------------------------ DMAs: a cursor over tiles and their slices, on the one issued last
  int at_tile = first, left;                   // the tile, and how many of its slices are still to be issued
  const char *rbase, *cbase[2], *sbase;
  uint32_t roff[NH][2], coff[2][2], soff;
  int64_t rstep = RK ? 128 * g.ldr : 128, cstep = CK ? 128 * g.ldc : 128;      // bytes from a slice to the next
  constexpr int S_SIZE = FOLD ? 4 : 1;
  // Scales by row, a dword each (64 a wave): FOLD: r's, by waves 0 .. 2 NH - 1 (the others bring the same again); else waves
  // 0 .. 3 bring r's and 4 .. 7 c's
  const bool r_wave = FOLD || wave < 4;
  int64_t s_step = (r_wave ? p.rs.slice : p.cs.slice) * S_SIZE;
  const uint32_t s_lds = (uint32_t)(Rg::SLICES * Rg::STAGE + (r_wave ? (wave % (2 * NH)) * 256 : NH * 512 + (wave - 4) * 256));
  int table_at = 0;                            // FOLD: where the next tile's block scales go (dwords), as table_of below
  auto table_next = [&](int at, int KT) __attribute__((always_inline)) -> int {
    const int next = at + 2 * ((KT + 63) & ~63);           // (whole DMAs of 64)
    return next + 2 * ((KT + 63) & ~63) > Rg::TABLES / 4 ? 0 : next;
  };
  auto open = [&]() __attribute__((always_inline)) {         // addresses of tile at_tile
    const Fp8Job& p = argument<J>();
    const DenseGemm& g = p.j.g;
    const Tile x = TILES::template at<NH>(p, at_tile);
    const int lane = lane_again();
    left = x.KT;
    const int n0 = x.nt * (EPI == kGated ? 128 : 256);
    const int64_t k0 = (int64_t)x.kt0 * 128;
    // tile column -> row of c
    auto c_row = [&](int col) __attribute__((always_inline)) -> int64_t {
      if constexpr (EPI == kGated) return min(n0 + (col & 127), g.e.N - 1) + (int64_t)(col >> 7) * g.e.N;
      return min((int64_t)(n0 + col), (int64_t)p.j.crows - 1);
    };
    rbase = static_cast<const char*>(g.r) + (RK ? k0 * g.ldr + x.m0 : x.m0 * g.ldr + k0) - rstep;
    cbase[0] = static_cast<const char*>(g.c) + x.e * p.c_expert + (CK ? k0 * g.ldc + n0 : n0 * g.ldc + k0) - cstep;
    // gated: the second column half is the up projection's rows, N rows on (more than 32-bit offsets reach)
    cbase[1] = cbase[0] + (EPI == kGated ? (int64_t)g.e.N * g.ldc : 0);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int ins = wave * 2 + q;
        if (h < NH) {
          const int row = min(h * 128 + Chunk8<RK>::row(ins, lane), x.rows - (RK ? 16 : 1));
          roff[h][q] = (uint32_t)(RK ? Chunk8<RK>::k(ins, lane) * g.ldr + row : row * g.ldr + Chunk8<RK>::k(ins, lane));
        }
        int col = Chunk8<CK>::row(ins, lane);
        if constexpr (EPI == kGated) col = min(col, g.e.N - 1 - n0);
        else col = min(h * 128 + col, p.j.crows - n0 - (CK ? 16 : 1));
        coff[h][q] = (uint32_t)(CK ? Chunk8<CK>::k(ins, lane) * g.ldc + col : col * g.ldc + Chunk8<CK>::k(ins, lane));
      }
    const int s_row = (r_wave ? wave % (2 * NH) : wave - 4) * 64 + lane;
    const int64_t s_at = r_wave ? (x.m0 + min(s_row, x.rows - 1)) * p.rs.row
                                : x.e * p.cs_expert + (p.c_blocks ? c_row(s_row) >> 7 : c_row(s_row)) * p.cs.row;
    // (a wave's first lane gives the base, so that a lane's offset fits in 32 bits)
    const int64_t s_first = ((int64_t)__builtin_amdgcn_readfirstlane((int)(s_at >> 32)) << 32) |
                            (uint32_t)__builtin_amdgcn_readfirstlane((int)s_at);
    sbase = static_cast<const char*>(r_wave ? p.rs.p : p.cs.p) + (s_first + x.kt0 * (r_wave ? p.rs.slice : p.cs.slice)) * S_SIZE - s_step;
    soff = (uint32_t)((s_at - s_first) * S_SIZE);
    if constexpr (FOLD) {                      // c's block scales of the whole tile
      const int half = (x.KT + 63) >> 6;
      for (int i = wave; i < 2 * half; i += 8) {
        const int h = i >= half;
        const int kt = min((i - h * half) * 64 + lane, x.KT - 1);
        const int64_t from = x.e * p.cs_expert + (c_row(h * 128) >> 7) * p.cs.row + x.kt0 * p.cs.slice;
        const uint32_t dst = lds0 + (uint32_t)(Rg::TABLE + (table_at + i * 64) * 4);
        if (p.cs.bytes) dma_lds_u8(static_cast<const uint8_t*>(p.cs.p) + from, (uint32_t)(kt * p.cs.slice), dst);
        else dma_lds_x1(static_cast<const float*>(p.cs.p) + from, (uint32_t)(kt * p.cs.slice * 4), dst);
      }
      table_at = table_next(table_at, x.KT);
    }
  };
  // DMA number n of the cursor's slice into the ring at `stage`, its scales at `place`: R0, scales, C0 (0 .. 4), C1 (5, 6), R1 (7, 8; of 256 rows)
  auto issue = [&](int n, int stage, int place) __attribute__((always_inline)) {
    const uint32_t to = lds0 + (uint32_t)(stage + wave * 2048);
    if (n < 2) dma_lds_x4(rbase, roff[0][n], to + n * 1024);
    else if (n == 2) {
      const uint32_t dst = lds0 + s_lds + (uint32_t)place;
      if constexpr (FOLD) dma_lds_x1(sbase, soff, dst);
      else dma_lds_u8(sbase, soff, dst);
    }
    else if (n < 5) dma_lds_x4(cbase[0], coff[0][n - 3], to + NH * REGION + (n - 3) * 1024);
    else if (n < 7) dma_lds_x4(cbase[1], coff[1][n - 5], to + (NH + 1) * REGION + (n - 5) * 1024);
    else if constexpr (NH == 2) dma_lds_x4(rbase, roff[1][n - 7], to + REGION + (n - 7) * 1024);
  };
  auto step = [&]() __attribute__((always_inline)) { rbase += rstep, cbase[0] += cstep, cbase[1] += cstep, sbase += s_step; };
  // Behind a slice's DMAs.  (Behind the last tile's last slice the cursor stays on it: what it brings again is not read.)
  auto advance = [&]() __attribute__((always_inline)) {
    if (--left > 0) return;
    const int next = share.next(at_tile);
    if (next < total) {
      at_tile = next;
      open();
    } else {
      rstep = cstep = s_step = 0;
      left = 0x7fffffff;
    }
  };

  // ------------------------------------------------------------------ products
  const Frag8<RK> fr(lane);
  const Frag8<CK> fc(lane);
  f32x4 acc[NH][2][4][2];
  i32x8 r[4], c[2][2];
  uint32_t rsc[4], csc[2][2];                  // FOLD: a half's columns have one scale, csc[h][0]
  int now = 0, sp = 0;                         // where the current slice is in the ring, and its scales (bytes)
  const char* table = lds + Rg::TABLE;         // FOLD: block scales of the current tile from the current slice on
  int table_half = 0;                          // and from one half to the other (bytes)
  auto after = [](int place, int size, int n) __attribute__((always_inline)) -> int {
    return n == 2 ? place ^ size : place == (n - 1) * size ? 0 : place + size;
  };
  auto read_r = [&](int i, int h, int stage, int s) __attribute__((always_inline)) {
    r[i] = fr.load(lds + stage + h * REGION, wm * 64 + i * 16);
    rsc[i] = *reinterpret_cast<const uint32_t*>(lds + Rg::SLICES * Rg::STAGE + s + (h * 128 + wm * 64 + i * 16 + l16) * 4);
  };
  auto read_c = [&](int h, int stage, int s, const char* t) __attribute__((always_inline)) {
    const char* from = lds + Rg::SLICES * Rg::STAGE + s + NH * 512 + (h * 128 + wn * 32) * 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[h][j] = fc.load(lds + stage + (NH + h) * REGION, wn * 32 + j * 16);
      if (!FOLD) csc[h][j] = *reinterpret_cast<const uint32_t*>(from + (j * 16 + l16) * 4);
    }
    if (FOLD) csc[h][0] = *reinterpret_cast<const uint32_t*>(t + h * table_half);
  };
  // A phase's products; then(i) reads into fragment i's place.  FOLD: a result is folded in three products after its own, when the
  // MFMA has long written it (so a phase's last three in the next one: `before` is the accumulator of the phase before)
  f32x4 pr[4];
  float prs[4];
  auto fold = [&](f32x4& a, int at, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) a[q] = fmaf(pr[at][q], prs[i], a[q]);
  };
  auto multiply = [&](f32x4 (&a)[4][2], f32x4 (&before)[4][2], int h, auto&& then) __attribute__((always_inline)) {
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
      then(i);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // A slice, without branches
  auto body = [&]() __attribute__((always_inline)) {
    const int next = after(now, Rg::STAGE, Rg::SLICES), sn = after(sp, Rg::SCALES, 3), s2 = after(sn, Rg::SCALES, 3);
    // published: `younger` DMAs (or stores) of this wave may be in flight, every read so far is done; then for the workgroup
    auto meet = [&](auto younger) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<decltype(younger)::value>();
      wait_lds();
      barrier();
    };
    // DMA n of the slice ahead, into the current one's place.  They go out one at a time between products: eight waves'
    // bursts behind a barrier would hold up every wave's next product until the addresses of all are taken
    auto ahead = [&](int n) __attribute__((always_inline)) { issue(n, now, NH == 2 ? s2 : sp); };
    if constexpr (NH == 2) {
      multiply(acc[0][0], acc[1][1], 0, [&](int i) __attribute__((always_inline)) {
        if (i == 0) {
          step();
          return;
        }
        if (i == 1) {
          meet(std::integral_constant<int, 9>{});     // C1, R1 of this slice are here; younger: the next slice
          read_c(1, now, sp, table);
        }
        ahead(i - 1);
        __builtin_amdgcn_sched_barrier(0);
      });
      multiply(acc[0][1], acc[0][0], 1, [&](int i) __attribute__((always_inline)) {
        read_r(i, 1, now, sp);
        if (i & 1) ahead(3 + i / 2);
      });
      multiply(acc[1][0], acc[0][1], 0, [&](int i) __attribute__((always_inline)) {
        if (i == 1) meet(std::integral_constant<int, 9>{});   // the next slice's R0, C0; younger: its C1, R1 and R0, scales, C0 of the one ahead
        if (i & 1) ahead(5 + i / 2);
        __builtin_amdgcn_sched_barrier(0);
      });
      read_c(0, next, sn, table + 4);                 // (behind the last slice: what the ring holds, not used)
      multiply(acc[1][1], acc[1][0], 1, [&](int i) __attribute__((always_inline)) {
        read_r(i, 0, next, sn);
        if (i & 1) ahead(7 + i / 2);
      });
    } else {
      read_c(1, now, sp, table);
      multiply(acc[0][0], acc[0][1], 0, [&](int i) __attribute__((always_inline)) {
        if (i == 0) step();
      });
      multiply(acc[0][1], acc[0][0], 1, [&](int i) __attribute__((always_inline)) {
        if (i == 0) return;
        if (i == 1) {
          meet(std::integral_constant<int, 7>{});     // the next slice; younger: the one behind it
          read_c(0, next, sn, table + 4);
          read_r(0, 0, next, sn);
        }
        read_r(i, 0, next, sn);
#pragma unroll
        for (int n = 0; n < 7; ++n)
          if (n / 3 == i - 1 || (n == 6 && i == 3)) ahead(n);
      });
    }
    now = next;
    sp = sn;
    table += 4;
#pragma unroll
    for (int a = 0; a < NH; ++a) formed(acc[a][0]), formed(acc[a][1]);
    if constexpr (FOLD) asm volatile("" : "+v"(pr[1]), "+v"(pr[2]), "+v"(pr[3]));
  };

  open();
#pragma unroll
  for (int a = 0; a < AHEAD; ++a) {
    step();
#pragma unroll
    for (int n = 0; n < DMAS; ++n) issue(n, a * Rg::STAGE, a * Rg::SCALES);
    advance();
  }
  wait_vmcnt<0>();                             // (the first slices)
  barrier();
  int table_of = 0;
  for (int t = first; t < total; t = share.next(t)) {
    const Tile x = TILES::template at<NH>(argument<J>(), t);
    const int n0 = x.nt * (EPI == kGated ? 128 : 256);
    if constexpr (FOLD) {
      table = lds + Rg::TABLE + table_of * 4;
      table_half = ((x.KT + 63) & ~63) * 4;
      table_of = table_next(table_of, x.KT);
    }
#pragma unroll
    for (int a = 0; a < NH; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[a][b][i][j] = f32x4{};
#pragma unroll
    for (int q = 0; q < 4; ++q) pr[q] = f32x4{}, prs[q] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) read_r(i, 0, now, sp);
    read_c(0, now, sp, table);
    for (int kt = 0; kt < x.KT; ++kt) {
      body();
      advance();
    }
    if constexpr (FOLD) {
#pragma unroll
      for (int n = 5; n < 8; ++n) fold(acc[NH - 1][1][n >> 1][n & 1], n & 3, n >> 1);
    }
    const Fp8Job& q = argument<J>();
    Job job = q.j;
    job.g.M = x.m0 + x.rows;
    job.g.e.out_f32 = 0;                       // (what is known of these products' epilogue)
    job.g.e.vec = 1;
    if constexpr (EPI == kGated) job.g.e.bias = job.g.e.res = nullptr;
    if constexpr (std::is_same_v<TILES, DwTiles>) {
      job.g.M = q.j.g.M;
      if (q.E) job.g.e.out = static_cast<uint16_t*>(job.g.e.out) + (int64_t)x.e * job.g.M * job.g.e.N;
    } else if (!q.E) {
      job.g.M = q.j.g.M;
    }
    if (Rg::PATCHED && EPI == kGrad && !job.part) {
      const int who = lane_again();
      const Patch patch(lds + Rg::PATCH + wave * 1024, who);
#pragma unroll
      for (int a = 0; a < NH; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int col = n0 + b * 128 + wn * 32;
          if (col >= job.g.e.N) continue;
          const int64_t m = x.m0 + a * 128 + wm * 64 + (who >> 2);
          uint16_t* out = static_cast<uint16_t*>(job.g.e.out) + col + 8 * (who & 3);
          i32x4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = patch.turn(acc[a][b][i]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (m + 16 * i < job.g.M) *reinterpret_cast<i32x4*>(out + (m + 16 * i) * job.g.e.ldo) = v[i];
          __builtin_amdgcn_sched_barrier(0);
        }
    } else {
#pragma unroll
      for (int a = 0; a < NH; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
#pragma unroll
          for (int i = 0; i < 4; ++i) eight_columns(acc[a][b][i][0], acc[a][b][i][1]);
          if (EPI == kGated && b == 0) continue;
          __builtin_amdgcn_sched_barrier(0);
          const int who = lane_again();
          const int64_t m = x.m0 + a * 128 + wm * 64 + (who & 15);
          const int col = n0 + wn * 32 + 8 * (who >> 4);
          if constexpr (EPI == kGated) store_rows<uint16_t, EPI>(job, x.split, m, col, acc[a][0], acc[a][1]);
          else store_rows<uint16_t, EPI>(job, x.split, m, col + b * 128, acc[a][b], acc[a][b]);
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  }
  wait_vmcnt<0>();                             // no DMA outlives the workgroup's LDS
}

// One workgroup a CU
template <int EPI, int NH>
__global__ __launch_bounds__(512, 1) void fp8_forward_kernel(Fp8Job p) {
  __shared__ __attribute__((aligned(1024))) char lds[Ring<NH, true>::BYTES];
  run_tiles<RowTiles, 0, false, false, EPI, NH, true>(p, lds, Share(place_in_round(), gridDim.x, 0, 0, false));
}

// Both gradients: the product with the shorter tiles fills the other's uneven end
struct Fill {
  int dw;             // which product fills
  int extra;          // tiles of it that take as long as one of the other's
  int others_first;
};
template <int NX, int NW, bool FOLD>
__global__ __launch_bounds__(512, 1) void fp8_gradients_kernel(Fp8Job dx, Fp8Job dw, Fill fill) {
  __shared__ __attribute__((aligned(1024))) char lds[Ring<2, true>::BYTES];
  static_assert(Ring<1, true>::BYTES == Ring<2, true>::BYTES, "one buffer for both");
  const int G = gridDim.x, q = place_in_round();
  const int heavy = (fill.dw ? RowTiles::count(argument<0>()) : DwTiles::count(argument<1>())) % G;
  const bool others = fill.others_first && heavy;
  run_tiles<DwTiles, 1, true, true, kGrad, NW, false>(argument<1>(), lds, Share(q, G, fill.dw ? heavy : 0, fill.extra, fill.dw && others));
  run_tiles<RowTiles, 0, false, true, kGrad, NX, FOLD>(argument<0>(), lds, Share(q, G, fill.dw ? 0 : heavy, fill.extra, !fill.dw && others));
  if (!dw.E || !dw.j.nt) return;
  // experts without rows: zeros
  const int64_t size = dw.j.g.M * dw.j.g.e.N / 8;          // 16-byte pieces of one expert's dw
  for (int i = dw.runs.count[2]; i < dw.E; ++i) {
    i32x4* out = reinterpret_cast<i32x4*>(dw.j.g.e.out) + dw.runs.order[i] * size;
    for (int64_t k = (int64_t)blockIdx.x * 512 + threadIdx.x; k < size; k += (int64_t)gridDim.x * 512) out[k] = i32x4{};
  }
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
inline dim3 fp8_grid(int64_t tiles) { return dim3((unsigned)(tiles < 256 ? (tiles + 7) / 8 * 8 : 256)); }

// Costs of a forward product's tiles, as in dense_plan.h, in slices of 128 k.  Fitted to 68 products of 40 to 16384 rows, each
// measured with both heights and every split (rms error 10%; the choices take 1.1% longer than the best measured, 14% at most).
constexpr TileCost kTilesFp8[] = {{256, 256, 1, 1.55, 1.55, 5.3}, {128, 256, 1, 0.96, 0.96, 3.8}};
constexpr JoinCost kJoinFp8 = {5.6, 3.9e6};

inline Plan plan_fp8(int64_t M, int64_t N, int64_t K, int gated) {
  return plan_forward<uint8_t>(kTilesFp8, kJoinFp8, M, N, K, gated);
}

}  // namespace
}  // namespace moe
