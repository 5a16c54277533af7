// Matrix products of the dense operators in bf16 on MFMA (gfx950).
//
// out[m][n] = epilogue(sum_k r[m][k] c[n][k]) (DenseGemm), float32 sums.  Three forms occur:
// forward (both operands stored along k), dx (c stored along n) and dw (both stored along
// their rows).  One pair of operand readers serves all of them:
//
//   along k    : a tile row is 128 bytes of LDS per slice of 64 k, its eight 16-byte chunks
//                XOR-permuted by the row, so the 16 rows of a fragment read hit distinct banks;
//                a fragment is one 16-byte read per lane.
//   along rows : a k row is 256 bytes of LDS (128 rows of the tile), its eight 32-byte units
//                XOR-permuted by k; a fragment is two transposing 8-byte reads per lane
//                (ds_read_tr16_b64: each group of 16 lanes reads four k rows of 16 elements and
//                every lane gets one column), so neither form needs a transposed copy in HBM.
//
// Both arrive by global->LDS DMA; the permutation is applied to the global addresses.  The
// last slice of a contraction that ends inside it takes its missing chunks from a zero
// chunk in memory, so both operands are zero there.  Rows past the matrix repeat its last one
// and are not stored.
//
// c sits on the MFMA's row side with its rows permuted (fragment j, row q: column 8 (q / 4) +
// 4 j + q % 4), so two fragments of a lane are eight consecutive columns of one output row:
// results leave the registers in 16-byte pieces without a pass through LDS.
#include <math.h>

#include "dense_device.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int KS = 64;                    // k per slice
constexpr int REGION = 128 * KS * 2;      // bytes of 128 operand rows in a slice (16 KB)

__device__ const i32x4 zero_chunk[1] = {{0, 0, 0, 0}};

__device__ __forceinline__ void dma_lds_x4_at(const void* p, uint32_t m0) {   // address per lane
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(m0) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void fence() { asm volatile("" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  fence();
  __builtin_amdgcn_s_barrier();
  fence();
}

// kPartial: float32 sums to job.part; kGrad: those, or with one split the plain bf16 result
enum { kLinear = 0, kGated = 1, kPartial = 2, kGrad = 3 };

// ---------------------------------------------------------------------------- DMA
// Where instruction `ins` (1 KB) of a 128-row region takes lane `lane`'s 16 bytes from.
struct Chunk {
  int row;    // tile row within the region (along k) or first of eight rows (along rows)
  int k;      // first k of the chunk (along k) or the k row (along rows)
};
template <bool KM, bool CSIDE>
__device__ __forceinline__ Chunk chunk_of(int ins, int lane) {
  Chunk c;
  if constexpr (!KM) {
    c.row = ins * 8 + (lane >> 3);
    const int swz = CSIDE ? (((c.row >> 1) & 1) | (((c.row >> 3) & 3) << 1)) : ((c.row >> 1) & 7);
    c.k = ((lane & 7) ^ swz) * 8;
  } else {
    c.k = ins * 4 + (lane >> 4);
    const int f = CSIDE ? 2 * (c.k & 3) : ((c.k & 3) | (((c.k >> 3) & 1) << 2));
    const int pos = lane & 15;
    c.row = (((pos >> 1) ^ f) * 2 + (pos & 1)) * 8;
  }
  return c;
}

// ---------------------------------------------------------------------------- fragments
// 16 rows x 32 k (k step s) of a region from row r0 (a multiple of 16)
template <bool KM>
struct RowFrag {
  uint32_t off[2];
  int f;
  __device__ __forceinline__ RowFrag(int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!KM) {
#pragma unroll
      for (int s = 0; s < 2; ++s) off[s] = (uint32_t)(i * 128 + (((4 * s + g) ^ (i >> 1)) << 4));
    } else {
      off[0] = (uint32_t)((8 * g + (i >> 2)) * 256 + (i & 3) * 8);
      f = (i >> 2) | ((g & 1) << 2);
    }
  }
  __device__ __forceinline__ bf16x8 load(const char* region, int r0, int s) const {
    if constexpr (!KM) {
      return *reinterpret_cast<const bf16x8*>(region + r0 * 128 + off[s]);
    } else {
      const char* p = region + off[0] + (((r0 >> 4) ^ f) << 5) + s * 32 * 256;
      return tr_pair(p, p + 4 * 256);
    }
  }
  static __device__ __forceinline__ bf16x8 tr_pair(const char* p, const char* q) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)lds_addr(p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)lds_addr(q));
    const s16x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
};
// fragment j of the 32 columns from c0 (a multiple of 32): row q is column c0 + 8 (q / 4) + 4 j + q % 4
template <bool KM>
struct ColFrag {
  uint32_t off[2];
  int f, half;
  __device__ __forceinline__ ColFrag(int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!KM) {
      const int swz = ((i >> 1) & 1) | ((i >> 2) << 1);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        off[s] = (uint32_t)((8 * (i >> 2) + (i & 3)) * 128 + (((4 * s + g) ^ swz) << 4));
    } else {
      off[0] = (uint32_t)((8 * g + (i >> 2)) * 256 + (i & 1) * 16);
      f = 2 * ((i >> 2) & 3);
      half = (i & 3) >> 1;
    }
  }
  __device__ __forceinline__ bf16x8 load(const char* region, int c0, int j, int s) const {
    if constexpr (!KM) {
      return *reinterpret_cast<const bf16x8*>(region + (c0 + 4 * j) * 128 + off[s]);
    } else {
      const char* p = region + off[0] + ((((c0 >> 4) + half) ^ f) << 5) + 8 * j + s * 32 * 256;
      return RowFrag<true>::tr_pair(p, p + 4 * 256);
    }
  }
};

// ---------------------------------------------------------------------------- operand streams
struct Job {
  DenseGemm g;
  int mt, nt;          // tiles
  int splits;          // contraction split over blockIdx.y
  int slices;          // slices of one split
  int crows;           // rows of c (gated: 2 I)
  float* part;         // [splits][M][ldpart] partial sums (splits > 1)
  int64_t ldpart;
};

// This lane's DMA sources for NI instructions (first, first + 1, ...) of one region whose
// rows are tile rows base_row .. base_row + 127
template <bool KM, bool CSIDE, int NI>
struct Stream {
  uint32_t off[NI];
  // row_of(tile row) gives the row's distance from the operand's tile origin, clamped
  template <typename F>
  __device__ __forceinline__ void init(int first, int lane, int64_t ld, F&& row_of) {
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      const Chunk c = chunk_of<KM, CSIDE>(first + q, lane);
      off[q] = KM ? (uint32_t)(c.k * ld * 2 + row_of(c.row) * 2) : (uint32_t)(row_of(c.row) * ld * 2 + c.k * 2);
    }
  }
  // full slice: base = operand tile origin advanced to the slice
  __device__ __forceinline__ void issue(const char* base, uint32_t lds, int q) const { dma_lds_x4(base, off[q], lds); }
  // last slice with `left` k in it
  __device__ __forceinline__ void issue_tail(const char* base, uint32_t lds, int q, int first, int lane, int left) const {
    const Chunk c = chunk_of<KM, CSIDE>(first + q, lane);
    const char* p = c.k < left ? base + off[q] : reinterpret_cast<const char*>(zero_chunk);
    dma_lds_x4_at(p, lds);
  }
};

// Tile (mt, nt) of workgroup b.  Consecutive workgroups go to the eight XCDs in turn; each XCD
// takes a contiguous run of tiles, ordered in groups of 8 tile rows with the row fastest, so
// the 32 tiles that run together on an XCD are 8 x 4 and share their operands in its L2.
__device__ __forceinline__ bool tile_of(const Job& job, int b, int& mt, int& nt) {
  const int total = job.mt * job.nt;
  const int per = (total + 7) >> 3;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= total) return false;
  const int grp = t / (8 * job.nt);
  const int rows = min(8, job.mt - grp * 8);
  const int l = t - grp * 8 * job.nt;
  mt = grp * 8 + l % rows;
  nt = l / rows;
  return true;
}

// Stores FM pieces of eight columns from n on: piece i is row m + 16 i, its sums acc[i] (and, gated, up[i])
template <int EPI, int FM>
__device__ __forceinline__ void store_rows(const Job& job, int split, int64_t m, int n, const f32x4 (&acc)[FM][2],
                                           const f32x4 (&up)[FM][2]) {
  const DenseEpi& e = job.g.e;
  if (EPI == kGrad && !job.part) {
    if (n >= e.N) return;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (m + 16 * i >= job.g.M) continue;
      float z[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] = acc[i][v >> 2][v & 3];
      Piece<uint16_t>::store(e.out, (m + 16 * i) * e.ldo + n, z);
    }
  } else if constexpr (EPI == kPartial || EPI == kGrad) {
    if (n >= job.crows) return;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (m + 16 * i >= job.g.M) continue;
      f32x4* out = reinterpret_cast<f32x4*>(job.part + ((int64_t)split * job.g.M + m + 16 * i) * job.ldpart + n);
      out[0] = acc[i][0];
      out[1] = acc[i][1];
    }
  } else {
    if (n >= e.N) return;
    const EpiBias<uint16_t, EPI == kGated> bias(e, n);
    EpiRes res[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) res[i] = epi_res<uint16_t>(e, m + 16 * i, job.g.M, n);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (m + 16 * i >= job.g.M) continue;
      float z[8], u[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] = acc[i][v >> 2][v & 3], u[v] = up[i][v >> 2][v & 3];
      epi_store_vec<uint16_t, EPI == kGated>(e, m + 16 * i, n, z, u, bias, res[i]);
    }
  }
}

// ---------------------------------------------------------------------------- 256 x 256 tiles
// Eight waves (two per SIMD) in a 2 x 4 grid, each 128 x 64 of the tile as four quadrants (64
// rows of row half 0 or 1 x 32 columns of column half 0 or 1).  A slice is four phases of one
// quadrant, 16 MFMAs; the fragments of a phase are read from LDS one phase ahead, so a wave's MFMAs
// never wait for its own reads, and the SIMD's other wave fills what is left:
//   phase   multiplies   reads            issues (DMA)
//   0       R0 x C0      C1(kt)           R0(kt+2)
//   1       R0 x C1      R1(kt)           C0(kt+2)     then: wait for R0, C0(kt+1); barrier
//   2       R1 x C0      R0(kt+1)         C1(kt+2)
//   3       R1 x C1      C0(kt+1)         R1(kt+2)     then: wait for C1, R1(kt+1); barrier
// Two slices live in LDS.  Each barrier publishes the regions read in the next two phases and frees
// those read in the last two, which the next two phases refill: a DMA has four to six phases
// (more than a slice's MFMA time) to land.  DMAs retire in issue order, two per region
// and wave, which gives the vmcnt of each wait.
constexpr int kLds256 = 2 * 4 * REGION;   // [slice parity][R0 R1 C0 C1]
template <bool RK, bool CK, int EPI>
__device__ __forceinline__ void tile_256(const Job& job, int block, int split, char* lds) {
  int mt, nt;
  if (!tile_of(job, block, mt, nt)) return;
  const DenseGemm& g = job.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int64_t m0 = (int64_t)mt * 256;
  const int n0 = nt * (EPI == kGated ? 128 : 256);
  const int64_t k0 = (int64_t)split * job.slices * KS;
  const int KT = (int)min((int64_t)job.slices, (g.K - k0 + KS - 1) / KS);
  const int left = (int)min((int64_t)KS, g.K - k0 - (int64_t)(KT - 1) * KS);   // k in the last slice

  // operand tile origins and the bytes from one slice to the next
  const char* rbase = static_cast<const char*>(g.r) + (RK ? k0 * g.ldr + m0 : m0 * g.ldr + k0) * 2;
  const char* cbase = static_cast<const char*>(g.c) + (CK ? k0 * g.ldc + n0 : (int64_t)n0 * g.ldc + k0) * 2;
  const int64_t rstep = RK ? (int64_t)KS * g.ldr * 2 : KS * 2, cstep = CK ? (int64_t)KS * g.ldc * 2 : KS * 2;
  Stream<RK, false, 2> sr[2];
  Stream<CK, true, 2> sc[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sr[h].init(wave * 2, lane, g.ldr, [&](int row) -> int64_t {
      // (along rows: whole chunks of eight)
      const int64_t last = RK ? (g.M - 1 - m0) / 8 * 8 : g.M - 1 - m0;
      return min((int64_t)(h * 128 + row), last);
    });
    sc[h].init(wave * 2, lane, g.ldc, [&](int row) -> int64_t {
      if constexpr (EPI == kGated) return (int64_t)h * g.e.N + min(row, g.e.N - 1 - n0);
      const int last = CK ? (job.crows - 1 - n0) / 8 * 8 : job.crows - 1 - n0;
      return min(h * 128 + row, last);
    });
  }
  const uint32_t lds0 = lds_addr(lds);
  auto issue_r = [&](int h, int kt) __attribute__((always_inline)) {
    const char* base = rbase + kt * rstep;
    const uint32_t dst = lds0 + (uint32_t)(((kt & 1) * 4 + h) * REGION + wave * 2048);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (kt == KT - 1 && left < KS) sr[h].issue_tail(base, dst + q * 1024, q, wave * 2, lane, left);
      else sr[h].issue(base, dst + q * 1024, q);
    }
  };
  auto issue_c = [&](int h, int kt) __attribute__((always_inline)) {
    const char* base = cbase + kt * cstep;
    const uint32_t dst = lds0 + (uint32_t)(((kt & 1) * 4 + 2 + h) * REGION + wave * 2048);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (kt == KT - 1 && left < KS) sc[h].issue_tail(base, dst + q * 1024, q, wave * 2, lane, left);
      else sc[h].issue(base, dst + q * 1024, q);
    }
  };

  const RowFrag<RK> fr(lane);
  const ColFrag<CK> fc(lane);
  f32x4 acc[2][2][4][2];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[a][b][i][j] = f32x4{};
  bf16x8 r0[4][2], r1[4][2], c0[2][2], c1[2][2];
  auto read_r = [&](bf16x8 (&r)[4][2], int h, int kt) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s) r[i][s] = fr.load(lds + ((kt & 1) * 4 + h) * REGION, wm * 64 + i * 16, s);
  };
  auto read_c = [&](bf16x8 (&c)[2][2], int h, int kt) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int s = 0; s < 2; ++s) c[j][s] = fc.load(lds + ((kt & 1) * 4 + 2 + h) * REGION, wn * 32, j, s);
  };
  auto multiply = [&](f32x4 (&a)[4][2], const bf16x8 (&r)[4][2], const bf16x8 (&c)[2][2]) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) a[i][j] = mfma_16x16x32_bf16(c[j][s], r[i][s], a[i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };
  // this wave's reads are done and (but for the youngest `more` regions) its DMAs have landed; the
  // barrier makes both hold for the workgroup
  auto publish = [&](bool more) __attribute__((always_inline)) {
    if (more) wait_vmcnt<8>();
    else wait_vmcnt<0>();
    wait_lds();
    barrier();
  };

  issue_r(0, 0), issue_c(0, 0), issue_c(1, 0), issue_r(1, 0);
  if (KT > 1) issue_r(0, 1), issue_c(0, 1), issue_c(1, 1), issue_r(1, 1);
  publish(KT > 1);
  read_r(r0, 0, 0);
  read_c(c0, 0, 0);
  wait_lds();
  barrier();       // (phase 0 refills what was just read)
  for (int kt = 0; kt < KT; ++kt) {
    const bool more = kt + 2 < KT, next = kt + 1 < KT;
    read_c(c1, 1, kt);
    if (more) issue_r(0, kt + 2);
    multiply(acc[0][0], r0, c0);

    read_r(r1, 1, kt);
    if (more) issue_c(0, kt + 2);
    multiply(acc[0][1], r0, c1);
    publish(more);

    if (next) read_r(r0, 0, kt + 1);
    if (more) issue_c(1, kt + 2);
    multiply(acc[1][0], r1, c0);

    if (next) read_c(c0, 0, kt + 1);
    if (more) issue_r(1, kt + 2);
    multiply(acc[1][1], r1, c1);
    publish(more);
  }

  const int row = lane & 15, col = 8 * (lane >> 4);
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int64_t m = m0 + a * 128 + wm * 64 + row;
    if constexpr (EPI == kGated) {
      store_rows<EPI>(job, split, m, n0 + wn * 32 + col, acc[a][0], acc[a][1]);
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) store_rows<EPI>(job, split, m, n0 + b * 128 + wn * 32 + col, acc[a][b], acc[a][b]);
    }
  }
}

template <bool RK, bool CK, int EPI>
__global__ __launch_bounds__(512, 1) void dense_256_kernel(Job job) {
  __shared__ __attribute__((aligned(1024))) char lds[kLds256];
  tile_256<RK, CK, EPI>(job, blockIdx.x, blockIdx.y, lds);
}

// ---------------------------------------------------------------------------- RR x 128 tiles
// Four waves (2 x 2), two slices in LDS, one barrier per slice; two (RR = 128) or three (RR =
// 64) workgroups share a CU, so one's waits are covered by the others' MFMAs.  A wave's
// columns are 32 of each half of the tile (gated: 32 gate and the matching 32 up columns).
template <int RR>
constexpr int lds_128() { return 2 * (RR * KS * 2 + REGION); }
template <int RR, bool RK, bool CK, int EPI>
__device__ __forceinline__ void tile_128(const Job& job, int block, int split, char* lds) {
  constexpr int FM = RR / 32;                              // 16-row fragments per wave
  constexpr int RBYTES = RR * KS * 2, STAGE = RBYTES + REGION;
  constexpr int NR = RBYTES / 4096, NC = REGION / 4096;    // DMA instructions per wave and slice
  static_assert(RR == 128 || !RK, "rows stored along k come in regions of 128");
  int mt, nt;
  if (!tile_of(job, block, mt, nt)) return;
  const DenseGemm& g = job.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (int64_t)mt * RR;
  const int n0 = nt * (EPI == kGated ? 64 : 128);
  const int64_t k0 = (int64_t)split * job.slices * KS;
  const int KT = (int)min((int64_t)job.slices, (g.K - k0 + KS - 1) / KS);
  const int left = (int)min((int64_t)KS, g.K - k0 - (int64_t)(KT - 1) * KS);
  const char* rbase = static_cast<const char*>(g.r) + (RK ? k0 * g.ldr + m0 : m0 * g.ldr + k0) * 2;
  const char* cbase = static_cast<const char*>(g.c) + (CK ? k0 * g.ldc + n0 : (int64_t)n0 * g.ldc + k0) * 2;
  const int64_t rstep = RK ? (int64_t)KS * g.ldr * 2 : KS * 2, cstep = CK ? (int64_t)KS * g.ldc * 2 : KS * 2;
  Stream<RK, false, NR> sr;
  Stream<CK, true, NC> sc;
  sr.init(wave * NR, lane, g.ldr, [&](int row) -> int64_t {
    const int64_t last = RK ? (g.M - 1 - m0) / 8 * 8 : g.M - 1 - m0;
    return min((int64_t)row, last);
  });
  sc.init(wave * NC, lane, g.ldc, [&](int row) -> int64_t {
    if constexpr (EPI == kGated) return (int64_t)(row >> 6) * g.e.N + min(row & 63, g.e.N - 1 - n0);
    const int last = CK ? (job.crows - 1 - n0) / 8 * 8 : job.crows - 1 - n0;
    return min(row, last);
  });
  const uint32_t lds0 = lds_addr(lds);
  auto issue = [&](int kt) __attribute__((always_inline)) {
    const uint32_t dst = lds0 + (uint32_t)((kt & 1) * STAGE);
    const char* rb = rbase + kt * rstep;
    const char* cb = cbase + kt * cstep;
    if (kt == KT - 1 && left < KS) {
#pragma unroll
      for (int q = 0; q < NR; ++q) sr.issue_tail(rb, dst + (wave * NR + q) * 1024, q, wave * NR, lane, left);
#pragma unroll
      for (int q = 0; q < NC; ++q) sc.issue_tail(cb, dst + RBYTES + (wave * NC + q) * 1024, q, wave * NC, lane, left);
    } else {
#pragma unroll
      for (int q = 0; q < NR; ++q) sr.issue(rb, dst + (wave * NR + q) * 1024, q);
#pragma unroll
      for (int q = 0; q < NC; ++q) sc.issue(cb, dst + RBYTES + (wave * NC + q) * 1024, q);
    }
  };
  const RowFrag<RK> fr(lane);
  const ColFrag<CK> fc(lane);
  f32x4 acc[2][FM][2];
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[b][i][j] = f32x4{};

  issue(0);
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<0>();     // slice kt has landed
    wait_lds();          // (and the reads of slice kt - 1 are done: its buffer is refilled next)
    barrier();
    if (kt + 1 < KT) issue(kt + 1);
    const char* R = lds + (kt & 1) * STAGE;
    const char* C = R + RBYTES;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8 r[FM], c[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) c[b][j] = fc.load(C, b * 64 + wn * 32, j, s);
#pragma unroll
      for (int i = 0; i < FM; ++i) r[i] = fr.load(R, wm * (RR / 2) + i * 16, s);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[b][i][j] = mfma_16x16x32_bf16(c[b][j], r[i], acc[b][i][j]);
    }
  }
  const int col = n0 + wn * 32 + 8 * (lane >> 4);
  const int64_t m = m0 + wm * (RR / 2) + (lane & 15);
  if constexpr (EPI == kGated) {
    store_rows<EPI>(job, split, m, col, acc[0], acc[1]);
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) store_rows<EPI>(job, split, m, col + b * 64, acc[b], acc[b]);
  }
}

template <int RR, bool RK, bool CK, int EPI>
__global__ __launch_bounds__(256, 2) void dense_128_kernel(Job job) {
  __shared__ __attribute__((aligned(1024))) char lds[lds_128<RR>()];
  tile_128<RR, RK, CK, EPI>(job, blockIdx.x, blockIdx.y, lds);
}

// ---------------------------------------------------------------------------- both gradients in one launch
// dx (r along k) in tiles of TA rows and dw (both operands along their rows) in tiles of TB: two
// products that do not depend on each other share the CUs, so one's last tiles are
// covered by the other's (2731 x 2048 x 5632: 352 and 704 tiles of 128 x 128 on 512 places, 75 us
// and 70 us one after the other).  The product with the longer tiles comes first.  Blocks
// [0, n_first) belong to the first one; a split's blocks follow one another.
template <int TA, int TB>
__global__ __launch_bounds__(TA == 256 ? 512 : 256, TA == 256 ? 1 : 2) void dense_pair_kernel(Job dx, Job dw, int n_first,
                                                                                             int dw_first) {
  constexpr int L = TA == 256 ? kLds256 : lds_128<128>();
  __shared__ __attribute__((aligned(1024))) char lds[L];
  const bool first = (int)blockIdx.x < n_first;
  const int b = first ? blockIdx.x : blockIdx.x - n_first;
  if (first == (dw_first != 0)) {
    const int n = (dw.mt * dw.nt + 7) / 8 * 8;
    if constexpr (TB == 256) tile_256<true, true, kGrad>(dw, b % n, b / n, lds);
    else tile_128<TB, true, true, kGrad>(dw, b % n, b / n, lds);
  } else {
    const int n = (dx.mt * dx.nt + 7) / 8 * 8;
    if constexpr (TA == 256) tile_256<false, true, kGrad>(dx, b % n, b / n, lds);
    else tile_128<TA, false, true, kGrad>(dx, b % n, b / n, lds);
  }
}

// ---------------------------------------------------------------------------- sum of the splits
// Adds the splits' partial sums in their order and applies the epilogue; one thread per eight columns.
template <bool GATED>
__device__ __forceinline__ void join(const Job& job, int64_t i) {
  const int n8 = (job.g.e.N + 7) / 8;
  if (i >= job.g.M * n8) return;
  const int64_t m = i / n8;
  const int n = (int)(i - m * n8) * 8;
  const EpiBias<uint16_t, GATED> bias(job.g.e, n);
  const EpiRes res = epi_res<uint16_t>(job.g.e, m, job.g.M, n);
  float z[8] = {}, u[8] = {};
  for (int s = 0; s < job.splits; ++s) {
    float v[8];
    const int64_t at = ((int64_t)s * job.g.M + m) * job.ldpart + n;
    Piece<float>::load(job.part, at, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] += v[j];
    if constexpr (GATED) {
      Piece<float>::load(job.part, at + job.g.e.N, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] += v[j];
    }
  }
  epi_store<uint16_t, GATED>(job.g.e, m, n, z, u, bias, res);
}

template <bool GATED>
__global__ __launch_bounds__(256) void dense_join_kernel(Job job) {
  join<GATED>(job, (int64_t)blockIdx.x * 256 + threadIdx.x);
}
__global__ __launch_bounds__(256) void dense_join_pair_kernel(Job a, Job b, int n_first) {
  if ((int)blockIdx.x < n_first) join<false>(a, (int64_t)blockIdx.x * 256 + threadIdx.x);
  else join<false>(b, (int64_t)(blockIdx.x - n_first) * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------- plan
struct Plan {
  int tile;      // 256, 128 or 64 (rows of a tile)
  int splits;
  int slices;    // per split
};

// The tile and split with the least estimated time.  Tiles go over the 256 CUs in rounds of the
// workgroups that a CU holds; a slice takes a workgroup at least `alone` us, and `shared` us of its CU;
// `fixed` us go to a tile's first DMA and epilogue, and a split adds a second launch and a pass over its
// partial sums.  The constants are fitted to 43 products of 60 to 8192 rows, each measured with every
// tile and split (rms error of the estimate 13%; the choices take 1.6% longer than the best ones).
struct TileCost {
  int rows, cols, per_cu;
  double alone, shared, fixed;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 1.115, 1.115, 7.0}, {128, 128, 2, 0.549, 0.38, 0.57}, {64, 128, 3, 0.328, 0.251, 0.02}};
constexpr double kJoinUs = 2.8, kJoinBytesPerUs = 3.36e6;
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};

Plan plan(int64_t M, int64_t N, int64_t K, int gated) {
  const int64_t cols = gated ? 2 * N : N;
  const int64_t KT = (K + KS - 1) / KS;
  Plan best{128, 1, (int)KT};
  double best_us = 1e30;
  for (const TileCost& t : kTiles) {
    const int64_t tiles = ((M + t.rows - 1) / t.rows) * ((cols + t.cols - 1) / t.cols);
    for (int want : kSplits) {
      if (want > 1 && KT / want < 3) break;
      const int64_t per = (KT + want - 1) / want;
      const int s = (int)((KT + per - 1) / per);      // (every split has slices)
      const int64_t queue = (tiles * s + 255) / 256;  // workgroups of one CU
      const int64_t rest = queue % t.per_cu;
      double us = (queue / t.per_cu) * (per * fmax(t.alone, t.per_cu * t.shared) + t.fixed);
      if (rest) us += per * fmax(t.alone, rest * t.shared) + t.fixed;
      if (s > 1) us += kJoinUs + (double)M * cols * 4 * (s + 1) / kJoinBytesPerUs;
      if (us < best_us) best_us = us, best = Plan{t.rows, s, (int)per};
    }
  }
  return best;
}
int64_t part_pitch(int64_t N, int gated) { return ((gated ? 2 * N : N) + 7) / 8 * 8; }

template <int EPI>
hipError_t launch_tiles(const Job& job, int tile, hipStream_t s) {
  const int total = job.mt * job.nt;
  const dim3 grid((unsigned)((total + 7) / 8 * 8), (unsigned)job.splits);
  if (tile == 256) hipLaunchKernelGGL((dense_256_kernel<false, false, EPI>), grid, dim3(512), 0, s, job);
  else if (tile == 128) hipLaunchKernelGGL((dense_128_kernel<128, false, false, EPI>), grid, dim3(256), 0, s, job);
  else hipLaunchKernelGGL((dense_128_kernel<64, false, false, EPI>), grid, dim3(256), 0, s, job);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------- plan of the gradients
struct PairPlan {
  int tiles;                     // index into kPairs
  int splits[2], slices[2];      // dx, dw
};
constexpr int kPairs[][2] = {{0, 0}, {1, 1}, {2, 1}};   // tiles of dx and of dw (index below)
// (fitted like kTiles, to 23 backward passes with every pair of tiles and splits: rms error 12%, choices
// 1% longer than the best; here the 64-row tiles have the LDS of the 128-row ones, two to a CU)
constexpr TileCost kPairTiles[] = {{256, 256, 1, 1.31, 1.21, 4.8}, {128, 128, 2, 0.638, 0.343, 0.82}, {64, 128, 2, 0.512, 0.405, 0.04}};

// dx [M0][N] over K0 and dw [M1][N] over K1; a product with no rows is left out.  Their tiles share
// the CUs: the time is the work of all of them over 256 CUs, at least the longest tile's own,
// and half a tile more for the uneven end.
PairPlan plan_pair(const int64_t (&M)[2], int64_t N, const int64_t (&K)[2]) {
  constexpr int kTry[] = {1, 2, 4, 8, 16};
  PairPlan best{1, {1, 1}, {1, 1}};
  double best_us = 1e30;
  for (int t = 0; t < 3; ++t) {
    for (int a : kTry) {
      for (int b : kTry) {
        PairPlan p{t, {a, b}, {1, 1}};
        double work = 0, longest = 0, shortest = 1e30, joined = 0;
        bool ok = true;
        for (int j = 0; j < 2; ++j) {
          const int want = j ? b : a;
          if (M[j] == 0 || K[j] == 0) {
            p.splits[j] = 1;
            ok = ok && want == 1;
            continue;
          }
          const TileCost& c = kPairTiles[kPairs[t][j]];
          const int64_t KT = (K[j] + KS - 1) / KS;
          const double whole = (double)((M[j] + c.rows - 1) / c.rows) * ((N + c.cols - 1) / c.cols);
          if (want > 1 && (KT / want < 3 || whole >= 512)) {   // (too short, or no need)
            ok = false;
            break;
          }
          const int64_t per = (KT + want - 1) / want;
          p.splits[j] = (int)((KT + per - 1) / per);
          p.slices[j] = (int)per;
          const double tiles = whole * p.splits[j];
          work += tiles * (per * c.shared + c.fixed);
          const double own = per * c.alone + c.fixed;
          longest = fmax(longest, own);
          shortest = fmin(shortest, own);
          if (p.splits[j] > 1) joined += (double)M[j] * N * 4 * (p.splits[j] + 1);
        }
        if (!ok) continue;
        double us = fmax(work / 256 + 0.47 * shortest, longest);
        if (joined > 0) us += 3.7 + joined / 3.3e6;
        if (us < best_us) best_us = us, best = p;
      }
    }
  }
  return best;
}
// bytes of the partial sums of product j
size_t pair_part(const PairPlan& p, int j, int64_t M, int64_t N) {
  return p.splits[j] > 1 ? ((size_t)p.splits[j] * M * N * 4 + 255) & ~size_t(255) : 0;
}

}  // namespace

size_t dense_gemm_workspace(int64_t M, int64_t N, int64_t K, int gated, bool f32, int vec) {
  if (f32 || M == 0 || dense_rows_take(M, K)) return 0;
  const Plan p = plan(M, N, K, gated);
  return p.splits > 1 || !vec ? (size_t)p.splits * M * part_pitch(N, gated) * 4 : 0;
}

hipError_t launch_dense_gemm(const DenseGemm& g, void* ws, bool f32, hipStream_t s) {
  if (f32) return launch_dense_gemm_f32(g, s);
  if (dense_rows_take(g.M, g.K)) return launch_dense_rows(g, s);
  const Plan p = plan(g.M, g.e.N, g.K, g.gated);
  Job job{};
  job.g = g;
  job.splits = p.splits;
  job.slices = p.slices;
  job.crows = g.gated ? 2 * g.e.N : g.e.N;
  job.mt = (int)((g.M + p.tile - 1) / p.tile);
  const bool join = p.splits > 1 || !g.e.vec;      // the tiles store partial sums
  const bool fused_gate = g.gated && !join;
  const int tn = (p.tile == 256 ? 256 : 128) / (fused_gate ? 2 : 1);
  job.nt = ((fused_gate ? g.e.N : job.crows) + tn - 1) / tn;
  if (!join) return g.gated ? launch_tiles<kGated>(job, p.tile, s) : launch_tiles<kLinear>(job, p.tile, s);
  job.part = static_cast<float*>(ws);
  job.ldpart = part_pitch(g.e.N, g.gated);
  hipError_t err = launch_tiles<kPartial>(job, p.tile, s);
  if (err != hipSuccess) return err;
  const int64_t pieces = g.M * ((g.e.N + 7) / 8);
  const dim3 grid((unsigned)((pieces + 255) / 256));
  if (g.gated) hipLaunchKernelGGL(dense_join_kernel<true>, grid, dim3(256), 0, s, job);
  else hipLaunchKernelGGL(dense_join_kernel<false>, grid, dim3(256), 0, s, job);
  return hipGetLastError();
}

size_t dense_gradients_workspace(int64_t T, int64_t N, int64_t cols, bool f32) {
  if (f32 || T == 0) return 0;
  size_t most = 0;
  for (int which = 1; which < 4; ++which) {        // dx, dw or both may be asked for
    const int64_t M[2] = {which & 1 ? T : 0, which & 2 ? cols : 0}, K[2] = {cols, T};
    const PairPlan p = plan_pair(M, N, K);
    const size_t need = pair_part(p, 0, M[0], N) + pair_part(p, 1, M[1], N);
    most = need > most ? need : most;
  }
  return most;
}

hipError_t launch_dense_gradients(const DenseGemm* dx, const DenseGemm* dw, void* ws, bool f32, hipStream_t s) {
  if (f32) {
    hipError_t err = dx ? launch_dense_gemm_f32(*dx, s) : hipSuccess;
    return err == hipSuccess && dw ? launch_dense_gemm_f32(*dw, s) : err;
  }
  const DenseGemm* g[2] = {dx, dw};
  const int64_t M[2] = {dx ? dx->M : 0, dw ? dw->M : 0}, K[2] = {dx ? dx->K : 0, dw ? dw->K : 0};
  const int64_t N = dx ? dx->e.N : dw->e.N;
  const PairPlan p = plan_pair(M, N, K);
  Job job[2] = {};
  int blocks[2] = {}, join_blocks[2] = {};
  size_t at = 0;
  for (int j = 0; j < 2; ++j) {
    if (!g[j]) continue;
    const TileCost& c = kPairTiles[kPairs[p.tiles][j]];
    Job& q = job[j];
    q.g = *g[j];
    q.splits = p.splits[j];
    q.slices = p.slices[j];
    q.crows = (int)N;
    q.mt = (int)((M[j] + c.rows - 1) / c.rows);
    q.nt = (int)((N + c.cols - 1) / c.cols);
    blocks[j] = (q.mt * q.nt + 7) / 8 * 8 * q.splits;
    if (q.splits > 1) {
      q.part = reinterpret_cast<float*>(static_cast<char*>(ws) + at);
      q.ldpart = N;
      at += pair_part(p, j, M[j], N);
      join_blocks[j] = (int)((M[j] * (N / 8) + 255) / 256);
    }
  }
  const int dw_first = !dx || (dw && p.slices[1] > p.slices[0]);
  const dim3 grid((unsigned)(blocks[0] + blocks[1]));
  const int n_first = blocks[dw_first];
  if (p.tiles == 0) hipLaunchKernelGGL((dense_pair_kernel<256, 256>), grid, dim3(512), 0, s, job[0], job[1], n_first, dw_first);
  else if (p.tiles == 1) hipLaunchKernelGGL((dense_pair_kernel<128, 128>), grid, dim3(256), 0, s, job[0], job[1], n_first, dw_first);
  else hipLaunchKernelGGL((dense_pair_kernel<64, 128>), grid, dim3(256), 0, s, job[0], job[1], n_first, dw_first);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || !(join_blocks[0] + join_blocks[1])) return err;
  hipLaunchKernelGGL(dense_join_pair_kernel, dim3((unsigned)(join_blocks[0] + join_blocks[1])), dim3(256), 0, s, job[0],
                     job[1], join_blocks[0]);
  return hipGetLastError();
}

}  // namespace moe
