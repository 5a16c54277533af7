// Tiles of the dense operators' matrix products on MFMA (gfx950).
//
// out[m][n] = epilogue(sum_k r[m][k] c[n][k]) (DenseGemm), float32 sums.  Three forms occur:
// forward (both operands stored along k), dx (c stored along n) and dw (both stored along
// their rows).  One pair of operand readers serves all of them, for bf16 and float32:
//
//   along k    : a tile row is 128 bytes of LDS per slice (64 k of bf16, 32 of float32), its eight 16-byte
//                chunks XOR-permuted by the row, so the 16 rows of a fragment read hit distinct banks; a
//                fragment is one 16-byte read per lane.  (float32: the four elements of a lane's chunk go to
//                four MFMAs, the lanes' four chunks being the MFMA's four k.)
//   along rows : a k row is 128 rows of the tile, 256 bytes of LDS in bf16, its eight 32-byte units
//                XOR-permuted by k; a fragment is two transposing 8-byte reads per lane
//                (ds_read_tr16_b64: each group of 16 lanes reads four k rows of 16 elements and
//                every lane gets one column), so neither form needs a transposed copy in HBM.  In float32 the
//                k row is 512 bytes, its 16-byte chunks XOR-permuted by k / 4, and a fragment four 4-byte reads.
//
// Both arrive by global->LDS DMA; the permutation is applied to the global addresses.  The
// last slice of a contraction that ends inside it takes its missing chunks from a zero
// chunk in memory, so both operands are zero there.  Rows past the matrix repeat its last one
// and are not stored.
//
// c sits on the MFMA's row side with its rows permuted (fragment j, row q: column 8 (q / 4) +
// 4 j + q % 4), so two fragments of a lane are eight consecutive columns of one output row:
// results leave the registers in pieces of eight without a pass through LDS.
#pragma once

#include <math.h>

#include "dense_device.h"
#include "dense_plan.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int REGION = 128 * 128;                     // bytes of 128 operand rows in a slice (16 KB)

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

// kPartial: float32 sums to job.part; kGrad: those, or with one split the plain result in the operands' type;
// kLinearWide: kLinear with wide_act (kernels of their own: as a branch in kLinear's, the longer code of both took 3% of
// 8192 x 2048 x 7168 without an activation)
enum { kLinear = 0, kGated = 1, kPartial = 2, kGrad = 3, kLinearWide = 4 };

// ---------------------------------------------------------------------------- DMA
// float32 stored along its rows: the XOR of a k row's 16-byte chunks, by g = (k / 4) % 4.  A fragment
// read takes k rows of four different g; its 16 rows are four neighbouring chunks of the first
// operand, and of the second (permuted columns) every other chunk of eight.
template <bool CSIDE>
__device__ __forceinline__ int chunk_xor_f32(int g) { return CSIDE ? ((g & 1) << 3) | (g >> 1) : g << 2; }

// Where instruction `ins` (1 KB) of a 128-row region takes lane `lane`'s 16 bytes from.
struct Chunk {
  int row;    // tile row within the region (along k) or first row of the chunk (along rows)
  int k;      // first k of the chunk (along k) or the k row (along rows)
};
template <typename T, bool KM, bool CSIDE>
__device__ __forceinline__ Chunk chunk_of(int ins, int lane) {
  constexpr int E = 16 / sizeof(T);     // elements of a chunk
  Chunk c;
  if constexpr (!KM) {
    c.row = ins * 8 + (lane >> 3);
    const int swz = CSIDE ? (((c.row >> 1) & 1) | (((c.row >> 3) & 3) << 1)) : ((c.row >> 1) & 7);
    c.k = ((lane & 7) ^ swz) * E;
  } else if constexpr (sizeof(T) == 2) {
    c.k = ins * 4 + (lane >> 4);
    const int f = CSIDE ? 2 * (c.k & 3) : ((c.k & 3) | (((c.k >> 3) & 1) << 2));
    const int pos = lane & 15;
    c.row = (((pos >> 1) ^ f) * 2 + (pos & 1)) * E;
  } else {
    c.k = ins * 2 + (lane >> 5);
    c.row = ((lane & 31) ^ chunk_xor_f32<CSIDE>((c.k >> 2) & 3)) * E;
  }
  return c;
}

// ---------------------------------------------------------------------------- fragments
template <typename T>
struct FragOf {
  typedef bf16x8 type;      // 16 rows x 32 k
};
template <>
struct FragOf<float> {
  typedef f32x4 type;       // 16 rows x 16 k: element j of lane group g is k 4 g + j
};
template <typename T>
using Frag = typename FragOf<T>::type;

__device__ __forceinline__ f32x4 multiply_add(bf16x8 c, bf16x8 r, f32x4 acc) { return mfma_16x16x32_bf16(c, r, acc); }
__device__ __forceinline__ f32x4 multiply_add(f32x4 c, f32x4 r, f32x4 acc) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(c[j], r[j], acc, 0, 0, 0);
  return acc;
}

// 16 rows of a region from row r0 (a multiple of 16), half s of the slice's k
template <typename T, bool KM>
struct RowFrag {
  uint32_t off[2];
  int f;
  __device__ __forceinline__ RowFrag(int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (!KM) {
#pragma unroll
      for (int s = 0; s < 2; ++s) off[s] = (uint32_t)(i * 128 + (((4 * s + g) ^ (i >> 1)) << 4));
    } else if constexpr (sizeof(T) == 2) {
      off[0] = (uint32_t)((8 * g + (i >> 2)) * 256 + (i & 3) * 8);
      f = (i >> 2) | ((g & 1) << 2);
    } else {
      off[0] = (uint32_t)(4 * g * 512 + (i & 3) * 4);
      f = (i >> 2) ^ chunk_xor_f32<false>(g);     // (r0 / 4 has none of i / 4's bits)
    }
  }
  __device__ __forceinline__ Frag<T> load(const char* region, int r0, int s) const {
    if constexpr (!KM) {
      return *reinterpret_cast<const Frag<T>*>(region + r0 * 128 + off[s]);
    } else if constexpr (sizeof(T) == 2) {
      const char* p = region + off[0] + (((r0 >> 4) ^ f) << 5) + s * 32 * 256;
      return tr_pair(p, p + 4 * 256);
    } else {
      const char* p = region + off[0] + (((r0 >> 2) ^ f) << 4) + s * 16 * 512;
      f32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const float*>(p + j * 512);
      return v;
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
template <typename T, bool KM>
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
    } else if constexpr (sizeof(T) == 2) {
      off[0] = (uint32_t)((8 * g + (i >> 2)) * 256 + (i & 1) * 16);
      f = 2 * ((i >> 2) & 3);
      half = (i & 3) >> 1;
    } else {
      off[0] = (uint32_t)(4 * g * 512 + (i & 3) * 4);
      f = chunk_xor_f32<true>(g);
      half = 2 * (i >> 2);
    }
  }
  __device__ __forceinline__ Frag<T> load(const char* region, int c0, int j, int s) const {
    if constexpr (!KM) {
      return *reinterpret_cast<const Frag<T>*>(region + (c0 + 4 * j) * 128 + off[s]);
    } else if constexpr (sizeof(T) == 2) {
      const char* p = region + off[0] + ((((c0 >> 4) + half) ^ f) << 5) + 8 * j + s * 32 * 256;
      return RowFrag<T, true>::tr_pair(p, p + 4 * 256);
    } else {
      const char* p = region + off[0] + ((((c0 >> 2) + half + j) ^ f) << 4) + s * 16 * 512;
      f32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const float*>(p + q * 512);
      return v;
    }
  }
};

// ---------------------------------------------------------------------------- operand streams
struct Job {
  DenseGemm g;
  int mt, nt;          // tiles
  int whole;           // 256 x 256 tiles, forward: tiles from this one on (a multiple of 256) are run as halves
  int splits;          // parts of the contraction
  int slices;          // slices of one split
  int crows;           // rows of c (gated: 2 I)
  float* part;         // [splits][M][ldpart] partial sums (splits > 1)
  int64_t ldpart;
  int second_parts;    // the join: odd partial sums come from dz's second part
};

// This lane's DMA sources for NI instructions (first, first + 1, ...) of one region whose
// rows are tile rows base_row .. base_row + 127
template <typename T, bool KM, bool CSIDE, int NI>
struct Stream {
  static constexpr int B = sizeof(T);
  uint32_t off[NI];
  // row_of(tile row) gives the row's distance from the operand's tile origin, clamped
  template <typename F>
  __device__ __forceinline__ void init(int first, int lane, int64_t ld, F&& row_of) {
#pragma unroll
    for (int q = 0; q < NI; ++q) {
      const Chunk c = chunk_of<T, KM, CSIDE>(first + q, lane);
      off[q] = KM ? (uint32_t)((c.k * ld + row_of(c.row)) * B) : (uint32_t)((row_of(c.row) * ld + c.k) * B);
    }
  }
  // full slice: base = operand tile origin advanced to the slice
  __device__ __forceinline__ void issue(const char* base, uint32_t lds, int q) const { dma_lds_x4(base, off[q], lds); }
  // last slice with `left` k in it
  __device__ __forceinline__ void issue_tail(const char* base, uint32_t lds, int q, int first, int lane, int left) const {
    const Chunk c = chunk_of<T, KM, CSIDE>(first + q, lane);
    const char* p = c.k < left ? base + off[q] : reinterpret_cast<const char*>(zero_chunk);
    dma_lds_x4_at(p, lds);
  }
};

// Tile t of a product: groups of 8 tile rows, the row fastest
__device__ __forceinline__ void tile_at(const Job& job, int t, int& mt, int& nt) {
  const int grp = t / (8 * job.nt);
  const int rows = min(8, job.mt - grp * 8);
  const int l = t - grp * 8 * job.nt;
  mt = grp * 8 + l % rows;
  nt = l / rows;
}
// Tile (mt, nt) of workgroup b.  Consecutive workgroups go to the eight XCDs in turn; each XCD
// takes a contiguous run of tiles, so the 32 tiles that run together on an XCD are 8 x 4 and
// share their operands in its L2.
__device__ __forceinline__ bool tile_of(const Job& job, int b, int& mt, int& nt) {
  const int total = job.mt * job.nt;
  const int per = (total + 7) >> 3;
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= total) return false;
  tile_at(job, t, mt, nt);
  return true;
}

// Stores FM pieces of eight columns from n on: piece i is row m + 16 i, its sums acc[i] (and, gated, up[i])
template <typename T, int EPI, int FM>
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
      Piece<T>::store(e.out, (m + 16 * i) * e.ldo + n, z);
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
    const EpiBias<T, EPI == kGated> bias(e, n);
    EpiRes res[FM];
#pragma unroll
    for (int i = 0; i < FM; ++i) res[i] = epi_res<T>(e, m + 16 * i, job.g.M, n);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if (m + 16 * i >= job.g.M) continue;
      float z[8], u[8];
#pragma unroll
      for (int v = 0; v < 8; ++v) z[v] = acc[i][v >> 2][v & 3], u[v] = up[i][v >> 2][v & 3];
      epi_store_vec<T, EPI == kGated, EPI == kLinearWide>(e, m + 16 * i, n, z, u, bias, res[i]);
    }
  }
}

// Byte address of tile origin (row0, k0) of an operand, and the bytes from one slice to the next
template <typename T, bool KM>
__device__ __forceinline__ const char* origin(const void* p, int64_t ld, int64_t row0, int64_t k0) {
  return static_cast<const char*>(p) + (KM ? k0 * ld + row0 : row0 * ld + k0) * (int64_t)sizeof(T);
}
template <typename T, bool KM>
__device__ __forceinline__ int64_t slice_bytes(int64_t ld) { return KM ? ks<T>() * ld * (int64_t)sizeof(T) : 128; }
// The last row that may start a read (along rows: a whole chunk)
template <typename T, bool KM>
__device__ __forceinline__ int64_t last_row(int64_t rows) {
  constexpr int E = 16 / sizeof(T);
  return KM ? (rows - 1) / E * E : rows - 1;
}

// ---------------------------------------------------------------------------- RR x 128 tiles
// Four waves (2 x 2), two slices in LDS, one barrier per slice; two (RR = 128) or three (RR =
// 64) workgroups share a CU, so one's waits are covered by the others' MFMAs.  A wave's
// columns are 32 of each half of the tile (gated: 32 gate and the matching 32 up columns).  RR = 32: float32.
template <int RR>
constexpr int lds_128() { return 2 * (RR * 128 + REGION); }
template <typename T, int RR, bool RK, bool CK, int EPI>
__device__ __forceinline__ void tile_128(const Job& job, int block, int split, char* lds) {
  constexpr int FM = RR / 32;                              // 16-row fragments per wave
  constexpr int KS = ks<T>();
  constexpr int RBYTES = RR * 128, STAGE = RBYTES + REGION;
  constexpr int NR = RBYTES / 4096, NC = REGION / 4096;    // DMA instructions per wave and slice
  static_assert(NC == 4, "a wave fills 32 rows of c's region");
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
  const char* rbase = origin<T, RK>(g.r, g.ldr, m0, k0);
  const char* cbase = origin<T, CK>(g.c, g.ldc, n0, k0);
  // gated: rows 64 .. 127 of c's region, the second two waves' instructions, are the up projection's,
  // N rows on (more than 32-bit offsets reach)
  if constexpr (EPI == kGated) cbase += (int64_t)(wave >> 1) * g.e.N * g.ldc * (int64_t)sizeof(T);
  const int64_t rstep = slice_bytes<T, RK>(g.ldr), cstep = slice_bytes<T, CK>(g.ldc);
  Stream<T, RK, false, NR> sr;
  Stream<T, CK, true, NC> sc;
  sr.init(wave * NR, lane, g.ldr, [&](int row) -> int64_t { return min((int64_t)row, last_row<T, RK>(g.M - m0)); });
  sc.init(wave * NC, lane, g.ldc, [&](int row) -> int64_t {
    if constexpr (EPI == kGated) return min(row & 63, g.e.N - 1 - n0);
    return min((int64_t)row, last_row<T, CK>(job.crows - n0));
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
  const RowFrag<T, RK> fr(lane);
  const ColFrag<T, CK> fc(lane);
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
    // the whole slice's fragments before its products: both halves' LDS latency is paid once (4096 x 2048
    // x 2048: 35.9 -> 34.2 us; the next slice's DMA behind the first products: 36.7)
    Frag<T> r[2][FM], c[2][2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) c[s][b][j] = fc.load(C, b * 64 + wn * 32, j, s);
#pragma unroll
      for (int i = 0; i < FM; ++i) r[s][i] = fr.load(R, wm * (RR / 2) + i * 16, s);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[b][i][j] = multiply_add(c[s][b][j], r[s][i], acc[b][i][j]);
    __builtin_amdgcn_sched_barrier(0);
  }
  const int col = n0 + wn * 32 + 8 * (lane >> 4);
  const int64_t m = m0 + wm * (RR / 2) + (lane & 15);
  if constexpr (EPI == kGated) {
    store_rows<T, EPI>(job, split, m, col, acc[0], acc[1]);
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) store_rows<T, EPI>(job, split, m, col + b * 64, acc[b], acc[b]);
  }
}

template <typename T, int RR, bool RK, bool CK, int EPI>
__global__ __launch_bounds__(256, 2) void dense_128_kernel(Job job) {
  __shared__ __attribute__((aligned(1024))) char lds[lds_128<RR>()];
  tile_128<T, RR, RK, CK, EPI>(job, blockIdx.x, blockIdx.y, lds);
}

// ---------------------------------------------------------------------------- sum of the splits
// Adds the splits' partial sums in their order and applies the epilogue; one thread per eight columns.
template <typename T, bool GATED>
__device__ __forceinline__ void join(const Job& job, int64_t i) {
  const int n8 = (job.g.e.N + 7) / 8;
  if (i >= job.g.M * n8) return;
  const int64_t m = i / n8;
  const int n = (int)(i - m * n8) * 8;
  const EpiBias<T, GATED> bias(job.g.e, n);
  const EpiRes res = epi_res<T>(job.g.e, m, job.g.M, n);
  float z[8] = {}, u[8] = {};
  const bool pairs = !GATED && job.second_parts;
  for (int s = 0; pairs && s < job.splits; s += 2) {   // (where the first part gave no finite sum, that is the result)
    float v[8], rest[8];
    const int64_t at = ((int64_t)s * job.g.M + m) * job.ldpart + n;
    Piece<float>::load(job.part, at, v);
    Piece<float>::load(job.part, at + job.g.M * job.ldpart, rest);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] += v[j];
      z[j] += fabsf(z[j]) < INFINITY ? rest[j] : 0.f;
    }
  }
  for (int s = 0; !pairs && s < job.splits; ++s) {
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
  epi_store<T, GATED>(job.g.e, m, n, z, u, bias, res);
}

template <typename T, bool GATED>
__global__ __launch_bounds__(256) void dense_join_kernel(Job job) {
  join<T, GATED>(job, (int64_t)blockIdx.x * 256 + threadIdx.x);
}
template <typename T>
__global__ __launch_bounds__(256) void dense_join_pair_kernel(Job a, Job b, int n_first) {
  if ((int)blockIdx.x < n_first) join<T, false>(a, (int64_t)blockIdx.x * 256 + threadIdx.x);
  else join<T, false>(b, (int64_t)(blockIdx.x - n_first) * 256 + threadIdx.x);
}

// ---------------------------------------------------------------------------- launches
// Launches a forward product: tiles(job, epilogue) launches the tile kernel
template <typename T, typename F>
hipError_t run_forward(const DenseGemm& g, const Plan& p, int tile_cols, void* ws, hipStream_t s, F&& tiles) {
  Job job{};
  job.g = g;
  job.splits = p.splits;
  job.slices = p.slices;
  job.crows = g.gated ? 2 * g.e.N : g.e.N;
  job.mt = (int)((g.M + p.tile - 1) / p.tile);
  const bool parts = p.splits > 1 || !g.e.vec;      // the tiles store partial sums
  const bool fused_gate = g.gated && !parts;
  const int tn = tile_cols / (fused_gate ? 2 : 1);
  job.nt = ((fused_gate ? g.e.N : job.crows) + tn - 1) / tn;
  const int64_t all = (int64_t)job.mt * job.nt;
  job.whole = (int)(parts ? all : whole_tiles(p.tile, all));
  if (parts) {
    job.part = static_cast<float*>(ws);
    job.ldpart = part_pitch(g.e.N, g.gated);
  }
  const bool wide = sizeof(T) == 2 && wide_act(g.e);
  hipError_t err = tiles(job, parts ? kPartial : (g.gated ? kGated : (wide ? kLinearWide : kLinear)));
  if (err != hipSuccess || !parts) return err;
  const int64_t pieces = g.M * ((g.e.N + 7) / 8);
  const dim3 grid((unsigned)((pieces + 255) / 256));
  if (g.gated) hipLaunchKernelGGL((dense_join_kernel<T, true>), grid, dim3(256), 0, s, job);
  else hipLaunchKernelGGL((dense_join_kernel<T, false>), grid, dim3(256), 0, s, job);
  return hipGetLastError();
}
inline dim3 tile_grid(const Job& job) {
  const int halved = job.mt * job.nt - job.whole;
  return dim3((unsigned)((job.whole + 7) / 8 * 8 + (halved + 7) / 8 * 16), (unsigned)job.splits);
}

// Launches the gradients: tiles(pair, grid, dx, dw, n_first, dw_first) launches the pair kernel
template <typename T, int NP, int NT, typename F>
hipError_t run_gradients(const int (&pairs)[NP][2], const TileCost (&costs)[NT], JoinCost joint, const DenseGemm* dx,
                         const DenseGemm* dw, bool two_parts, void* ws, hipStream_t s, F&& tiles) {
  const DenseGemm* g[2] = {dx, dw};
  const int64_t M[2] = {dx ? dx->M : 0, dw ? dw->M : 0}, K[2] = {dx ? dx->K : 0, dw ? dw->K : 0};
  const int64_t N = dx ? dx->e.N : dw->e.N;
  const PairPlan p = plan_pair<T>(pairs, costs, joint, M, N, K);
  Job job[2] = {}, sum[2] = {};
  int blocks[2] = {}, join_blocks[2] = {};
  size_t at = 0;
  for (int j = 0; j < 2; ++j) {
    if (!g[j]) continue;
    const TileCost& c = costs[pairs[p.tiles][j]];
    Job& q = job[j];
    q.g = *g[j];
    q.splits = p.splits[j];
    q.slices = p.slices[j];
    q.crows = (int)N;
    q.mt = (int)((M[j] + c.rows - 1) / c.rows);
    q.nt = (int)((N + c.cols - 1) / c.cols);
    blocks[j] = (q.mt * q.nt + 7) / 8 * 8 * q.splits;
    const bool halve = two_parts && j == 0;
    if (q.splits > 1 || halve) {
      q.part = reinterpret_cast<float*>(static_cast<char*>(ws) + at);
      q.ldpart = N;
      at += pair_part(p, j, M[j], N, two_parts);
      sum[j] = q;
      if (halve) sum[j].g.M /= 2, sum[j].splits *= 2, sum[j].second_parts = 1;      // (a split's second T rows follow its first)
      join_blocks[j] = (int)((sum[j].g.M * (N / 8) + 255) / 256);
    }
  }
  const int dw_first = !dx || (dw && p.slices[1] > p.slices[0]);
  hipError_t err = tiles(p.tiles, dim3((unsigned)(blocks[0] + blocks[1])), job[0], job[1], blocks[dw_first], dw_first);
  if (err != hipSuccess || !(join_blocks[0] + join_blocks[1])) return err;
  hipLaunchKernelGGL(dense_join_pair_kernel<T>, dim3((unsigned)(join_blocks[0] + join_blocks[1])), dim3(256), 0, s, sum[0],
                     sum[1], join_blocks[0]);
  return hipGetLastError();
}

}  // namespace
}  // namespace moe
