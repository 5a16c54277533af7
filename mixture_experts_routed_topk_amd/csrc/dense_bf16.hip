// bf16 matrix products of the dense operators (gfx950): the 256 x 256 tiles, both gradients in one
// launch, and the choice of tiles.  dense_tile.h has the operand readers and the smaller tiles.
#include "dense_tile.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------- 256 x 256 tiles
// Eight waves (two per SIMD) in a 2 x 4 grid, each 128 x 64 of the tile as four quadrants (64
// rows of row half 0 or 1 x 32 columns of column half 0 or 1).  A slice is four phases of one
// quadrant, 16 MFMAs; the fragments of a phase are read from LDS one phase ahead, so a wave's MFMAs
// never wait for its own reads, and the SIMD's other wave fills what is left:
//   phase   reads        multiplies       issues (DMA)
//   0       C1(kt)       R0 x C0          R0(kt+2)
//   1       R1(kt)       R0 x C1          C0(kt+2)     then: wait for R0, C0(kt+1); barrier
//   2       R0(kt+1)     R1 x C0          C1(kt+2)
//   3       C0(kt+1)     R1 x C1          R1(kt+2)     then: wait for C1, R1(kt+1); barrier
// Two slices live in LDS.  Each barrier publishes the regions read in the next two phases and frees
// those read in the last two, which the next two phases refill: a DMA has four to six phases
// (more than a slice's MFMA time) to land.  DMAs retire in issue order, two per region
// and wave, which gives the vmcnt of each wait.  The order inside a phase is measured (8192 x 7168 x
// 4096: 354 us; DMAs before the products 374, before the reads 378; reads spread between
// the products 364-379).  With every tile reading the same, L2-resident operands the time is the same
// within 2%: the loop is bound by what a CU does, not by its operand stream.
// NH = 1 is half a tile, 128 rows from m0: R1, its reads and products and its DMAs are left out.
constexpr int kLds256 = 2 * 4 * REGION;   // [slice parity][R0 R1 C0 C1]
template <bool RK, bool CK, int EPI, int NH>
__device__ __forceinline__ void tile_256(const Job& job, int64_t m0, int nt, int split, char* lds) {
  using T = uint16_t;
  constexpr int KS = ks<T>();
  const DenseGemm& g = job.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int n0 = nt * (EPI == kGated ? 128 : 256);
  const int64_t k0 = (int64_t)split * job.slices * KS;
  const int KT = (int)min((int64_t)job.slices, (g.K - k0 + KS - 1) / KS);
  const int left = (int)min((int64_t)KS, g.K - k0 - (int64_t)(KT - 1) * KS);   // k in the last slice

  // operand tile origins and the bytes from one slice to the next
  const char* rbase = origin<T, RK>(g.r, g.ldr, m0, k0);
  const char* cbase = origin<T, CK>(g.c, g.ldc, n0, k0);
  const int64_t rstep = slice_bytes<T, RK>(g.ldr), cstep = slice_bytes<T, CK>(g.ldc);
  // gated: the second column half is the up projection's rows, N rows on (more than 32-bit offsets reach)
  const char* const chalf[2] = {cbase, cbase + (EPI == kGated ? (int64_t)g.e.N * g.ldc * (int64_t)sizeof(T) : 0)};
  Stream<T, RK, false, 2> sr[NH];
  Stream<T, CK, true, 2> sc[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h < NH)
      sr[h].init(wave * 2, lane, g.ldr,
                 [&](int row) -> int64_t { return min((int64_t)(h * 128 + row), last_row<T, RK>(g.M - m0)); });
    sc[h].init(wave * 2, lane, g.ldc, [&](int row) -> int64_t {
      if constexpr (EPI == kGated) return min(row, g.e.N - 1 - n0);
      return min((int64_t)(h * 128 + row), last_row<T, CK>(job.crows - n0));
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
    const char* base = chalf[h] + kt * cstep;
    const uint32_t dst = lds0 + (uint32_t)(((kt & 1) * 4 + 2 + h) * REGION + wave * 2048);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (kt == KT - 1 && left < KS) sc[h].issue_tail(base, dst + q * 1024, q, wave * 2, lane, left);
      else sc[h].issue(base, dst + q * 1024, q);
    }
  };

  const RowFrag<T, RK> fr(lane);
  const ColFrag<T, CK> fc(lane);
  f32x4 acc[NH][2][4][2];
#pragma unroll
  for (int a = 0; a < NH; ++a)
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
    if (more) wait_vmcnt<4 + 2 * NH>();
    else wait_vmcnt<0>();
    wait_lds();
    barrier();
  };

  issue_r(0, 0), issue_c(0, 0), issue_c(1, 0);
  if constexpr (NH == 2) issue_r(1, 0);
  if (KT > 1) {
    issue_r(0, 1), issue_c(0, 1), issue_c(1, 1);
    if constexpr (NH == 2) issue_r(1, 1);
  }
  publish(KT > 1);
  read_r(r0, 0, 0);
  read_c(c0, 0, 0);
  wait_lds();
  barrier();       // (phase 0 refills what was just read)
  for (int kt = 0; kt < KT; ++kt) {
    const bool more = kt + 2 < KT, next = kt + 1 < KT;
    read_c(c1, 1, kt);
    multiply(acc[0][0], r0, c0);
    if (more) issue_r(0, kt + 2);

    if constexpr (NH == 2) read_r(r1, 1, kt);
    multiply(acc[0][1], r0, c1);
    if (more) issue_c(0, kt + 2);
    publish(more);

    if (next) read_r(r0, 0, kt + 1);
    if constexpr (NH == 2) multiply(acc[1][0], r1, c0);
    if (more) issue_c(1, kt + 2);

    if (next) read_c(c0, 0, kt + 1);
    if constexpr (NH == 2) {
      multiply(acc[1][1], r1, c1);
      if (more) issue_r(1, kt + 2);
    }
    publish(more);
  }

  const int row = lane & 15, col = 8 * (lane >> 4);
#pragma unroll
  for (int a = 0; a < NH; ++a) {
    const int64_t m = m0 + a * 128 + wm * 64 + row;
    if constexpr (EPI == kGated) {
      store_rows<T, EPI>(job, split, m, n0 + wn * 32 + col, acc[a][0], acc[a][1]);
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) store_rows<T, EPI>(job, split, m, n0 + b * 128 + wn * 32 + col, acc[a][b], acc[a][b]);
    }
  }
}

template <bool RK, bool CK, int EPI>
__device__ __forceinline__ void whole_256(const Job& job, int block, int split, char* lds) {
  int mt, nt;
  if (tile_of(job, block, mt, nt)) tile_256<RK, CK, EPI, 2>(job, (int64_t)mt * 256, nt, split, lds);
}

// Forward.  HALVES: the tiles from job.whole on are run as two workgroups of 128 rows each, on one XCD
// one after the other (they share c's rows); a kernel of its own, since in the common one the extra
// path costs 2% (6144 x 2048 x 7168: 160 against 168 us).
template <int EPI, bool HALVES>
__global__ __launch_bounds__(512, 1) void dense_256_kernel(Job job) {
  __shared__ __attribute__((aligned(1024))) char lds[kLds256];
  if constexpr (!HALVES) {
    whole_256<false, false, EPI>(job, blockIdx.x, blockIdx.y, lds);
  } else {
    const int total = job.mt * job.nt;
    const int b = (int)blockIdx.x - job.whole;
    int mt, nt;
    if (b < 0) {
      tile_at(job, (blockIdx.x & 7) * (job.whole >> 3) + (blockIdx.x >> 3), mt, nt);
      tile_256<false, false, EPI, 2>(job, (int64_t)mt * 256, nt, 0, lds);
    } else {
      const int per = (total - job.whole + 7) >> 3;
      const int t = job.whole + (b & 7) * per + (b >> 4);
      if (t >= total) return;
      tile_at(job, t, mt, nt);
      const int64_t m0 = (int64_t)mt * 256 + ((b >> 3) & 1) * 128;
      if (m0 < job.g.M) tile_256<false, false, EPI, 1>(job, m0, nt, 0, lds);
    }
  }
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
    if constexpr (TB == 256) whole_256<true, true, kGrad>(dw, b % n, b / n, lds);
    else tile_128<uint16_t, TB, true, true, kGrad>(dw, b % n, b / n, lds);
  } else {
    const int n = (dx.mt * dx.nt + 7) / 8 * 8;
    if constexpr (TA == 256) whole_256<false, true, kGrad>(dx, b % n, b / n, lds);
    else tile_128<uint16_t, TA, false, true, kGrad>(dx, b % n, b / n, lds);
  }
}

// ---------------------------------------------------------------------------- launches
template <int EPI>
void launch_tiles(const Job& job, int tile, hipStream_t s) {
  const dim3 grid = tile_grid(job);
  if (tile == 256) {
    if (EPI != kPartial && job.whole < job.mt * job.nt) {
      hipLaunchKernelGGL((dense_256_kernel<EPI, EPI != kPartial>), grid, dim3(512), 0, s, job);
    } else {
      hipLaunchKernelGGL((dense_256_kernel<EPI, false>), grid, dim3(512), 0, s, job);
    }
  }
  else if (tile == 128) hipLaunchKernelGGL((dense_128_kernel<uint16_t, 128, false, false, EPI>), grid, dim3(256), 0, s, job);
  else hipLaunchKernelGGL((dense_128_kernel<uint16_t, 64, false, false, EPI>), grid, dim3(256), 0, s, job);
}

}  // namespace

size_t dense_gemm_workspace(int64_t M, int64_t N, int64_t K, int gated, bool f32, int vec) {
  if (M == 0 || dense_rows_take(M, K, f32)) return 0;
  return f32 ? dense_gemm_f32_workspace(M, N, K, gated, vec) : forward_part(plan_bf16(M, N, K, gated), M, N, gated, vec);
}

hipError_t launch_dense_gemm(const DenseGemm& g, void* ws, bool f32, hipStream_t s) {
  if (dense_rows_take(g.M, g.K, f32)) return launch_dense_rows(g, f32, s);
  if (f32) return launch_dense_gemm_f32(g, ws, s);
  const Plan p = plan_bf16(g.M, g.e.N, g.K, g.gated);
  return run_forward<uint16_t>(g, p, p.tile == 256 ? 256 : 128, ws, s, [&](const Job& job, int epi) {
    if (epi == kPartial) launch_tiles<kPartial>(job, p.tile, s);
    else if (epi == kGated) launch_tiles<kGated>(job, p.tile, s);
    else if (epi == kLinearWide) launch_tiles<kLinearWide>(job, p.tile, s);
    else launch_tiles<kLinear>(job, p.tile, s);
    return hipGetLastError();
  });
}

size_t dense_gradients_workspace(int64_t rows, int64_t N, int64_t cols, bool f32, bool two_parts) {
  if (rows == 0) return 0;
  return f32 ? dense_gradients_f32_workspace(rows, N, cols)
             : gradients_part<uint16_t>(kPairsBf16, kPairTilesBf16, kPairJoinBf16, rows, N, cols, two_parts);
}

hipError_t launch_dense_gradients(const DenseGemm* dx, const DenseGemm* dw, void* ws, bool f32, bool two_parts,
                                  hipStream_t s) {
  if (f32) return launch_dense_gradients_f32(dx, dw, ws, s);
  return run_gradients<uint16_t>(kPairsBf16, kPairTilesBf16, kPairJoinBf16, dx, dw, two_parts, ws, s,
                                 [&](int pair, dim3 grid, const Job& x, const Job& w, int n_first, int dw_first) {
    if (pair == 0) hipLaunchKernelGGL((dense_pair_kernel<256, 256>), grid, dim3(512), 0, s, x, w, n_first, dw_first);
    else if (pair == 1) hipLaunchKernelGGL((dense_pair_kernel<128, 128>), grid, dim3(256), 0, s, x, w, n_first, dw_first);
    else hipLaunchKernelGGL((dense_pair_kernel<64, 128>), grid, dim3(256), 0, s, x, w, n_first, dw_first);
    return hipGetLastError();
  });
}

}  // namespace moe
