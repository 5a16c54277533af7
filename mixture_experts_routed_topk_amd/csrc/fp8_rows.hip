// e4m3 products with block scales on few rows (decode steps), forward (gfx950).
//
// One pass over the weights: a workgroup takes 16 weight rows (gated: 8 gate rows and the matching 8 up rows), its waves
// every NW-th slice of 128 k.  A wave brings a slice's codes into LDS of its own by DMA, eight whole 128-byte lines an
// instruction, several slices ahead and without a barrier.  (Straight into the MFMA's registers a lane would read 16 bytes
// of a row and its neighbours other rows: those loads kept a CU's address unit busy for 120 cycles a slice.)  A slice's result
// is folded in times the row's and the block's scale; the waves' float32 sums meet in LDS and are added in wave order.
//
// Rows of several experts: a workgroup takes one expert with rows, found from the offsets, and its rows by eights.
//
// Bound by the launch (3.4 us of an empty shape), then by the weights' bytes.  Calls back to back, weights in the caches: 16 rows, 1408 -> 2048 4.0 us;
// one row, 2048 -> 2 x 5632 4.9 us (7.0 from HBM: 3.3 TB/s), 11008 -> 2 x 4096 17.6 us (5.1 TB/s); 64 rows, 7168 -> 2048 12.1 us.
#include "dense_tile.h"
#include "fp8_tile.h"

namespace moe {
namespace {

constexpr int kLong = 4096;           // K from which on eight waves share a contraction (of up to 32 rows)
// Rows times slices
constexpr int kMaxScales = 4096;
constexpr int max_scales(int RD, int NW) { return RD == 8 || NW == 8 ? kMaxScales : RD * 8 * kLong / 128; }

// Expert number `which` of those with rows, as the tables of larger products have them (offsets taken into [0, T] and made
// non-decreasing): its number (-1: fewer experts have rows) and its rows.  Every wave finds it by itself.
struct Run {
  int e, start, end;
};
__device__ __forceinline__ Run find_run(const int32_t* __restrict__ offsets, int E, int T, int which, int lane) {
  int before = min(max(offsets[0], 0), T);         // the end of the runs before this lane's 64
  for (int base = 0; base < E; base += 64) {
    int end = max(before, base + lane < E ? min(offsets[base + lane + 1], T) : 0);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(end, d, 64);
      if (lane >= d) end = max(end, o);
    }
    const int up = __shfl_up(end, 1, 64), start = lane ? up : before;
    uint64_t live = __ballot(end > start);
    const int n = __popcll(live);
    if (which < n) {
      for (int i = 0; i < which; ++i) live &= live - 1;
      const int at = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)live) - 1);
      return {base + at, __builtin_amdgcn_readlane(start, at), __builtin_amdgcn_readlane(end, at)};
    }
    which -= n;
    before = __builtin_amdgcn_readlane(end, 63);
  }
  return {-1, 0, 0};
}

// RD: groups of eight rows of r, 1, 2, 4 or 8 (RUNS: of a run at a time)
template <int RD, bool GATED, int NW, bool UE8, bool RUNS>
__global__ __launch_bounds__(NW * 64) void fp8_rows_kernel(Fp8Gemm p) {
  constexpr int MT = (RD + 1) / 2;                 // fragments of 16 rows
  // Slices of a wave in flight: what lets the 160 KB of a CU hold three workgroups of four waves and up to 32 rows (2 x 5632 columns are
  // 704 workgroups, which 512 places would take in two rounds: 16 rows of 2048 7.0 us, 5.4 so), or one of the others
  constexpr int U = MT == 4 ? 3 : MT == 2 ? 2 : RD == 2 && NW == 4 ? 3 : 4;
  constexpr int SLICE = (2 + RD) * 1024;
  constexpr int DMAS = 2 + RD;
  constexpr int COLS = GATED ? 8 : 16;
  __shared__ __attribute__((aligned(1024))) char ring[NW * U * SLICE];
  __shared__ float sr[max_scales(RD, NW)], sb[2][RD == 8 || NW == 8 ? kMaxSlices : kLong / 128];
  static_assert(U * SLICE >= MT * 1024, "the sums take the ring's place");
  f32x4 (*red)[NW][64] = reinterpret_cast<f32x4 (*)[NW][64]>(ring);
  const DenseGemm& g = p.g;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int grp = lane >> 4, i16 = lane & 15;
  const int n0 = blockIdx.x * COLS, N = g.e.N;
  const int KT = (int)(g.K / 128);
  const int mine = (KT - wave + NW - 1) / NW;      // slices wave, wave + NW, ..
  Run run{0, 0, (int)g.M};
  if constexpr (RUNS) {
    run = find_run(p.offsets, p.E, (int)g.M, blockIdx.y, lane);
    if (run.e < 0) return;
  }
  const char* const weights = static_cast<const char*>(g.c) + run.e * p.c_expert;
  const int64_t scales = run.e * p.cs_expert;
  for (int row0 = run.start; row0 < run.end; row0 += RD * 8) {
    const int rows = RUNS ? min(RD * 8, run.end - row0) : (int)g.M;
    if (RUNS && row0 > run.start) __syncthreads();   // (the sums of the rows before may still be read)
    // lane's piece of rows 0 .. 7 and 8 .. 15 of c (gated: of gate and up), and of r's; rows past the matrix repeat its last one and are not stored
    const char* src[DMAS];
#pragma unroll
    for (int d = 0; d < DMAS; ++d) {
      const int ins = d & 1;
      const int64_t row = ins * 8 + (lane >> 3);
      if (d < 2) src[d] = weights + (GATED ? n0 + (lane >> 3) + (int64_t)ins * N : n0 + row) * g.ldc;
      else src[d] = static_cast<const char*>(g.r) + (row0 + min((d - 2) / 2 * 16 + (int)row, rows - 1)) * g.ldr;
      src[d] += Chunk8<false>::k(ins, lane) + wave * 128;
    }
    char* own = ring + wave * U * SLICE;
    auto issue = [&](int u) __attribute__((always_inline)) {
      const uint32_t to = lds_addr(own) + (uint32_t)(u % U * SLICE);
#pragma unroll
      for (int d = 0; d < DMAS; ++d) dma_lds_x4_at(src[d] + (int64_t)u * NW * 128, to + d * 1024);
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < mine) issue(u);

    // all scales (x's are packed)
    for (int i = threadIdx.x; i < rows * KT; i += NW * 64) sr[i] = static_cast<const float*>(p.rs.p)[(int64_t)row0 * KT + i];
    for (int i = threadIdx.x; i < (GATED ? 2 : 1) * KT; i += NW * 64) {
      const int h = i >= KT, kt = i - h * KT;
      const int64_t at = scales + ((n0 >> 7) + h * (int64_t)(N >> 7)) * p.cs.row + kt;
      sb[h][kt] = UE8 ? ue8m0_value(static_cast<const uint8_t*>(p.cs.p)[at]) : static_cast<const float*>(p.cs.p)[at];
    }
    __syncthreads();

    const Frag8<false> frag(lane), r_frag(RD == 1 ? lane & ~8 : lane);     // (eight rows: twice)
    f32x4 acc[MT];
    const float* my_sr[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      acc[i] = f32x4{};
      my_sr[i] = sr + min(i * 16 + i16, rows - 1) * KT;
    }
    const float* my_sb = sb[GATED ? grp >> 1 : 0];   // (result columns 4 grp .. 4 grp + 3; gated: lane groups 2 and 3 hold the up rows)
    for (int u = 0; u < mine; ++u) {
      const int behind = mine - 1 - u;               // slices in flight behind this one, at most U - 1
      if (behind >= U - 1) wait_vmcnt<(U - 1) * DMAS>();
      else if (U > 3 && behind == 2) wait_vmcnt<2 * DMAS>();
      else if (U > 2 && behind == 1) wait_vmcnt<DMAS>();
      else wait_vmcnt<0>();
      const char* at = own + u % U * SLICE;
      const i32x8 c = frag.load(at, 0);
      const int kt = wave + u * NW;
      const float b = my_sb[kt];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const f32x4 z = mfma_16x16x128_e4m3(c, r_frag.load(at, (i + 1) * 16), f32x4{});
        const float s = my_sr[i][kt] * b;
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(z[q], s, acc[i][q]);
      }
      if (u + U < mine) {
        wait_lds();                                  // the place has been read
        issue(u + U);
      }
    }

    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) red[i][wave][lane] = acc[i];
    __syncthreads();
    for (int t = threadIdx.x; t < MT * 16 * COLS; t += NW * 64) {
      const int i = t / (16 * COLS), q = t / COLS % 16, c = t % COLS;
      const int m = i * 16 + q;
      if (m >= rows) continue;
      float z = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        z += red[i][w][(c >> 2) * 16 + q][c & 3];
        if (GATED) u += red[i][w][(2 + (c >> 2)) * 16 + q][c & 3];
      }
      epi_store1<uint16_t, GATED>(g.e, row0 + m, n0 + c, z, u);
    }
  }
}

template <int RD, int NW, bool UE8, bool RUNS>
void launch_rows(const Fp8Gemm& g, hipStream_t s) {
  const dim3 grid((unsigned)(g.g.gated ? g.g.e.N / 8 : g.g.e.N / 16), RUNS ? (unsigned)(g.g.M < g.E ? g.g.M : g.E) : 1);
  if (g.g.gated) hipLaunchKernelGGL((fp8_rows_kernel<RD, true, NW, UE8, RUNS>), grid, dim3(NW * 64), 0, s, g);
  else hipLaunchKernelGGL((fp8_rows_kernel<RD, false, NW, UE8, RUNS>), grid, dim3(NW * 64), 0, s, g);
}
template <int RD, bool UE8, bool RUNS = false>
void launch_waves(const Fp8Gemm& g, hipStream_t s) {
  if constexpr (RD == 8) launch_rows<RD, 4, UE8, RUNS>(g, s);
  else if (g.g.K > kLong) launch_rows<RD, 8, UE8, RUNS>(g, s);
  else launch_rows<RD, 4, UE8, RUNS>(g, s);
}
template <bool UE8>
void launch_heights(const Fp8Gemm& g, hipStream_t s) {
  if (g.E) return launch_waves<1, UE8, true>(g, s);
  // (one row in 7168 -> 2 x 2048: 5.3 us, 8 rows 5.6, 16 6.7, 32 8.2, 64 14.6)
  if (g.g.M <= 8) launch_waves<1, UE8>(g, s);
  else if (g.g.M <= 16) launch_waves<2, UE8>(g, s);
  else if (g.g.M <= 32) launch_waves<4, UE8>(g, s);
  else launch_waves<8, UE8>(g, s);
}

}  // namespace

// One matrix: what LDS holds the scales of.  us a call, rows against tiles (fp8_tile.h), 32 rows: 2048 -> 8192 6.0 / 14.1, 7168 -> 2048 6.4 / 16.6, 512 -> 512
// 3.9 / 9.0; 64 rows: 12.2 / 18.7, 11.9 / 19.9, 4.7 / 9.3; gated 2048 -> 2 x 1408 6.6 / 17.0, 2 x 8192 22.8 / 23.2, 1024 -> 2 x 7168 15.2 / 13.2 (the only one
// of 18 shapes where tiles win).
// Runs, eight rows of one at a time: 4 rows of 60 runs, 2048 -> 1408 5.2 / 23.4, gated 5.8 / 23.6; 16 rows 10.7 / 24.7, 19.4 / 27.0; 64 rows
// 28.6 / 29.3, 50.7 / 50.6, of 256 runs, 7168 -> 512 44.7 / 59.0, 103.6 / 90.1; 128 rows of 32, 7168 -> 2048 114 / 103, 221 / 187.
// Long runs pass over their matrix once for every eight rows, from the caches: 64 rows of one run, 2048 -> 1408 15.6 / 23.7 (as one matrix 6.3),
// 7168 -> 2048 24.4 / 58.3 (11.9), of two 9.2 / 22.9 and 16.0 / 56.9, of four 6.9 / 22.9 and 20.5 / 56.6; gated, 32 rows of one 9.6 / 23.1 (4.4)
// and 15.7 / 56.2 (8.1), of four 5.6 / 23.0 and 26.0 / 55.5.
bool fp8_rows_take(int64_t M, int64_t K, int E, bool gated) {
  return E ? M <= (gated ? 32 : 64) : M <= 64 && M * (K / 128) <= kMaxScales;
}

hipError_t launch_fp8_rows(const Fp8Gemm& g, hipStream_t s) {
  if (g.cs.bytes) launch_heights<true>(g, s);
  else launch_heights<false>(g, s);
  return hipGetLastError();
}

}  // namespace moe
