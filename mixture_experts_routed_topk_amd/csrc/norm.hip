// Root-mean-square norm with the residual's addition, forward and backward (gfx950).
//
// Forward, per row: h = x + residual (rounded to the rows' type, since h is what the next
// layer's residual and the backward pass read; the norm is taken of that stored h),
//   rstd = (mean_j h_j^2 + eps)^-1/2,   y_j = h_j rstd weight_j,
// and y is stored, or quantised to e4m3 with one float32 scale amax / 448 per 128 columns (the
// rule of moe_quantize_rows_fp8, applied to the float32 y), or both.  Backward, with n = h rstd and g = dy weight:
//   dx_j = rstd (g_j - n_j mean_i(g_i n_i)) + dh_j,   dweight_j = sum_t dy_j n_j.
//
// Memory-bound: every row is read once and held in registers between the statistic and the
// result, in pieces of eight elements.  A row belongs to WPR waves (1, 4 or 16), each lane
// holding NV pieces; with one wave to a row the statistic needs no LDS.  The backward kernel
// walks rows with a fixed grid, so a lane keeps the float32 sums of its columns of dweight
// in registers over all its rows; the grid's partial rows are summed in a fixed order by a
// second kernel (no atomics: the result does not depend on timing).
#include "dense_device.h"

namespace moe {
namespace {

template <int WPR>
constexpr int rows_per_block() { return WPR >= 4 ? 1 : 4 / WPR; }
template <int WPR>
constexpr int block_threads() { return WPR * rows_per_block<WPR>() * kWave; }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Sum over the WPR waves of a row; every lane gets it.  `slot` alternates between calls, so
// one barrier a call is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float (*red)[16], int slot) {
  v = wave_sum(v);
  if constexpr (WPR == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < WPR; ++w) t += red[slot][w];
  return t;
}

template <typename T, int WPR, int NV, bool QUANT>
__global__ __launch_bounds__(block_threads<WPR>()) void rms_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  constexpr int RPB = rows_per_block<WPR>(), LPR = WPR * kWave;   // rows per block, lanes per row
  const int lane = threadIdx.x % LPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
  if (row >= a.T) return;                        // (whole rows: the lanes of a row agree; WPR > 1 has one row)
  const int np = a.H / 8;
  using Raw = typename Piece<T>::Raw;
  Raw x[NV], r[NV], w[NV];
  // every load of the row before the first use (lanes past the row repeat its first piece)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * LPR + lane < np ? i * LPR + lane : 0;
    x[i] = Piece<T>::raw(a.x, row * a.ldx + p * 8);
    if (a.res) r[i] = Piece<T>::raw(a.res, row * a.ldr + p * 8);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) w[i] = Piece<T>::raw(a.weight, (i * LPR + lane < np ? i * LPR + lane : 0) * 8);
  float v[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * LPR + lane;
    if (p < np) {
      Piece<T>::widen(x[i], v[i]);
      if (a.res) {
        float d[8];
        Piece<T>::widen(r[i], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = Piece<T>::round(v[i][j] + d[j]);
        Piece<T>::store(a.h, row * a.ldh + p * 8, v[i]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += v[i][j] * v[i][j];
    }
  }
  ss = row_sum<WPR>(ss, red, 0);
  const float rstd = 1.0f / sqrtf(ss / (float)a.H + a.eps);
  if (lane == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int p = i * LPR + lane;
    if (p < np) {
      float wf[8];
      Piece<T>::widen(w[i], wf);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * wf[j];
      if (!QUANT || a.y) Piece<T>::store(a.y, row * a.ldy + p * 8, v[i]);
      if constexpr (QUANT) {   // 16 lanes hold a group of 128 columns (H % 128 == 0: whole groups)
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d, 16));
        const float s0 = amax / 448.0f, s = s0 > 0.f ? s0 : 1.0f;
        uint32_t lo = 0, hi = 0;
        // v / s from one reciprocal: the quotient's error is taken back once, which rounds as the
        // division does (eight IEEE divisions and the e4m3 rounding in integer steps take as long as
        // the row's memory traffic)
        if (s0 > 0x1p-96f && s0 < 0x1p96f) {   // (a NaN keeps its sign in its code)
          const float inv = 1.0f / s;
          float d[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float quo = v[i][j] * inv;
            d[j] = fmaf(fmaf(-quo, s, v[i][j]), inv, quo);
          }
          lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], lo, false);
          lo = __builtin_amdgcn_cvt_pk_fp8_f32(d[2], d[3], lo, true);
          hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[4], d[5], hi, false);
          hi = __builtin_amdgcn_cvt_pk_fp8_f32(d[6], d[7], hi, true);
        } else {
          // 1 / s or the correction may leave float32's range; and a scale of few bits may lie so far below
          // amax / 448 that a value passes 464 times it, where the conversion gives NaN and the rule saturates
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            lo |= f32_to_e4m3(v[i][j] / s) << (8 * j);
            hi |= f32_to_e4m3(v[i][4 + j] / s) << (8 * j);
          }
        }
        *reinterpret_cast<uint2*>(a.q + row * a.H + p * 8) = make_uint2(lo, hi);
        if ((lane & 15) == 0) a.q_scale[row * (a.H / 128) + p / 16] = s;
      }
    }
  }
}

template <typename T, int WPR, int NV>
__global__ __launch_bounds__(block_threads<WPR>()) void rms_norm_backward_kernel(NormArgs a) {
  __shared__ float red[2][16];
  constexpr int RPB = rows_per_block<WPR>(), LPR = WPR * kWave;
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int np = a.H / 8;
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  using Raw = typename Piece<T>::Raw;
  struct Row {
    Raw dy[NV], h[NV], dh[NV];
    float rstd;
  } next;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {   // (lanes past the row repeat its first piece)
    next.rstd = a.rstd_in[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * LPR + lane < np ? i * LPR + lane : 0;
      next.dy[i] = Piece<T>::raw(a.dy, row * a.ldy + p * 8);
      next.h[i] = Piece<T>::raw(a.hin, row * a.ldh + p * 8);
      if (a.res) next.dh[i] = Piece<T>::raw(a.res, row * a.ldr + p * 8);
    }
  };
  // sixteen waves leave a lane 128 registers: no room for a second row, nor for g and n beside dy and h.  Even so
  // those instances spill (43 and 83 registers of bf16 and float32 rows up to 32768, 323 and 424 beyond), which
  // costs them half their rate and more: 2048 x 16384 with dh 125 us in bf16 (2.15 TB/s) and 219 in float32, 512 x
  // 65536 255 and 365 us, against 4.1 to 4.8 TB/s up to 8192
  constexpr bool kAhead = WPR < 16;
  int slot = 0;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  if (row < a.T) fetch(row);
  for (; row < a.T; row += step) {
    const Row cur = next;
    if (kAhead && row + step < a.T) fetch(row + step);   // the next row's loads cover this row's reduction
    // g = dy w and n = h rstd of piece i; kept over the reduction, or formed again after it
    float gk[NV][8], nk[NV][8];
    auto form = [&](int i, int p, float (&dy)[8], float (&g)[8], float (&n)[8]) __attribute__((always_inline)) {
      float w[8];
      Piece<T>::widen(cur.dy[i], dy);
      Piece<T>::widen(cur.h[i], n);
      Piece<T>::load(a.weight, p * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] *= cur.rstd, g[j] = dy[j] * w[j];
    };
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * LPR + lane;
      if (p < np) {
        float dy[8];
        form(i, p, dy, gk[i], nk[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dw[i][j] += dy[j] * nk[i][j];
          dot += gk[i][j] * nk[i][j];
        }
      }
    }
    dot = row_sum<WPR>(dot, red, slot) / (float)a.H;
    slot ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * LPR + lane;
      if (p < np) {
        float d[8];
        if (!kAhead) form(i, p, d, gk[i], nk[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = cur.rstd * (gk[i][j] - nk[i][j] * dot);
        if (a.res) {
          float r[8];
          Piece<T>::widen(cur.dh[i], r);
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] += r[j];
        }
        Piece<T>::store(a.dx, row * a.ldx + p * 8, d);
      }
    }
    if (!kAhead && row + step < a.T) fetch(row + step);
  }
  if (a.part) {   // one partial row per row slot of the grid
    float* out = a.part + ((int64_t)blockIdx.x * RPB + sub) * a.H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int p = i * LPR + lane;
      if (p < np) Piece<float>::store(out, p * 8, dw[i]);
    }
  }
}

// Lanes of a row hold at most 4 pieces (2048 columns a wave) while a row fits four waves, so
// a row's registers stay few enough for several blocks per CU (backward in float32 with 4 pieces: one); longer
// rows take 16 waves, and past 32768 columns 8 pieces, where the float32 forward spills too (104 registers; 512 x
// 65536 185 us, 2.9 TB/s).
template <typename F>
hipError_t by_width(int H, F&& f) {
  const int np = H / 8;
  using std::integral_constant;
  if (np <= 64) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  if (np <= 128) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (np <= 256) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
  if (np <= 512) return f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (np <= 1024) return f(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  if (np <= 4096) return f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});   // H <= 65536
}
int rows_of_block(int H) { return H / 8 <= 256 ? rows_per_block<1>() : 1; }

int64_t backward_blocks(int64_t T, int H) {
  const int64_t need = (T + rows_of_block(H) - 1) / rows_of_block(H);
  // two blocks of four waves, or one of sixteen, per CU (float32 with 4 pieces a lane: one after the other)
  const int64_t most = H / 8 <= 1024 ? 512 : 256;
  return need < most ? need : most;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, bool f32, hipStream_t s) {
  return by_width(a.H, [&](auto wpr, auto nv) -> hipError_t {
    constexpr int W = decltype(wpr)::value, N = decltype(nv)::value;
    const dim3 grid((unsigned)((a.T + rows_per_block<W>() - 1) / rows_per_block<W>())), block(block_threads<W>());
    if (f32) hipLaunchKernelGGL((rms_norm_kernel<float, W, N, false>), grid, block, 0, s, a);
    else if (a.q) hipLaunchKernelGGL((rms_norm_kernel<uint16_t, W, N, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_norm_kernel<uint16_t, W, N, false>), grid, block, 0, s, a);
    return hipGetLastError();
  });
}

int64_t norm_backward_parts(int64_t T, int H) { return backward_blocks(T, H) * rows_of_block(H); }

hipError_t launch_rms_norm_backward(const NormArgs& a, bool f32, hipStream_t s) {
  hipError_t err = by_width(a.H, [&](auto wpr, auto nv) -> hipError_t {
    constexpr int W = decltype(wpr)::value, N = decltype(nv)::value;
    const dim3 grid((unsigned)backward_blocks(a.T, a.H)), block(block_threads<W>());
    if (f32) hipLaunchKernelGGL((rms_norm_backward_kernel<float, W, N>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((rms_norm_backward_kernel<uint16_t, W, N>), grid, block, 0, s, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || !a.dweight) return err;
  return launch_column_sum(a.part, norm_backward_parts(a.T, a.H), a.H, a.dweight, f32, s);
}

}  // namespace moe
