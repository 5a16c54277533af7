// Elementwise part of the dense operators' backward pass (gfx950).
//
// linear: dz = dy act'(pre).  gated: dz = [da up act'(gate), da act(gate)], pre = [gate, up].
// dz goes to scratch in the operands' type (the type the MFMA products take; each dz is
// rounded once, as the saved pre-activations were; TWO: what that takes is kept as a second part), with zeros in the columns between the
// last one and its pitch so that rows can be read in whole 16-byte pieces.  The bias gradient sums the
// float32 dz before that rounding: a workgroup sums its rows' columns in registers, and the
// workgroups' partial rows are added in a fixed order by column_sum_kernel.
//
// Memory-bound: one read of dy and pre, one write of dz.
#include "dense_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kDzRows = 8;       // rows of one workgroup: two per wave, both in flight at once (8192 x 2048 gated: 16 rows 7 us slower)

// Eight columns starting at n of a row whose columns end at N (zeros past it)
template <typename T>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, int N, bool vec, float v[8]) {
  if (vec && n + 8 <= N) {
    Piece<T>::load(p, at + n, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = n + i < N ? Piece<T>::get(p, at + n + i) : 0.f;
  }
}

// Two bf16 values with those that are not finite replaced by zero
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t v) {
  if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
  if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
  return v;
}

// What rounding to T takes from v; nothing where that is infinite
template <typename T>
__device__ __forceinline__ float rest(float v) {
  const float r = Piece<T>::round(v);
  return fabsf(r) < INFINITY ? v - r : 0.f;
}

// Workgroup (x, y): columns 512 y .. 512 y + 511 (eight a lane) of rows 8 x .. 8 x + 7; wave w takes rows
// w and w + 4.  The four waves' column sums meet in LDS.
template <typename T, typename D, bool GATED, bool TWO>
__global__ __launch_bounds__(kThreads) void dz_kernel(DzArgs a, int vec) {
  constexpr bool FAST = sizeof(T) == 2;
  constexpr int ROWS = kDzRows / 4;
  __shared__ float red[GATED ? 2 : 1][4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = blockIdx.y * 512 + lane * 8;
  if constexpr (TWO) {                               // workgroups behind dz's: x's rows, then their finite values
    const int dz_groups = ((GATED ? a.N : (int)a.ldz) + 511) / 512;
    if ((int)blockIdx.y >= dz_groups) {
      const int k = n - dz_groups * 512;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int64_t t = (int64_t)blockIdx.x * kDzRows + wave + 4 * r;
        if (t >= a.T || k >= a.K) continue;
        i32x4 v = Piece<uint16_t>::raw(a.x, t * a.ldx + k);
        *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(a.x2) + t * a.K + k) = v;
        // (an infinity times dz's first part is the result; times the second it could make that NaN)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (int)finite_bf16x2((uint32_t)v[i]);
        *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(a.x2) + (t + a.T) * a.K + k) = v;
      }
      return;
    }
  }
  const int width = GATED ? a.N : (int)a.ldz;        // columns written (with the pitch's zeros)
  float s0[8] = {}, s1[8] = {};
  if (n < width) {
    float d[ROWS][8], z[ROWS][8], u[ROWS][8];
    const int64_t t0 = (int64_t)blockIdx.x * kDzRows + wave;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t t = min(t0 + 4 * r, a.T - 1);    // (rows past the end repeat the last and are dropped below)
      load8<D>(a.dy, t * a.ldy, n, a.N, vec, d[r]);
      if (a.pre) load8<T>(a.pre, t * a.ldp, n, a.N, vec, z[r]);
      if (GATED) load8<T>(a.pre, t * a.ldp + a.N, n, a.N, vec, u[r]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int64_t t = t0 + 4 * r;
      if (t >= a.T) continue;
      if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ActPair p = act_pair<FAST>(a.act, z[r][i]);
          const float da = d[r][i];
          d[r][i] = times_slope(a.act, da * u[r][i], p.slope);
          u[r][i] = da * p.value;
          s1[i] += u[r][i];
        }
      } else if (a.pre) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          d[r][i] = n + i < a.N ? times_slope(a.act, d[r][i], act_pair<FAST>(a.act, z[r][i]).slope) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s0[i] += d[r][i];
      if (a.dz) {
        Piece<T>::store(a.dz, t * a.ldz + n, d[r]);
        if constexpr (GATED) Piece<T>::store(a.dz, t * a.ldz + a.N + n, u[r]);
        if constexpr (TWO) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            d[r][i] = rest<T>(d[r][i]);
            if (GATED) u[r][i] = rest<T>(u[r][i]);
          }
          Piece<T>::store(a.dz, (t + a.T) * a.ldz + n, d[r]);
          if constexpr (GATED) Piece<T>::store(a.dz, (t + a.T) * a.ldz + a.N + n, u[r]);
        }
      }
    }
  }
  if (!a.part) return;
  Piece<float>::store(red[0][wave], lane * 8, s0);
  if constexpr (GATED) Piece<float>::store(red[1][wave], lane * 8, s1);
  __syncthreads();
  const int64_t cols = GATED ? 2 * (int64_t)a.N : a.N;
  float* out = a.part + blockIdx.x * cols;
  for (int c = threadIdx.x; c < 512; c += kThreads) {
    const int col = blockIdx.y * 512 + c;
    if (col >= a.N) break;
    out[col] = ((red[0][0][c] + red[0][1][c]) + red[0][2][c]) + red[0][3][c];
    if constexpr (GATED) out[a.N + col] = ((red[1][0][c] + red[1][1][c]) + red[1][2][c]) + red[1][3][c];
  }
}

// 64 columns a workgroup; wave w adds rows w, w + 16, ... and the sixteen sums are added in order
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(kSumWaves * kWave) void column_sum_kernel(const float* __restrict__ part, int64_t rows,
                                                                       int64_t cols, void* __restrict__ out, int f32) {
  __shared__ float red[kSumWaves][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * kWave + lane;
  float s = 0.f;
  if (c < cols) {
    int64_t r = wave;
    for (; r + 7 * kSumWaves < rows; r += 8 * kSumWaves) {   // eight loads in flight
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = part[(r + i * kSumWaves) * cols + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; r < rows; r += kSumWaves) s += part[r * cols + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) s += red[w][lane];
    if (f32) Piece<float>::put(out, c, s);
    else Piece<uint16_t>::put(out, c, s);
  }
}

__global__ __launch_bounds__(kThreads) void zero_bytes_kernel(uint8_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = 0;
}

template <typename T, typename D, bool TWO>
hipError_t launch(const DzArgs& a, int vec, hipStream_t s) {
  const int64_t width = a.gated ? a.N : a.ldz;
  const dim3 grid((unsigned)dz_parts(a.T), (unsigned)((width + 511) / 512 + (TWO ? (a.K + 511) / 512 : 0)));
  if (a.gated) hipLaunchKernelGGL((dz_kernel<T, T, true, TWO>), grid, dim3(kThreads), 0, s, a, vec);
  else hipLaunchKernelGGL((dz_kernel<T, D, false, TWO>), grid, dim3(kThreads), 0, s, a, vec);
  return hipGetLastError();
}

}  // namespace

int64_t dz_parts(int64_t T) { return (T + kDzRows - 1) / kDzRows; }

hipError_t launch_dz(const DzArgs& a, bool f32, hipStream_t s) {
  auto ok = [](const void* p, int64_t ld, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * esz) % 16 == 0;
  };
  const int esz = f32 ? 4 : 2;
  const int vec = ok(a.dy, a.ldy, a.dy_f32 ? 4 : esz) && (!a.pre || ok(a.pre, a.ldp, esz));
  hipError_t err;
  if (f32) err = launch<float, float, false>(a, vec, s);
  else if (a.x2) err = a.dy_f32 ? launch<uint16_t, float, true>(a, vec, s) : launch<uint16_t, uint16_t, true>(a, vec, s);
  else err = a.dy_f32 ? launch<uint16_t, float, false>(a, vec, s) : launch<uint16_t, uint16_t, false>(a, vec, s);
  if (err != hipSuccess || !a.dbias) return err;
  return launch_column_sum(a.part, dz_parts(a.T), a.gated ? 2 * (int64_t)a.N : a.N, a.dbias, f32, s);
}

hipError_t launch_column_sum(const float* part, int64_t rows, int64_t cols, void* out, bool f32, hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((cols + kWave - 1) / kWave)), dim3(kSumWaves * kWave), 0, s, part,
                     rows, cols, out, f32 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t s) {
  const int64_t b = (bytes + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(zero_bytes_kernel, dim3((unsigned)(b < 1 ? 1 : (b > 4096 ? 4096 : b))), dim3(kThreads), 0, s,
                     static_cast<uint8_t*>(p), bytes);
  return hipGetLastError();
}

}  // namespace moe
