// Elementwise part of the dense operators' backward pass (gfx950).
//
// linear: dz = dy act'(pre).  gated: dz = [da up act'(gate), da act(gate)], pre = [gate, up].
// dz goes to scratch in the operands' type (the type the MFMA products take; each dz is
// rounded once, as the saved pre-activations were), with zeros in the columns between the
// last one and its pitch so that rows can be read in whole 16-byte pieces.  The bias gradient sums the
// float32 dz before that rounding: a workgroup sums its rows' columns in registers, and the
// workgroups' partial rows are added in a fixed order by column_sum_kernel.
//
// Memory-bound: one read of dy and pre, one write of dz.
#include "dense_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kDzRows = 64;      // rows of one workgroup: partial rows cost 1/64 of dz at most twice over

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

// Workgroup (x, y): columns 8 * (256 y + tid) .. + 7 of rows 64 x .. 64 x + 63
template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads) void dz_kernel(DzArgs a, int vec) {
  constexpr bool FAST = sizeof(T) == 2;
  const int n = (blockIdx.y * kThreads + threadIdx.x) * 8;
  const int width = GATED ? a.N : (int)a.ldz;        // columns written (with the pitch's zeros)
  if (n >= width) return;
  const int64_t r0 = (int64_t)blockIdx.x * kDzRows, r1 = min(a.T, r0 + kDzRows);
  float s0[8] = {}, s1[8] = {};
  for (int64_t t = r0; t < r1; ++t) {
    float d[8], z[8], u[8];
    if (a.dy_f32) load8<float>(a.dy, t * a.ldy, n, a.N, vec, d);
    else load8<T>(a.dy, t * a.ldy, n, a.N, vec, d);
    if (a.pre) load8<T>(a.pre, t * a.ldp, n, a.N, vec, z);
    if constexpr (GATED) {
      load8<T>(a.pre, t * a.ldp + a.N, n, a.N, vec, u);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float da = d[i];
        d[i] = da * u[i] * act_slope<FAST>(a.act, z[i]);
        u[i] = da * act_fn<FAST>(a.act, z[i]);
        s1[i] += u[i];
      }
    } else if (a.pre) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = n + i < a.N ? d[i] * act_slope<FAST>(a.act, z[i]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s0[i] += d[i];
    if (a.dz) {
      Piece<T>::store(a.dz, t * a.ldz + n, d);
      if constexpr (GATED) Piece<T>::store(a.dz, t * a.ldz + a.N + n, u);
    }
  }
  if (a.part) {
    const int64_t cols = GATED ? 2 * (int64_t)a.N : a.N;
    float* out = a.part + blockIdx.x * cols;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (n + i < a.N) {
        out[n + i] = s0[i];
        if (GATED) out[a.N + n + i] = s1[i];
      }
  }
}

// 64 columns a workgroup; wave w adds rows w, w + 4, ... and the four sums are added in order
__global__ __launch_bounds__(kThreads) void column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t cols,
                                                              void* __restrict__ out, int f32) {
  __shared__ float red[4][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * kWave + lane;
  float s = 0.f;
  if (c < cols)
    for (int64_t r = wave; r < rows; r += 4) s += part[r * cols + c];
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < cols) {
    s = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
    if (f32) Piece<float>::put(out, c, s);
    else Piece<uint16_t>::put(out, c, s);
  }
}

__global__ __launch_bounds__(kThreads) void zero_bytes_kernel(uint8_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) p[i] = 0;
}

template <typename T>
hipError_t launch(const DzArgs& a, int vec, hipStream_t s) {
  const int64_t width = a.gated ? a.N : a.ldz;
  const dim3 grid((unsigned)dz_parts(a.T), (unsigned)((width + 8 * kThreads - 1) / (8 * kThreads)));
  if (a.gated) hipLaunchKernelGGL((dz_kernel<T, true>), grid, dim3(kThreads), 0, s, a, vec);
  else hipLaunchKernelGGL((dz_kernel<T, false>), grid, dim3(kThreads), 0, s, a, vec);
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
  hipError_t err = f32 ? launch<float>(a, vec, s) : launch<uint16_t>(a, vec, s);
  if (err != hipSuccess || !a.dbias) return err;
  return launch_column_sum(a.part, dz_parts(a.T), a.gated ? 2 * (int64_t)a.N : a.N, a.dbias, f32, s);
}

hipError_t launch_column_sum(const float* part, int64_t rows, int64_t cols, void* out, bool f32, hipStream_t s) {
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((cols + kWave - 1) / kWave)), dim3(kThreads), 0, s, part, rows,
                     cols, out, f32 ? 1 : 0);
  return hipGetLastError();
}

hipError_t launch_zero_bytes(void* p, int64_t bytes, hipStream_t s) {
  const int64_t b = (bytes + kThreads - 1) / kThreads;
  hipLaunchKernelGGL(zero_bytes_kernel, dim3((unsigned)(b < 1 ? 1 : (b > 4096 ? 4096 : b))), dim3(kThreads), 0, s,
                     static_cast<uint8_t*>(p), bytes);
  return hipGetLastError();
}

}  // namespace moe
