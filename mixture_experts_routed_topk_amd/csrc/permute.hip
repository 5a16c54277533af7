// Rows in expert order and back, and the gradient of the way back (gfx950).
//
// inv[t * k + j] is the sorted position of slot (t, j), as the routing bookkeeping leaves it, or -1:
//   permute            y[inv] = x[t]                     (also the rows' scales, for e4m3 codes)
//   unpermute          out[t] = sum_j w[t, j] y[inv]     (w = 1: the gradient of permute)
//   its gradient       dy[inv] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[inv]>
// All three go by token, whose k rows follow from inv: no atomics are needed, and the sums over j are in slot order.  Rows of
// eight slots go together, so with k <= 8 nothing is read twice; with more, permute and the gradient read a token's row ceil(k / 8) times.  A position outside [0, rows) is treated as
// -1.  Memory-bound, in pieces of 16 bytes; a token's row belongs to 64 lanes, or to 256 where it has
// more than 64 pieces.  4096 tokens of eight slots: codes of 7168 with their scales 61 us (0.27 GB, 4.4 TB/s, most of it stores); the gradient
// of the way back in bf16, a quarter of the slots dropped, 157 us (0.77 GB, 4.9 TB/s).  8192 tokens of four slots, 2048 bf16: the gradient
// of permute 34 us (0.17 GB, 4.9 TB/s).
#include "../../include/moe_experts.h"
#include "dense_device.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;          // slots whose rows are in flight together

struct PermuteArgs {
  int64_t T, rows;
  int k;
  int pieces;                      // 16-byte pieces of a row
  int64_t ldt, ldy;                // pitches in bytes
  const int32_t* inv;
  const float* w;                  // null: 1
  const char* src;                 // permute: x; unpermute: y; gradient: dout
  char* dst;                       // permute: y; unpermute: out; gradient: dy (may be null)
  const char* y;                   // gradient: y (may be dst)
  float* dw;                       // gradient: may be null
  const float* scale;              // permute: [T][groups], null without
  float* scale_out;                // [rows][groups]
  int groups;
};

__device__ __forceinline__ int64_t position(const PermuteArgs& a, int64_t t, int j) {
  const int64_t p = j < a.k ? a.inv[t * a.k + j] : -1;
  return p < a.rows ? p : -1;
}

template <int TPR>
__global__ __launch_bounds__(kThreads) void permute_kernel(PermuteArgs a) {
  const int64_t t = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (t >= a.T) return;
  const int lane = threadIdx.x % TPR;
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    int64_t at[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) at[u] = position(a, t, j0 + u);
    for (int c = lane; c < a.pieces; c += TPR) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(a.src + t * a.ldt + (int64_t)c * 16);
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (at[u] >= 0) *reinterpret_cast<i32x4*>(a.dst + at[u] * a.ldy + (int64_t)c * 16) = v;
    }
    for (int c = lane; c < a.groups; c += TPR) {
      const float v = a.scale[t * a.groups + c];
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
        if (at[u] >= 0) a.scale_out[at[u] * a.groups + c] = v;
    }
  }
}

// a 16-byte piece as float32 values
template <typename T>
struct Sixteen {
  static constexpr int N = 16 / sizeof(T);
  static __device__ __forceinline__ void widen(i32x4 r, float (&v)[N]) {
    if constexpr (sizeof(T) == 2) {
      Piece<T>::widen(r, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __int_as_float(r[i]);
    }
  }
  static __device__ __forceinline__ i32x4 narrow(const float (&v)[N]) {
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) r[i] = (int)pack_bf16x2(v[2 * i], v[2 * i + 1]);
      else r[i] = __float_as_int(v[i]);
    }
    return r;
  }
};

template <typename T, int TPR, bool WEIGHTS>
__global__ __launch_bounds__(kThreads) void unpermute_kernel(PermuteArgs a) {
  constexpr int N = Sixteen<T>::N;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (t >= a.T) return;
  for (int c = threadIdx.x % TPR; c < a.pieces; c += TPR) {
    float s[N] = {};
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
      int64_t at[kSlots];
      i32x4 raw[kSlots];
      float w[kSlots];
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        at[u] = position(a, t, j0 + u);
        w[u] = WEIGHTS && j0 + u < a.k ? a.w[t * a.k + j0 + u] : 1.0f;
      }
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        raw[u] = i32x4{};
        if (at[u] >= 0) raw[u] = *reinterpret_cast<const i32x4*>(a.src + at[u] * a.ldy + (int64_t)c * 16);
      }
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (at[u] < 0) continue;         // (its weight may be anything)
        float v[N];
        Sixteen<T>::widen(raw[u], v);
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = WEIGHTS ? fmaf(w[u], v[i], s[i]) : s[i] + v[i];
      }
    }
    *reinterpret_cast<i32x4*>(a.dst + t * a.ldt + (int64_t)c * 16) = Sixteen<T>::narrow(s);
  }
}

// DOT: dw is wanted
template <typename T, int TPR, bool DOT>
__global__ __launch_bounds__(kThreads) void unpermute_backward_kernel(PermuteArgs a) {
  constexpr int N = Sixteen<T>::N;
  __shared__ float red[kThreads / 64][kSlots];
  const int64_t t = (int64_t)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  if (t >= a.T) return;                  // (TPR == 256: the whole workgroup)
  const int lane = threadIdx.x % TPR, wave = threadIdx.x >> 6;
  for (int j0 = 0; j0 < a.k; j0 += kSlots) {
    int64_t at[kSlots];
    float w[kSlots], dot[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; ++u) {
      at[u] = position(a, t, j0 + u);
      w[u] = a.w && j0 + u < a.k ? a.w[t * a.k + j0 + u] : 1.0f;
      dot[u] = 0.f;
    }
    for (int c = lane; c < a.pieces; c += TPR) {
      float d[N];
      i32x4 raw[kSlots];
      const i32x4 own = *reinterpret_cast<const i32x4*>(a.src + t * a.ldt + (int64_t)c * 16);
      if constexpr (DOT) {
#pragma unroll
        for (int u = 0; u < kSlots; ++u) {
          raw[u] = i32x4{};
          if (at[u] >= 0) raw[u] = *reinterpret_cast<const i32x4*>(a.y + at[u] * a.ldy + (int64_t)c * 16);
        }
      }
      Sixteen<T>::widen(own, d);
#pragma unroll
      for (int u = 0; u < kSlots; ++u) {
        if (at[u] < 0) continue;
        if constexpr (DOT) {
          float v[N];
          Sixteen<T>::widen(raw[u], v);
#pragma unroll
          for (int i = 0; i < N; ++i) dot[u] = fmaf(d[i], v[i], dot[u]);
        }
        if (a.dst) {
          float v[N];
#pragma unroll
          for (int i = 0; i < N; ++i) v[i] = w[u] * d[i];
          *reinterpret_cast<i32x4*>(a.dst + at[u] * a.ldy + (int64_t)c * 16) = Sixteen<T>::narrow(v);
        }
      }
    }
    if constexpr (DOT) {
#pragma unroll
      for (int u = 0; u < kSlots; ++u)
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) dot[u] += __shfl_xor(dot[u], x, 64);
      if constexpr (TPR == 64) {
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if (lane == u && j0 + u < a.k) a.dw[t * a.k + j0 + u] = dot[u];
      } else {
        __syncthreads();                 // (red may still be read)
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
          if ((threadIdx.x & 63) == 0) red[wave][u] = dot[u];
        __syncthreads();
        if (threadIdx.x < kSlots && j0 + (int)threadIdx.x < a.k)
          a.dw[t * a.k + j0 + threadIdx.x] =
              ((red[0][threadIdx.x] + red[1][threadIdx.x]) + red[2][threadIdx.x]) + red[3][threadIdx.x];
      }
    }
  }
}

constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxSorted = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxPitch = int64_t(1) << 22;
constexpr int kMaxWidth = 65536;
constexpr int kMaxSlots = 1024;

bool aligned(const void* q, uintptr_t to) { return (reinterpret_cast<uintptr_t>(q) & (to - 1)) == 0; }
bool pitch_ok(int64_t ld, int64_t cols, int unit) { return ld == 0 || (ld >= cols && ld <= kMaxPitch && ld % unit == 0); }

moe_status check(const moe_permute_problem* p, bool codes) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (p->dtype != MOE_F32 && p->dtype != MOE_BF16 && !(codes && p->dtype == MOE_FP8_E4M3)) return MOE_ERR_UNSUPPORTED;
  const int unit = p->dtype == MOE_FP8_E4M3 ? 16 : 8;
  if (p->T < 0 || p->T > kMaxRows || p->rows < 0 || p->rows > kMaxSorted || p->k < 1 || p->k > kMaxSlots || p->H < 8 ||
      p->H > kMaxWidth || p->H % (p->dtype == MOE_FP8_E4M3 ? 128 : 8) != 0 || !pitch_ok(p->ldt, p->H, unit) ||
      !pitch_ok(p->ldy, p->H, unit))
    return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}
PermuteArgs args_of(const moe_permute_problem& p) {
  const int e = p.dtype == MOE_F32 ? 4 : p.dtype == MOE_BF16 ? 2 : 1;
  PermuteArgs a{};
  a.T = p.T;
  a.rows = p.rows;
  a.k = p.k;
  a.pieces = p.H * e / 16;
  a.ldt = (p.ldt ? p.ldt : p.H) * e;
  a.ldy = (p.ldy ? p.ldy : p.H) * e;
  return a;
}
template <int TPR>
dim3 grid(const PermuteArgs& a) { return dim3((unsigned)((a.T + kThreads / TPR - 1) / (kThreads / TPR))); }

template <typename T, int TPR>
void launch_unpermute(const PermuteArgs& a, hipStream_t s) {
  if (a.w) hipLaunchKernelGGL((unpermute_kernel<T, TPR, true>), grid<TPR>(a), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((unpermute_kernel<T, TPR, false>), grid<TPR>(a), dim3(kThreads), 0, s, a);
}
template <typename T, int TPR>
void launch_backward(const PermuteArgs& a, hipStream_t s) {
  if (a.dw) hipLaunchKernelGGL((unpermute_backward_kernel<T, TPR, true>), grid<TPR>(a), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((unpermute_backward_kernel<T, TPR, false>), grid<TPR>(a), dim3(kThreads), 0, s, a);
}

moe_status launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_permute(const moe_permute_problem* p, const void* x, const float* x_scale, const int32_t* inv, void* y,
                       float* y_scale, void* stream) {
  const moe_status st = check(p, true);
  if (st != MOE_OK) return st;
  if (!x_scale != !y_scale) return MOE_ERR_NULL_ARG;
  if (x_scale && p->dtype != MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  if (p->T == 0 || p->rows == 0) return MOE_OK;
  if (!x || !inv || !y) return MOE_ERR_NULL_ARG;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(inv, 4) || !aligned(x_scale, 4) || !aligned(y_scale, 4))
    return MOE_ERR_BAD_SHAPE;
  (void)hipGetLastError();
  PermuteArgs a = args_of(*p);
  a.inv = inv;
  a.src = static_cast<const char*>(x);
  a.dst = static_cast<char*>(y);
  a.scale = x_scale;
  a.scale_out = y_scale;
  a.groups = x_scale ? p->H / 128 : 0;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.pieces > 64) hipLaunchKernelGGL((permute_kernel<256>), grid<256>(a), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((permute_kernel<64>), grid<64>(a), dim3(kThreads), 0, s, a);
  return launched();
}

moe_status moe_unpermute(const moe_permute_problem* p, const void* y, const int32_t* inv, const float* topk_w, void* out,
                         void* stream) {
  const moe_status st = check(p, false);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if ((!y && p->rows) || !inv || !out) return MOE_ERR_NULL_ARG;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(inv, 4) || !aligned(topk_w, 4)) return MOE_ERR_BAD_SHAPE;
  (void)hipGetLastError();
  PermuteArgs a = args_of(*p);
  a.inv = inv;
  a.w = topk_w;
  a.src = static_cast<const char*>(y);
  a.dst = static_cast<char*>(out);
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->dtype == MOE_F32) a.pieces > 64 ? launch_unpermute<float, 256>(a, s) : launch_unpermute<float, 64>(a, s);
  else a.pieces > 64 ? launch_unpermute<uint16_t, 256>(a, s) : launch_unpermute<uint16_t, 64>(a, s);
  return launched();
}

moe_status moe_unpermute_backward(const moe_permute_problem* p, const void* dout, const void* y, const int32_t* inv,
                                  const float* topk_w, void* dy, float* dtopk_w, void* stream) {
  const moe_status st = check(p, false);
  if (st != MOE_OK) return st;
  if (p->T == 0 || (!dy && !dtopk_w)) return MOE_OK;
  if (!dout || !inv || (dtopk_w && !y && p->rows)) return MOE_ERR_NULL_ARG;
  if (!aligned(dout, 16) || !aligned(y, 16) || !aligned(dy, 16) || !aligned(inv, 4) || !aligned(topk_w, 4) ||
      !aligned(dtopk_w, 4))
    return MOE_ERR_BAD_SHAPE;
  (void)hipGetLastError();
  PermuteArgs a = args_of(*p);
  a.inv = inv;
  a.w = topk_w;
  a.src = static_cast<const char*>(dout);
  a.dst = static_cast<char*>(dy);
  a.y = static_cast<const char*>(y);
  a.dw = dtopk_w;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p->dtype == MOE_F32) a.pieces > 64 ? launch_backward<float, 256>(a, s) : launch_backward<float, 64>(a, s);
  else a.pieces > 64 ? launch_backward<uint16_t, 256>(a, s) : launch_backward<uint16_t, 64>(a, s);
  return launched();
}

}  // extern "C"
