// Device helpers of the dense operators: 8-element row pieces, activations and the store of
// a product's elements (DenseEpi).
#pragma once

#include "dense_internal.h"
#include "device_common.h"

namespace moe {

// ---------------------------------------------------------------------------- row pieces
template <typename T>
struct Piece;   // eight consecutive elements of a row as float32

template <>
struct Piece<float> {
  static __device__ __forceinline__ void load(const void* p, int64_t at, float v[8]) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    const f32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  }
  static __device__ __forceinline__ void store(void* p, int64_t at, const float v[8]) {
    f32x4* q = reinterpret_cast<f32x4*>(static_cast<float*>(p) + at);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  }
  static __device__ __forceinline__ float get(const void* p, int64_t at) { return static_cast<const float*>(p)[at]; }
  static __device__ __forceinline__ void put(void* p, int64_t at, float v) { static_cast<float*>(p)[at] = v; }
  static __device__ __forceinline__ float round(float v) { return v; }
};

template <>
struct Piece<uint16_t> {   // bf16 bits
  static __device__ __forceinline__ void load(const void* p, int64_t at, float v[8]) {
    const i32x4 a = *reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo((uint32_t)a[i]), v[2 * i + 1] = bf16_hi((uint32_t)a[i]);
  }
  static __device__ __forceinline__ void store(void* p, int64_t at, const float v[8]) {
    i32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = (int)pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(p) + at) = a;
  }
  static __device__ __forceinline__ float get(const void* p, int64_t at) {
    return bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
  }
  static __device__ __forceinline__ void put(void* p, int64_t at, float v) {
    static_cast<uint16_t*>(p)[at] = (uint16_t)f32_to_bf16_bits(v);
  }
  static __device__ __forceinline__ float round(float v) { return bf16_to_f32((uint16_t)f32_to_bf16_bits(v)); }
};

// ---------------------------------------------------------------------------- activations
// act(z) and its slope.  FAST as in gate_fn: silu on the hardware exp and reciprocal, a few
// float32 ulps off, for results that are rounded to bf16.
template <bool FAST>
__device__ __forceinline__ float act_fn(int act, float z) {
  if (act == kActNone) return z;
  return gate_fn<FAST>(act - kActSilu + kGateSilu, z);
}
static_assert(kActGelu - kActSilu + kGateSilu == kGateGelu && kActRelu - kActSilu + kGateSilu == kGateRelu,
              "activations keep the gates' order");

template <bool FAST>
__device__ __forceinline__ float act_slope(int act, float z) {
  if (act == kActSilu) {   // s (1 + z (1 - s)), s = 1 / (1 + e^-z)
    const float s = FAST ? __builtin_amdgcn_rcpf(1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
    return s * (1.0f + z * (1.0f - s));
  }
  if (act == kActGelu) {   // Phi(z) + z phi(z)
    const float phi = 0.39894228040143268f * expf(-0.5f * z * z);
    return 0.5f * erfcf(-0.70710678118654752f * z) + z * phi;
  }
  if (act == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  return 1.0f;
}

// ---------------------------------------------------------------------------- element store
// Eight columns n .. n + 7 (n a multiple of 8) of output row m; z (and, gated, u) are the
// float32 sums.  T is the operands' type.  Columns past e.N are not touched.
template <typename T, bool GATED>
__device__ __forceinline__ void epi_store(const DenseEpi& e, int64_t m, int n, float z[8], float u[8]) {
  constexpr bool FAST = sizeof(T) == 2;
  if (n >= e.N) return;
  const int cnt = min(8, e.N - n);
  if (e.bias) {
    if (e.vec) {   // (bias shares the alignment rule)
      float b[8];
      Piece<T>::load(e.bias, n, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += b[i];
      if (GATED) {
        Piece<T>::load(e.bias, e.N + n, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] += b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) {
          z[i] += Piece<T>::get(e.bias, n + i);
          if (GATED) u[i] += Piece<T>::get(e.bias, e.N + n + i);
        }
    }
  }
  if (e.pre) {
    const int64_t at = m * e.ldp + n;
    if (e.vec) {
      Piece<T>::store(e.pre, at, z);
      if (GATED) Piece<T>::store(e.pre, at + e.N, u);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < cnt) {
          Piece<T>::put(e.pre, at + i, z[i]);
          if (GATED) Piece<T>::put(e.pre, at + e.N + i, u[i]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = act_fn<FAST>(e.act, z[i]) * (GATED ? u[i] : 1.0f);
  const int64_t at = m * e.ldo + n, rat = m * e.ldr + n;
  if (e.vec) {
    if (e.res) {
      float r[8];
      if (e.out_f32) Piece<float>::load(e.res, rat, r);
      else Piece<T>::load(e.res, rat, r);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] += r[i];
    }
    if (e.out_f32) Piece<float>::store(e.out, at, z);
    else Piece<T>::store(e.out, at, z);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) {
        float v = z[i];
        if (e.res) v += e.out_f32 ? Piece<float>::get(e.res, rat + i) : Piece<T>::get(e.res, rat + i);
        if (e.out_f32) Piece<float>::put(e.out, at + i, v);
        else Piece<T>::put(e.out, at + i, v);
      }
  }
}

}  // namespace moe
