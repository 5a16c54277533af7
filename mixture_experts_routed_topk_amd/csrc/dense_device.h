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
  struct Raw {
    f32x4 a, b;
  };
  static __device__ __forceinline__ Raw raw(const void* p, int64_t at) {
    const f32x4* q = reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + at);
    return {q[0], q[1]};
  }
  static __device__ __forceinline__ void widen(const Raw& r, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r.a[i], v[4 + i] = r.b[i];
  }
  static __device__ __forceinline__ void load(const void* p, int64_t at, float v[8]) { widen(raw(p, at), v); }
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
  typedef i32x4 Raw;
  static __device__ __forceinline__ Raw raw(const void* p, int64_t at) {
    return *reinterpret_cast<const i32x4*>(static_cast<const uint16_t*>(p) + at);
  }
  static __device__ __forceinline__ void widen(const Raw& a, float v[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo((uint32_t)a[i]), v[2 * i + 1] = bf16_hi((uint32_t)a[i]);
  }
  static __device__ __forceinline__ void load(const void* p, int64_t at, float v[8]) { widen(raw(p, at), v); }
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
// Gauss tail of the normal distribution and its density: for |z| with x = |z| / sqrt 2, erfc(x) =
// e^(-x^2) erfcx(x) and erfcx(x) = t p(t), t = 1 / (1 + c x), p a polynomial fitted here in the minimax
// sense to the relative error.  For results rounded to bf16, degree 7 with c = 0.455 (5.1e-7 for x >= 0; in float32
// Phi is off by 4.0e-7, and by 4.4e-6 of itself at z = -12); for float32 results (WIDE), degree 9 with
// c = 0.44 (2.6e-8; in float32 Phi is off by at most 7e-7 + 1.2e-7 z^2 of itself).  One exponential serves Phi and the
// density.  (erfcf and expf: 45 us of vector work in the backward pass of 2731 x 5632 elements.)
struct Gauss {
  float cdf;       // Phi(z)
  float density;   // phi(z)
};
template <bool WIDE>
__device__ __forceinline__ Gauss gauss(float z) {
  constexpr float wide[10] = {-0.039485052f, 0.19474044f,  -0.33856088f, 0.20246184f, -0.047061890f,
                              0.13442233f,   0.17246558f, 0.22454564f,  0.24822831f, 0.24824367f};
  constexpr float narrow[8] = {0.068594001f, -0.23870015f, 0.19744349f, 0.038967494f,
                               0.19179685f,  0.22839320f,  0.25680113f, 0.25670451f};
  constexpr int n = WIDE ? 10 : 8;
  const float e = __expf(-0.5f * z * z);
  const float t = __builtin_amdgcn_rcpf(1.0f + ((WIDE ? 0.44f : 0.455f) * 0.70710678118654752f) * fabsf(z));
  float p = WIDE ? wide[0] : narrow[0];
#pragma unroll
  for (int i = 1; i < n; ++i) p = p * t + (WIDE ? wide[i] : narrow[i % 8]);
  const float tail = 0.5f * p * t * e;
  return {z < 0.f ? tail : 1.0f - tail, 0.39894228040143268f * e};
}

// How an activation is computed.  kActBf16, for results rounded to bf16 (dz among them; dbias is rounded to bf16 after
// its sum): silu on the hardware exp and reciprocal (as in gate_fn), gelu by gauss.  kActWide, for float32
// results of bf16 operands: silu by exp and a division, gelu by the longer gauss.  kActF32: float32 operands.
enum ActKind { kActBf16, kActWide, kActF32 };
template <ActKind KIND>
__device__ __forceinline__ float act_fn(int act, float z) {
  constexpr bool FAST = KIND == kActBf16;
  if (act == kActNone) return z;
  if (KIND != kActF32 && act == kActGelu) return z * gauss<KIND == kActWide>(z).cdf;
  if (act == kActRelu) return z <= 0.0f ? 0.0f : z;   // (NaN stays NaN, as in the other activations)
  return gate_fn<FAST>(act - kActSilu + kGateSilu, z);
}
static_assert(kActGelu - kActSilu + kGateSilu == kGateGelu && kActRelu - kActSilu + kGateSilu == kGateRelu,
              "activations keep the gates' order");

template <ActKind KIND>
__device__ __forceinline__ void act8(int act, float z[8]) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_fn<KIND>(kActSilu, z[i]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_fn<KIND>(kActGelu, z[i]);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = act_fn<KIND>(kActRelu, z[i]);
  }
}

// act(z) and act'(z) together (they share the exponential)
struct ActPair {
  float value, slope;
};
template <bool FAST>
__device__ __forceinline__ ActPair act_pair(int act, float z) {
  if (act == kActSilu) {   // z s and s (1 + z (1 - s)), s = 1 / (1 + e^-z)
    const float s = FAST ? __builtin_amdgcn_rcpf(1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
    return {z * s, s * (1.0f + z * (1.0f - s))};
  }
  if (act == kActGelu) {   // z Phi(z) and Phi(z) + z phi(z)
    if (FAST) {
      const Gauss g = gauss<false>(z);
      return {z * g.cdf, g.cdf + z * g.density};
    }
    const float cdf = 0.5f * erfcf(-0.70710678118654752f * z);
    return {z * cdf, cdf + z * (0.39894228040143268f * expf(-0.5f * z * z))};
  }
  if (act == kActRelu) return {z <= 0.0f ? 0.0f : z, z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z)};
  return {z, 1.0f};
}
// d act'(z): where relu is closed nothing, whatever d holds
__device__ __forceinline__ float times_slope(int act, float d, float slope) {
  return act == kActRelu && slope == 0.0f ? 0.0f : d * slope;
}

// ---------------------------------------------------------------------------- element store
// What the store of eight columns n .. n + 7 (n a multiple of 8) reads besides the sums: the
// bias (the same for every row) and the residual.  Kernels load them for several pieces
// before the first store: a load behind a store waits for it, since the two may alias.
template <typename T, bool GATED>
struct EpiBias {
  typename Piece<T>::Raw z, u;
  __device__ __forceinline__ EpiBias(const DenseEpi& e, int n) : z(), u() {
    if (!e.bias || !e.vec || n >= e.N) return;
    z = Piece<T>::raw(e.bias, n);
    if (GATED) u = Piece<T>::raw(e.bias, e.N + n);
  }
};
struct EpiRes {
  i32x4 lo, hi;   // 16 bytes of bf16, or 32 of float32
};
template <typename T>
__device__ __forceinline__ EpiRes epi_res(const DenseEpi& e, int64_t m, int64_t M, int n) {
  EpiRes r = {};
  if (!e.res || !e.vec || n >= e.N || m >= M) return r;
  const char* p = static_cast<const char*>(e.res) + (m * e.ldr + n) * (e.out_f32 ? 4 : (int)sizeof(T));
  r.lo = *reinterpret_cast<const i32x4*>(p);
  if (e.out_f32) r.hi = *reinterpret_cast<const i32x4*>(p + 16);
  return r;
}

// Stores eight columns of output row m; z (and, gated, u) are the float32 sums.  T is the
// operands' type, WIDE whether float32 results of bf16 operands have an activation (wide_act).  e.vec and n < e.N.
template <typename T, bool GATED, bool WIDE>
__device__ __forceinline__ void epi_store_vec(const DenseEpi& e, int64_t m, int n, float z[8], float u[8],
                                              const EpiBias<T, GATED>& bias, const EpiRes& res) {
  if (e.bias) {
    float b[8];
    Piece<T>::widen(bias.z, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += b[i];
    if (GATED) {
      Piece<T>::widen(bias.u, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] += b[i];
    }
  }
  if (e.pre) {
    Piece<T>::store(e.pre, m * e.ldp + n, z);
    if (GATED) Piece<T>::store(e.pre, m * e.ldp + e.N + n, u);
  }
  act8<sizeof(T) == 4 ? kActF32 : (WIDE ? kActWide : kActBf16)>(e.act, z);
  if (GATED) {
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] *= u[i];
  }
  if (e.res) {
    float r[8];
    if (e.out_f32) Piece<float>::widen({__builtin_bit_cast(f32x4, res.lo), __builtin_bit_cast(f32x4, res.hi)}, r);
    else Piece<uint16_t>::widen(res.lo, r);    // (float32 operands have float32 outputs)
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] += r[i];
  }
  if (e.out_f32) Piece<float>::store(e.out, m * e.ldo + n, z);
  else Piece<T>::store(e.out, m * e.ldo + n, z);
}

// One element (m, n) of the output.
template <typename T, bool GATED>
__device__ __forceinline__ void epi_store1(const DenseEpi& e, int64_t m, int n, float z, float u) {
  if (e.bias) {
    z += Piece<T>::get(e.bias, n);
    if (GATED) u += Piece<T>::get(e.bias, e.N + n);
  }
  if (e.pre) {
    Piece<T>::put(e.pre, m * e.ldp + n, z);
    if (GATED) Piece<T>::put(e.pre, m * e.ldp + e.N + n, u);
  }
  if constexpr (sizeof(T) == 4) z = act_fn<kActF32>(e.act, z);
  else z = !GATED && e.out_f32 ? act_fn<kActWide>(e.act, z) : act_fn<kActBf16>(e.act, z);
  if (GATED) z *= u;
  if (e.res) z += e.out_f32 ? Piece<float>::get(e.res, m * e.ldr + n) : Piece<T>::get(e.res, m * e.ldr + n);
  if (e.out_f32) Piece<float>::put(e.out, m * e.ldo + n, z);
  else Piece<T>::put(e.out, m * e.ldo + n, z);
}

// Eight columns in either way; columns past e.N are not touched.
template <typename T, bool GATED>
__device__ __forceinline__ void epi_store(const DenseEpi& e, int64_t m, int n, float z[8], float u[8],
                                          const EpiBias<T, GATED>& bias, const EpiRes& res) {
  if (n >= e.N) return;
  if (e.vec) {
    if (sizeof(T) == 2 && !GATED && wide_act(e)) epi_store_vec<T, GATED, sizeof(T) == 2 && !GATED>(e, m, n, z, u, bias, res);
    else epi_store_vec<T, GATED, false>(e, m, n, z, u, bias, res);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (n + i < e.N) epi_store1<T, GATED>(e, m, n + i, z[i], u[i]);
}

}  // namespace moe
