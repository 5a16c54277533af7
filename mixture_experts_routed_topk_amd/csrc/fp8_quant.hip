// Quantisers of the e4m3 products: the backward pass's operands, weights in blocks, and the
// table of an expert-sorted batch's row tiles (gfx950).
//
// A group's scale is a power of two where the block-scaled MFMA is to apply it: the smallest s with
// amax <= 448 s (1 for a group of zeros, at least 2^-126).  x / s is then exact, so a code carries one
// rounding.  The gradient dz goes to e4m3 twice, from the same float32 values, because the two products
// contract over different indices: in groups of 128 columns for dx = dz w and of 128 rows for dw =
// dz^T x.  Both keep dz's row order, as the products read either storage order.
//
// A workgroup takes 128 rows x 128 columns: one group of each kind per row and column.  Its values are read once
// and held in registers (a thread: four rows, eight columns); row maxima go over 16 lanes, column maxima over a
// wave's four rows and the eight waves.  Memory-bound: two bytes read and two written per element of dz, two and
// one of x.  16384 rows of 32 runs, dz 2 x 2048 and x 7168 columns with silu: 0.69 GB in 157 us (4.4 TB/s).  2731 rows, dz 5632 and x 2048 columns
// with GELU: 0.11 GB in 32 us; there the erf's polynomial and the maxima keep the vector units busy for about 22.
#include "dense_device.h"
#include "fp8_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 4;              // rows of a thread: 32 apart

// UE8M0 byte of the smallest power of two s >= 2^-126 with top <= 448 s; 127 for 0.  448 = 1.75 * 2^8.
__device__ __forceinline__ int pow2_over(float top) {
  const uint32_t u = __float_as_uint(top);
  const int b = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return u == 0 ? 127 : (b < 1 ? 1 : b);
}
__device__ __forceinline__ float pow2(int b) { return __uint_as_float((uint32_t)b << 23); }   // 1 <= b <= 254

// codes of eight values times f (the values are at most 448 after that; infinities and NaN give NaN)
__device__ __forceinline__ uint2 codes8(const float v[8], float f) {
  uint32_t lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * f, v[1] * f, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * f, v[3] * f, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * f, v[5] * f, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * f, v[7] * f, hi, true);
  return make_uint2(lo, hi);
}

// The largest of 16 neighbouring lanes, for each of them (rotations by DPP: no trip through LDS)
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, false)));   // by 8
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xf, 0xf, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xf, 0xf, false)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xf, 0xf, false)));
}
// join(v, v of the lane 16 on), then of the lane 32 on, for each lane
template <typename F>
__device__ __forceinline__ float across_rows(float v, F&& join) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = join(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return join(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Codes of a 128 x 128 tile.  col: first of this thread's eight columns in the outputs of pitch C
struct TileOut {
  uint8_t* row_codes;      // null: not wanted
  void* row_scale;         // [rows][C / 128]
  int row_f32;
  uint8_t* col_codes;      // of this tile: [128][C], rows past the tile's are zeros; null: not wanted
  uint8_t* col_scale;      // of this tile: [C]
  float* sums;             // of this tile: [C], null: not wanted
};
__device__ __forceinline__ void store_tile(const float (&v)[kRows][8], const TileOut& o, int64_t row0, int rows, int col, int C,
                                           float (*red)[kWaves][128]) {
  const int sub = threadIdx.x & 15, rr = threadIdx.x >> 4, wave = threadIdx.x >> 6;
  if (o.row_codes) {
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = rr + 32 * u;
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[u][i]));
      top = row_max(top);
      const int b = pow2_over(top);
      if (r < rows) {
        *reinterpret_cast<uint2*>(o.row_codes + (row0 + r) * C + col) = codes8(v[u], pow2(254 - b));
        if (sub == 0) {
          const int64_t at = (row0 + r) * (C / 128) + col / 128;
          if (o.row_f32) static_cast<float*>(o.row_scale)[at] = pow2(b);
          else static_cast<uint8_t*>(o.row_scale)[at] = (uint8_t)b;
        }
      }
    }
  }
  if (!o.col_codes && !o.sums) return;
  float top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top[i] = 0.f;
#pragma unroll
    for (int u = 0; u < kRows; ++u) top[i] = fmaxf(top[i], fabsf(v[u][i]));
    top[i] = across_rows(top[i], [](float a, float b) { return fmaxf(a, b); });
  }
  __syncthreads();                     // (red may still be read from the tile's other half)
  if ((threadIdx.x & 48) == 0) Piece<float>::store(red[0][wave], sub * 8, top);
  if (o.sums) {
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum[i] = 0.f;
#pragma unroll
      for (int u = 0; u < kRows; ++u) sum[i] += v[u][i];
      sum[i] = across_rows(sum[i], [](float a, float b) { return a + b; });
    }
    if ((threadIdx.x & 48) == 0) Piece<float>::store(red[1][wave], sub * 8, sum);
  }
  __syncthreads();
  if (o.sums && threadIdx.x < 16) {
    float s[8] = {};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      float t[8];
      Piece<float>::load(red[1][w], sub * 8, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += t[i];
    }
    Piece<float>::store(o.sums, col, s);
  }
  if (!o.col_codes) return;
  float f[8];
  uint32_t bytes[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) top[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    float t[8];
    Piece<float>::load(red[0][w], sub * 8, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = fmaxf(top[i], t[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int b = pow2_over(top[i]);
    bytes[i] = (uint32_t)b;
    f[i] = pow2(254 - b);
  }
  if (threadIdx.x < 16) {
    uint2 s;
    s.x = bytes[0] | bytes[1] << 8 | bytes[2] << 16 | bytes[3] << 24;
    s.y = bytes[4] | bytes[5] << 8 | bytes[6] << 16 | bytes[7] << 24;
    *reinterpret_cast<uint2*>(o.col_scale + col) = s;
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = v[u][i] * f[i];
    *reinterpret_cast<uint2*>(o.col_codes + (int64_t)(rr + 32 * u) * C + col) = codes8(w, 1.0f);
  }
}

// A thread's values as they are stored; rows past the tile's are zeros
__device__ __forceinline__ void load_tile(const void* p, int64_t ld, int64_t row0, int rows, int col, i32x4 (&raw)[kRows]) {
  const int rr = threadIdx.x >> 4;
#pragma unroll
  for (int u = 0; u < kRows; ++u) raw[u] = Piece<uint16_t>::raw(p, (row0 + min(rr + 32 * u, rows - 1)) * ld + col);
#pragma unroll
  for (int u = 0; u < kRows; ++u) raw[u] &= rr + 32 * u < rows ? -1 : 0;
}

// Workgroup (x, y): column block x of dz, or behind those of x; row tile y
template <int ACT, bool GATED>
__global__ __launch_bounds__(kThreads) void groups_kernel(GroupsArgs a, int dz_blocks) {
  __shared__ float red[2][kWaves][128];
  const int tile = blockIdx.y;
  int64_t row0 = (int64_t)tile * 128;
  int rows = (int)min((int64_t)128, a.T - row0);
  if (a.tiles) {
    if (tile >= a.count[0]) return;
    const RowTile t = a.tiles[tile];
    row0 = t.start + (tile - t.first) * 128;
    rows = min(128, t.end - (int)row0);
  }
  const int sub = threadIdx.x & 15;
  const int64_t cols = GATED ? 2 * (int64_t)a.N : a.N;
  float v[kRows][8];
  i32x4 raw[kRows];
  if ((int)blockIdx.x >= dz_blocks) {
    const int col = ((int)blockIdx.x - dz_blocks) * 128 + sub * 8;
    load_tile(a.x, a.ldx, row0, rows, col, raw);
#pragma unroll
    for (int u = 0; u < kRows; ++u) Piece<uint16_t>::widen(raw[u], v[u]);
    store_tile(v, TileOut{nullptr, nullptr, 0, a.xc + (int64_t)tile * 128 * a.K, a.xc_scale + (int64_t)tile * a.K, nullptr}, row0, rows, col, a.K, red);
    return;
  }
  const int col = (int)blockIdx.x * 128 + sub * 8;
  TileOut o{a.zr, a.zr_scale, a.zr_f32, a.zc ? a.zc + tile * 128 * cols : nullptr, a.zc_scale ? a.zc_scale + tile * cols : nullptr,
            a.part ? a.part + tile * cols : nullptr};
  load_tile(a.dy, a.ldy, row0, rows, col, raw);
  if constexpr (GATED) {
    // one half after the other, from the operands as they were loaded: both halves' float32 values would take the registers of a workgroup
    i32x4 gate[kRows], up[kRows];
    load_tile(a.pre, a.ldp, row0, rows, col, gate);
    load_tile(a.pre, a.ldp, row0, rows, a.N + col, up);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float da[8], ug[8], z[8];
      Piece<uint16_t>::widen(gate[u], z);
      Piece<uint16_t>::widen(raw[u], da);
      Piece<uint16_t>::widen(up[u], ug);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = times_slope(ACT, da[i] * ug[i], act_pair<true>(ACT, z[i]).slope);
      __builtin_amdgcn_sched_barrier(0);
    }
    store_tile(v, o, row0, rows, col, (int)cols, red);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kRows; ++u) asm volatile("" : "+v"(gate[u]), "+v"(raw[u]));
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float da[8], z[8];
      Piece<uint16_t>::widen(gate[u], z);
      Piece<uint16_t>::widen(raw[u], da);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = da[i] * act_pair<true>(ACT, z[i]).value;
      __builtin_amdgcn_sched_barrier(0);
    }
    store_tile(v, o, row0, rows, a.N + col, (int)cols, red);
  } else {
    if constexpr (ACT != kActNone) {
      i32x4 pre[kRows];
      load_tile(a.pre, a.ldp, row0, rows, col, pre);
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        float z[8];
        Piece<uint16_t>::widen(pre[u], z);
        Piece<uint16_t>::widen(raw[u], v[u]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = times_slope(ACT, v[u][i], act_pair<true>(ACT, z[i]).slope);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kRows; ++u) Piece<uint16_t>::widen(raw[u], v[u]);
    }
    store_tile(v, o, row0, rows, col, (int)cols, red);
  }
}

// ---------------------------------------------------------------------------- weights
// One pass: a block is held in registers between its maximum and its codes.  60 x 2816 x 2048 bf16: 190 us, 1.04 GB at 5.5 TB/s.
// Workgroup (x, y, z): block (y, x) of matrix z.  The float32 scale follows the rule of the row quantiser: amax / 448
// correctly rounded, codes as the float32 quotient rounds.
template <typename T, bool UE8>
__global__ __launch_bounds__(kThreads) void blocks_kernel(const void* __restrict__ w, int N, int K, uint8_t* __restrict__ q,
                                                          void* __restrict__ scale) {
  __shared__ float red[kWaves];
  const int sub = threadIdx.x & 15, rr = threadIdx.x >> 4;
  const int64_t first = ((int64_t)blockIdx.z * N + blockIdx.y * 128) * K + (int64_t)blockIdx.x * 128;
  typename Piece<T>::Raw raw[kRows];
  float v[kRows][8];
#pragma unroll
  for (int u = 0; u < kRows; ++u) raw[u] = Piece<T>::raw(w, first + (int64_t)(rr + 32 * u) * K + sub * 8);
  float top = 0.f;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    Piece<T>::widen(raw[u], v[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[u][i]));
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) top = fmaxf(top, red[i]);
  const int64_t at = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  uint8_t* out = q + first + (int64_t)rr * K + sub * 8;
  if constexpr (UE8) {
    const int b = pow2_over(top);
    if (threadIdx.x == 0) static_cast<uint8_t*>(scale)[at] = (uint8_t)b;
#pragma unroll
    for (int u = 0; u < kRows; ++u) *reinterpret_cast<uint2*>(out + (int64_t)(32 * u) * K) = codes8(v[u], pow2(254 - b));
  } else {
    const float s0 = top / 448.0f, s = s0 > 0.f ? s0 : 1.0f;
    if (threadIdx.x == 0) static_cast<float*>(scale)[at] = s;
    if (s0 > 0x1p-96f && s0 < 0x1p96f) {   // v / s from one reciprocal, its error taken back once: rounds as the division
      const float inv = 1.0f / s;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float quo = v[u][i] * inv;
          d[i] = fmaf(fmaf(-quo, s, v[u][i]), inv, quo);
        }
        *reinterpret_cast<uint2*>(out + (int64_t)(32 * u) * K) = codes8(d, 1.0f);
      }
    } else {   // (a scale of few bits saturates, as in the row quantiser)
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo |= f32_to_e4m3(v[u][i] / s) << (8 * i);
          hi |= f32_to_e4m3(v[u][4 + i] / s) << (8 * i);
        }
        *reinterpret_cast<uint2*>(out + (int64_t)(32 * u) * K) = make_uint2(lo, hi);
      }
    }
  }
}

// ---------------------------------------------------------------------------- runs of rows
constexpr int kMaxE = 1024;

// Inclusive scans over N values of each of a workgroup's kMaxE threads, side by side
template <int N, typename F>
__device__ __forceinline__ void scan(int32_t (&v)[N], int32_t (&lds)[N][16], F&& join) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int32_t o = __shfl_up(v[n], d, 64);
      if (lane >= d) v[n] = join(v[n], o);
    }
  }
  if (lane == 63) {
#pragma unroll
    for (int n = 0; n < N; ++n) lds[n][wave] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 15; ++w) {                // (no value is negative)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = join(v[n], w < wave ? lds[n][w] : 0);
  }
}

__device__ void list_tiles(RowTile* out, const int32_t* start, const int32_t* first, int E, int n) {
  for (int i = threadIdx.x; i < n; i += kMaxE) {
    int lo = 0, hi = E - 1;           // the last expert whose first tile is at most i, and which has one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    out[i] = RowTile{lo, start[lo], start[lo + 1], first[lo], first[lo + 1] - first[lo], {}};
  }
}

__global__ __launch_bounds__(kMaxE) void runs_kernel(Runs r, const int32_t* __restrict__ offsets, int T, int E) {
  __shared__ int32_t alive, ends[1][16], sums[3][16], start[kMaxE + 1], first[kMaxE + 1], group[kMaxE + 1];
  const int e = threadIdx.x;
  const int32_t begin0 = min(max(offsets[0], 0), T);
  int32_t end[1] = {e < E ? min(max(offsets[e + 1], begin0), T) : 0};
  scan(end, ends, [](int32_t a, int32_t b) { return a > b ? a : b; });
  if (e < E) start[e + 1] = end[0];
  if (e == 0) start[0] = begin0, first[0] = 0, group[0] = 0;
  __syncthreads();
  const int cnt = e < E ? end[0] - start[e] : 0;
  // row tiles, 128-row tiles and experts with rows, up to this one (threads past E have none)
  int32_t sum[3] = {(cnt + r.height - 1) / r.height, (cnt + 127) / 128, cnt > 0 ? 1 : 0};
  scan(sum, sums, [](int32_t a, int32_t b) { return a + b; });
  if (e < E) first[e + 1] = sum[0], group[e + 1] = sum[1];
  if (e == kMaxE - 1) r.count[0] = sum[0], r.count[1] = sum[1], r.count[2] = alive = sum[2];
  __syncthreads();
  if (e < E) r.order[cnt > 0 ? sum[2] - 1 : alive + e - sum[2]] = e;
  for (int i = e; i <= E; i += kMaxE) r.group[i] = group[i];
  list_tiles(r.tiles, start, first, E, first[E]);
  if (r.height != 128) list_tiles(r.groups, start, group, E, group[E]);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t runs_bytes(int64_t T, int E, int height) {
  if (E == 0) return 0;
  return up256(4 * (2 * (size_t)E + 4)) + up256(sizeof(RowTile) * (size_t)max_row_tiles(T, E, height)) +
         (height == 128 ? 0 : up256(sizeof(RowTile) * (size_t)max_row_tiles(T, E, 128)));
}

Runs runs_at(void* ws, int64_t T, int E, int height) {
  Runs r{};
  r.height = height;
  r.group = static_cast<int32_t*>(ws);
  r.order = r.group + E + 1;
  r.count = r.order + E;
  char* p = static_cast<char*>(ws) + up256(4 * (2 * (size_t)E + 4));
  r.tiles = reinterpret_cast<RowTile*>(p);
  r.groups = height == 128 ? r.tiles : reinterpret_cast<RowTile*>(p + up256(sizeof(RowTile) * (size_t)max_row_tiles(T, E, height)));
  return r;
}

hipError_t launch_runs(const Runs& r, const int32_t* offsets, int64_t T, int E, hipStream_t s) {
  hipLaunchKernelGGL(runs_kernel, dim3(1), dim3(kMaxE), 0, s, r, offsets, (int)T, E);
  return hipGetLastError();
}

hipError_t launch_groups(const GroupsArgs& a, hipStream_t s) {
  const int dz_blocks = a.zr || a.zc || a.part ? a.N / 128 : 0, x_blocks = a.xc ? a.K / 128 : 0;
  const dim3 grid((unsigned)(dz_blocks + x_blocks), (unsigned)a.max_tiles);
  auto launch = [&](auto act, auto gated) {
    hipLaunchKernelGGL((groups_kernel<decltype(act)::value, decltype(gated)::value>), grid, dim3(kThreads), 0, s, a, dz_blocks);
  };
  auto by_act = [&](auto gated) {
    if (a.act == kActSilu) launch(std::integral_constant<int, kActSilu>{}, gated);
    else if (a.act == kActGelu) launch(std::integral_constant<int, kActGelu>{}, gated);
    else launch(std::integral_constant<int, kActRelu>{}, gated);
  };
  if (a.gated) by_act(std::true_type{});
  else if (a.pre) by_act(std::false_type{});
  else launch(std::integral_constant<int, kActNone>{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_blocks(const void* w, bool f32, int count, int N, int K, bool ue8m0, uint8_t* q, void* scale, hipStream_t s) {
  const dim3 grid((unsigned)(K / 128), (unsigned)(N / 128), (unsigned)count);
  if (f32 && ue8m0) hipLaunchKernelGGL((blocks_kernel<float, true>), grid, dim3(kThreads), 0, s, w, N, K, q, scale);
  else if (f32) hipLaunchKernelGGL((blocks_kernel<float, false>), grid, dim3(kThreads), 0, s, w, N, K, q, scale);
  else if (ue8m0) hipLaunchKernelGGL((blocks_kernel<uint16_t, true>), grid, dim3(kThreads), 0, s, w, N, K, q, scale);
  else hipLaunchKernelGGL((blocks_kernel<uint16_t, false>), grid, dim3(kThreads), 0, s, w, N, K, q, scale);
  return hipGetLastError();
}

}  // namespace moe
