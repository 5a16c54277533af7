// C ABI of the e4m3 products with block scales and of the weights' quantiser: argument
// validation (before any HIP call), workspace layouts and launches.
#include <hip/hip_runtime.h>

#include "../../include/moe_experts.h"
#include "fp8_internal.h"

namespace moe {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxPitch = int64_t(1) << 22;     // tile offsets fit in 32 bits
constexpr int kMaxWidth = 65536;
constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxElements = int64_t(1) << 34;  // of any matrix, or of all experts' together: grids stay below 2^32 threads

bool aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }
bool aligned4(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0; }
template <typename... P>
bool all_aligned16(P... p) { return (aligned16(p) && ...); }
bool width_ok(int w) { return w >= 128 && w <= kMaxWidth && w % 128 == 0; }
bool pitch_ok(int64_t ld, int64_t cols, int unit) { return ld == 0 || (ld >= cols && ld <= kMaxPitch && ld % unit == 0); }
int64_t pitch(int64_t ld, int64_t cols) { return ld ? ld : cols; }
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

moe_status check(const moe_fp8_problem* p, bool gated) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (p->scale_fmt != MOE_SCALE_F32 && p->scale_fmt != MOE_SCALE_UE8M0) return MOE_ERR_UNSUPPORTED;
  if (p->act < (gated ? MOE_ACT_SILU : MOE_ACT_NONE) || p->act > MOE_ACT_RELU) return MOE_ERR_UNSUPPORTED;
  if (p->E != 0 && p->act != MOE_ACT_NONE && !gated) return MOE_ERR_UNSUPPORTED;
  const int64_t cols = (gated ? 2 : 1) * (int64_t)p->N;
  const int64_t experts = p->E > 1 ? p->E : 1;
  if (p->T < 0 || p->T > kMaxRows || !width_ok(p->K) || !width_ok(p->N) || p->E < 0 || p->E > kMaxExperts ||
      p->T * cols > kMaxElements || p->T * p->K > kMaxElements || experts * cols * p->K > kMaxElements)
    return MOE_ERR_BAD_SHAPE;
  if (!pitch_ok(p->ldx, p->K, 16) || !pitch_ok(p->lddx, p->K, 8) || !pitch_ok(p->ldy, p->N, 8) || !pitch_ok(p->ldr, p->N, 8) ||
      !pitch_ok(p->ldp, cols, 8))
    return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

struct Size {
  int64_t T, K, cols;
  int N, E, gated, act, ue8m0;
};
Size size_of(const moe_fp8_problem& p, bool gated) {
  return {p.T, p.K, (gated ? 2 : 1) * (int64_t)p.N, p.N, p.E, gated, p.act, p.scale_fmt == MOE_SCALE_UE8M0};
}

// c and its scales: weights [cols][K], blocks [cols / 128][K / 128]
void set_weights(Fp8Gemm& g, const Size& z, const void* w, const void* w_scale, bool along_k) {
  g.g.c = w;
  g.g.ldc = z.K;
  g.g.c_kmajor = !along_k;
  const int64_t kb = z.K / 128;
  g.cs = along_k ? Fp8Scales{w_scale, kb, 1, z.ue8m0} : Fp8Scales{w_scale, 1, kb, z.ue8m0};
  g.c_blocks = 1;
  g.E = z.E;
  g.c_expert = z.cols * z.K;
  g.cs_expert = z.cols / 128 * kb;
}

Fp8Gemm forward_gemm(const Size& z) {
  Fp8Gemm g{};
  g.g.M = z.T;
  g.g.K = z.K;
  g.g.gated = z.gated;
  g.g.e.N = z.N;
  g.E = z.E;
  g.few = fp8_rows_take(z.T, z.K, z.E, z.gated);
  return g;
}
// The tables of runs, of tiles of `height` rows (0: none are needed), then the product's own
struct ForwardLayout {
  int height;
  size_t gemm, total;
};
ForwardLayout forward_layout(const Size& z, const Fp8Gemm& g) {
  ForwardLayout L{};
  if (z.T == 0) return L;
  L.height = z.E && !g.few ? fp8_grouped_height(z.T, z.E, z.K, z.cols) : 0;
  L.gemm = L.height ? up256(runs_bytes(z.T, z.E, L.height)) : 0;
  L.total = L.gemm + fp8_gemm_workspace(g);
  return L;
}

struct BackwardLayout {
  size_t runs, zr, zr_scale, zc, zc_scale, xc, xc_scale, part, gemm, total;
  int64_t tiles;                // 128-row tiles at most
  int height;                   // of dx's tiles by runs
};
BackwardLayout backward_layout(const Size& z, bool bias) {
  BackwardLayout L{};
  if (z.T == 0) return L;
  L.tiles = z.E ? max_row_tiles(z.T, z.E, 128) : (z.T + 127) / 128;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  L.height = z.E ? fp8_dx_height(z.T, z.E, z.cols, z.ue8m0) : 0;
  L.runs = take(z.E ? runs_bytes(z.T, z.E, L.height) : 0);
  L.zr = take(z.T * z.cols);
  L.zr_scale = take(z.T * (z.cols / 128) * 4);
  L.zc = take(L.tiles * 128 * z.cols);
  L.zc_scale = take(L.tiles * z.cols);
  L.xc = take(L.tiles * 128 * z.K);
  L.xc_scale = take(L.tiles * z.K);
  L.part = take(bias ? L.tiles * z.cols * 4 : 0);
  L.gemm = take(fp8_gradients_workspace(z.T, z.K, z.cols, z.E));
  L.total = o;
  return L;
}

#define MOE_HIP_CHECK(expr)                       \
  do {                                            \
    if ((expr) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

moe_status run_forward(const moe_fp8_problem* p, bool gated, const uint8_t* x_q, const float* x_scale, const uint8_t* w_q,
                       const void* w_scale, const int32_t* offsets, const void* bias, const void* residual, void* y, void* pre,
                       void* workspace, size_t workspace_bytes, hipStream_t s) {
  const moe_status st = check(p, gated);
  if (st != MOE_OK) return st;
  const Size z = size_of(*p, gated);
  if (z.E && (bias || residual || (pre && !gated))) return MOE_ERR_UNSUPPORTED;
  if (z.T == 0) return MOE_OK;
  Fp8Gemm g = forward_gemm(z);
  const ForwardLayout L = forward_layout(z, g);
  if (!x_q || !x_scale || !w_q || !w_scale || !y || (z.E && !offsets) || (L.total && !workspace)) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(x_q, w_q, bias, residual, y, pre, workspace) || !aligned4(x_scale) || (!z.ue8m0 && !aligned4(w_scale)) ||
      !aligned4(offsets))
    return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();   // an error left by an earlier, unrelated HIP call is not ours
  char* ws = static_cast<char*>(workspace);
  g.g.r = x_q;
  g.g.ldr = pitch(p->ldx, z.K);
  g.rs = Fp8Scales{x_scale, z.K / 128, 1, 0};
  set_weights(g, z, w_q, w_scale, true);
  g.g.e.out = y;
  g.g.e.ldo = pitch(p->ldy, z.N);
  g.g.e.bias = bias;
  g.g.e.res = residual;
  g.g.e.ldr = pitch(p->ldr, z.N);
  g.g.e.pre = pre;
  g.g.e.ldp = pitch(p->ldp, z.cols);
  g.g.e.act = z.act;
  g.g.e.vec = 1;
  g.offsets = offsets;
  if (L.height) {
    g.runs = runs_at(ws, z.T, z.E, L.height);
    MOE_HIP_CHECK(launch_runs(g.runs, offsets, z.T, z.E, s));
  }
  MOE_HIP_CHECK(launch_fp8_gemm(g, ws + L.gemm, s));
  return MOE_OK;
}

moe_status run_backward(const moe_fp8_problem* p, bool gated, const void* dy, const void* x, const uint8_t* w_q,
                        const void* w_scale, const int32_t* offsets, const void* pre, void* dx, void* dw, void* dbias,
                        void* workspace, size_t workspace_bytes, hipStream_t s) {
  const moe_status st = check(p, gated);
  if (st != MOE_OK) return st;
  const Size z = size_of(*p, gated);
  if (z.E && dbias) return MOE_ERR_UNSUPPORTED;
  const bool need_pre = z.act != MOE_ACT_NONE;
  const BackwardLayout L = backward_layout(z, dbias != nullptr);
  if (z.T > 0 && (!dy || (need_pre && !pre) || (dx && (!w_q || !w_scale)) || (dw && !x) || (z.E && !offsets) || !workspace))
    return MOE_ERR_NULL_ARG;
  if (!all_aligned16(dy, x, w_q, pre, dx, dw, dbias, workspace) || (!z.ue8m0 && !aligned4(w_scale)) || !aligned4(offsets))
    return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();
  if (z.T == 0) {
    if (dw) MOE_HIP_CHECK(launch_zero_bytes(dw, (z.E ? z.E : 1) * z.cols * z.K * 2, s));
    if (dbias) MOE_HIP_CHECK(launch_zero_bytes(dbias, z.cols * 2, s));
    return MOE_OK;
  }
  if (!dx && !dw && !dbias) return MOE_OK;
  char* ws = static_cast<char*>(workspace);
  auto bytes = [&](size_t at) { return reinterpret_cast<uint8_t*>(ws + at); };
  Runs runs{};
  if (z.E) {
    runs = runs_at(ws + L.runs, z.T, z.E, L.height);
    MOE_HIP_CHECK(launch_runs(runs, offsets, z.T, z.E, s));
  }
  GroupsArgs a{};
  a.T = z.T;
  a.N = z.N;
  a.gated = z.gated;
  a.act = z.act;
  a.dy = dy;
  a.ldy = pitch(p->ldy, z.N);
  a.pre = need_pre ? pre : nullptr;
  a.ldp = pitch(p->ldp, z.cols);
  if (dx) {
    a.zr = bytes(L.zr);
    a.zr_scale = bytes(L.zr_scale);
    a.zr_f32 = !z.ue8m0;
  }
  if (dw) {
    a.zc = bytes(L.zc);
    a.zc_scale = bytes(L.zc_scale);
    a.x = x;
    a.ldx = pitch(p->ldx, z.K);
    a.K = (int)z.K;
    a.xc = bytes(L.xc);
    a.xc_scale = bytes(L.xc_scale);
  }
  a.part = dbias ? reinterpret_cast<float*>(ws + L.part) : nullptr;
  a.tiles = z.E ? runs.groups : nullptr;
  a.count = z.E ? runs.count + 1 : nullptr;
  a.max_tiles = L.tiles;
  MOE_HIP_CHECK(launch_groups(a, s));
  if (dbias) MOE_HIP_CHECK(launch_column_sum(a.part, L.tiles, z.cols, dbias, false, s));
  Fp8Gemm gx{}, gw{};
  if (dx) {
    Fp8Gemm& g = gx;
    g.g.r = a.zr;
    g.g.ldr = z.cols;
    g.rs = Fp8Scales{a.zr_scale, z.cols / 128, 1, z.ue8m0};
    set_weights(g, z, w_q, w_scale, false);
    g.g.M = z.T;
    g.g.K = z.cols;
    g.g.e.out = dx;
    g.g.e.ldo = pitch(p->lddx, z.K);
    g.g.e.N = (int)z.K;
    g.g.e.vec = 1;
    g.runs = runs;
  }
  if (dw) {
    Fp8Gemm& g = gw;
    g.g.r = a.zc;
    g.g.ldr = z.cols;
    g.g.r_kmajor = 1;
    g.rs = Fp8Scales{a.zc_scale, 1, z.cols, 1};
    g.g.c = a.xc;
    g.g.ldc = z.K;
    g.g.c_kmajor = 1;
    g.cs = Fp8Scales{a.xc_scale, 1, z.K, 1};
    g.E = z.E;
    g.runs = runs;
    g.g.M = z.cols;
    g.g.K = L.tiles * 128;
    g.g.e.out = dw;
    g.g.e.ldo = z.K;
    g.g.e.N = (int)z.K;
    g.g.e.vec = 1;
  }
  if (dx || dw) MOE_HIP_CHECK(launch_fp8_gradients(dx ? &gx : nullptr, dw ? &gw : nullptr, ws + L.gemm, s));
  return MOE_OK;
}

moe_status workspace_size(const moe_fp8_problem* p, bool gated, int backward, size_t* bytes) {
  const moe_status st = check(p, gated);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  const Size z = size_of(*p, gated);
  *bytes = backward ? backward_layout(z, backward != MOE_BACKWARD_NO_BIAS).total : forward_layout(z, forward_gemm(z)).total;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_blocks_fp8(const void* w, int32_t dtype, int32_t count, int32_t N, int32_t K, int32_t scale_fmt,
                                   uint8_t* q, void* scales, void* stream) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || (scale_fmt != MOE_SCALE_F32 && scale_fmt != MOE_SCALE_UE8M0))
    return MOE_ERR_UNSUPPORTED;
  const bool rows_ok = width_ok(N) || (N % 2 == 0 && width_ok(N / 2));      // (gate and up rows)
  if (count < 0 || count > kMaxExperts || !rows_ok || !width_ok(K) || (int64_t)count * N * K > kMaxElements)
    return MOE_ERR_BAD_SHAPE;
  if (count == 0) return MOE_OK;
  if (!w || !q || !scales) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(w, q) || (scale_fmt == MOE_SCALE_F32 && !aligned4(scales))) return MOE_ERR_BAD_SHAPE;
  (void)hipGetLastError();
  MOE_HIP_CHECK(launch_blocks(w, dtype == MOE_F32, count, N, K, scale_fmt == MOE_SCALE_UE8M0, q, scales,
                              static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_linear_fp8_workspace_size(const moe_fp8_problem* p, int backward, size_t* bytes) {
  return workspace_size(p, false, backward, bytes);
}

moe_status moe_linear_fp8(const moe_fp8_problem* p, const uint8_t* x_q, const float* x_scale, const uint8_t* w_q,
                          const void* w_scale, const int32_t* offsets, const void* bias, const void* residual, void* y,
                          void* pre, void* workspace, size_t workspace_bytes, void* stream) {
  return run_forward(p, false, x_q, x_scale, w_q, w_scale, offsets, bias, residual, y, pre, workspace, workspace_bytes,
                     static_cast<hipStream_t>(stream));
}

moe_status moe_linear_fp8_backward(const moe_fp8_problem* p, const void* dy, const void* x, const uint8_t* w_q,
                                   const void* w_scale, const int32_t* offsets, const void* pre, void* dx, void* dw,
                                   void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  return run_backward(p, false, dy, x, w_q, w_scale, offsets, pre, dx, dw, dbias, workspace, workspace_bytes,
                      static_cast<hipStream_t>(stream));
}

moe_status moe_gated_linear_fp8_workspace_size(const moe_fp8_problem* p, int backward, size_t* bytes) {
  return workspace_size(p, true, backward ? MOE_BACKWARD_NO_BIAS : MOE_FORWARD, bytes);
}

moe_status moe_gated_linear_fp8(const moe_fp8_problem* p, const uint8_t* x_q, const float* x_scale, const uint8_t* w_gate_up_q,
                                const void* w_scale, const int32_t* offsets, void* a, void* pre, void* workspace,
                                size_t workspace_bytes, void* stream) {
  return run_forward(p, true, x_q, x_scale, w_gate_up_q, w_scale, offsets, nullptr, nullptr, a, pre, workspace,
                     workspace_bytes, static_cast<hipStream_t>(stream));
}

moe_status moe_gated_linear_fp8_backward(const moe_fp8_problem* p, const void* da, const void* x, const uint8_t* w_gate_up_q,
                                         const void* w_scale, const int32_t* offsets, const void* pre, void* dx, void* dw,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  return run_backward(p, true, da, x, w_gate_up_q, w_scale, offsets, pre, dx, dw, nullptr, workspace, workspace_bytes,
                      static_cast<hipStream_t>(stream));
}

}  // extern "C"
