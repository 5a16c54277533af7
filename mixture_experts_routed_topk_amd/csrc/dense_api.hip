// C ABI of the dense operators around the routed experts: argument validation (before any
// HIP call), workspace layouts and launches.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/moe_experts.h"
#include "dense_internal.h"

namespace moe {
namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;   // one workgroup of 1024 threads to a row stays below 2^32 threads
constexpr int64_t kMaxPitch = int64_t(1) << 22;   // tile offsets fit in 32 bits
constexpr int kMaxWidth = 65536;                  // H, I, K
constexpr int kMaxOutputs = 1 << 20;              // N
constexpr int64_t kMaxElements = int64_t(1) << 34;  // of any matrix: a thread to eight of them stays below 2^32 threads

bool aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }
bool aligned4(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0; }
template <typename... P>
bool all_aligned16(P... p) { return (aligned16(p) && ...); }
bool type_ok(int t) { return t == MOE_F32 || t == MOE_BF16; }
bool width_ok(int w) { return w >= 8 && w <= kMaxWidth && w % 8 == 0; }
bool pitch_ok(int64_t ld, int64_t cols, bool vec) {
  return ld == 0 || (ld >= cols && ld <= kMaxPitch && (!vec || ld % 8 == 0));
}
int64_t pitch(int64_t ld, int64_t cols) { return ld ? ld : cols; }
size_t up256(size_t v) { return (v + 255) & ~size_t(255); }
size_t esize(int t) { return t == MOE_F32 ? 4 : 2; }

moe_status check(const moe_norm_problem* p) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (!type_ok(p->dtype)) return MOE_ERR_UNSUPPORTED;
  if (p->T < 0 || p->T > kMaxRows || !width_ok(p->H) || !(p->eps >= 0.f) || !isfinite(p->eps)) return MOE_ERR_BAD_SHAPE;
  for (int64_t ld : {p->ldx, p->ldr, p->ldh, p->ldy})
    if (!pitch_ok(ld, p->H, true)) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

moe_status check(const moe_linear_problem* p) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (!type_ok(p->dtype) || (p->out_dtype != p->dtype && p->out_dtype != MOE_F32)) return MOE_ERR_UNSUPPORTED;
  if (p->act < MOE_ACT_NONE || p->act > MOE_ACT_RELU) return MOE_ERR_UNSUPPORTED;
  if (p->T < 0 || p->T > kMaxRows || !width_ok(p->K) || p->N < 1 || p->N > kMaxOutputs ||
      p->T * p->N > kMaxElements || p->T * p->K > kMaxElements || (int64_t)p->N * p->K > kMaxElements)
    return MOE_ERR_BAD_SHAPE;
  if (!pitch_ok(p->ldx, p->K, true) || !pitch_ok(p->lddx, p->K, true)) return MOE_ERR_BAD_SHAPE;
  for (int64_t ld : {p->ldy, p->ldr, p->ldp})
    if (!pitch_ok(ld, p->N, false)) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

moe_status check(const moe_gated_problem* p) {
  if (!p) return MOE_ERR_NULL_ARG;
  if (!type_ok(p->dtype)) return MOE_ERR_UNSUPPORTED;
  if (p->act < MOE_ACT_SILU || p->act > MOE_ACT_RELU) return MOE_ERR_UNSUPPORTED;
  if (p->T < 0 || p->T > kMaxRows || !width_ok(p->H) || !width_ok(p->I) || p->T * p->H > kMaxElements ||
      2 * p->T * p->I > kMaxElements)
    return MOE_ERR_BAD_SHAPE;
  if (!pitch_ok(p->ldx, p->H, true) || !pitch_ok(p->lddx, p->H, true) || !pitch_ok(p->lda, p->I, true) ||
      !pitch_ok(p->ldp, 2 * (int64_t)p->I, true))
    return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

// The backward pass of a linear or gated projection in one form: dz has `cols` columns, the
// products contract over T (dw) and over dz's columns (dx).
struct Backward {
  int64_t T;
  int K;             // columns of x
  int N;             // columns of dy
  int64_t cols;      // columns of dz (gated: 2 N)
  int dtype, dy_dtype, act, gated;
  int64_t ldx, ldy, ldp, lddx;
};
Backward backward_of(const moe_linear_problem& p) {
  return {p.T, p.K, p.N, p.N, p.dtype, p.out_dtype, p.act, 0,
          pitch(p.ldx, p.K), pitch(p.ldy, p.N), pitch(p.ldp, p.N), pitch(p.lddx, p.K)};
}
Backward backward_of(const moe_gated_problem& p) {
  return {p.T, p.H, p.I, 2 * (int64_t)p.I, p.dtype, p.dtype, p.act, 1,
          pitch(p.ldx, p.H), pitch(p.lda, p.I), pitch(p.ldp, 2 * (int64_t)p.I), pitch(p.lddx, p.H)};
}

// dz is dy itself when nothing is to be done to it and the products can read its rows in
// 16-byte pieces; otherwise it is written to the workspace.
bool dz_is_dy(const Backward& b) {
  return !b.gated && b.act == MOE_ACT_NONE && b.dy_dtype == b.dtype && b.N % 8 == 0 && b.ldy % 8 == 0;
}
// With few rows the products take dz in two bf16 parts, its rounding and what that took.  One part puts dw off by 2.3 to
// 2.6e-3 of its norm at any number of rows, 1.7e-3 of it from its own rounding; two leave the 1.7e-3.  Many rows do without:
// the products are bound by the MFMA and would take twice as long.  Few rows are bound by the weights, and up to 32
// one 64-row tile holds both parts, so the weights are read once: the limit is where that ends, and with 33 rows the
// gradients have the precision of many.  The sum of the parts costs 2 to 5 us (16 rows, gated
// 2048 x 1408: 19.6 against 15.9 us, 7168 x 2048: 37.6 against 34.6).
constexpr int64_t kTwoPartRows = 32;
bool dz_in_two_parts(const Backward& b) {
  // (a bf16 dy that relu's slope only keeps or drops is a bf16 dz already)
  const bool exact = b.dy_dtype == MOE_BF16 && !b.gated && (b.act == MOE_ACT_NONE || b.act == MOE_ACT_RELU);
  return b.dtype == MOE_BF16 && b.T <= kTwoPartRows && !exact;
}
int64_t dz_pitch(const Backward& b) { return (b.cols + 7) / 8 * 8; }

struct BackwardLayout {
  size_t dz, x2, part, gemm, total;
};
BackwardLayout layout(const Backward& b, bool bias) {
  BackwardLayout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = up256(o + bytes);
    return at;
  };
  const bool f32 = b.dtype == MOE_F32;
  const bool two = dz_in_two_parts(b);
  const int64_t rows = two ? 2 * b.T : b.T;        // of the products' dz and x
  L.dz = take(dz_is_dy(b) ? 0 : (size_t)rows * dz_pitch(b) * esize(b.dtype));
  L.x2 = take(two ? (size_t)rows * b.K * esize(b.dtype) : 0);
  L.part = take(bias ? (size_t)dz_parts(b.T) * b.cols * 4 : 0);
  L.gemm = take(dense_gradients_workspace(rows, b.K, b.cols, f32, two));
  L.total = o;
  return L;
}

// rows of y, residual and pre start on 16 bytes and end on whole pieces of eight
bool stores_pieces(const moe_linear_problem& p) {
  return p.N % 8 == 0 && pitch(p.ldy, p.N) % 8 == 0 && pitch(p.ldr, p.N) % 8 == 0 && pitch(p.ldp, p.N) % 8 == 0;
}
size_t forward_bytes(const moe_linear_problem& p) {
  return dense_gemm_workspace(p.T, p.N, p.K, 0, p.dtype == MOE_F32, stores_pieces(p));
}

#define MOE_HIP_CHECK(expr)                       \
  do {                                            \
    if ((expr) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

moe_status run_backward(const Backward& b, const void* dy, const void* x, const void* w, const void* pre, void* dx,
                        void* dw, void* dbias, void* workspace, size_t workspace_bytes, hipStream_t s) {
  const bool f32 = b.dtype == MOE_F32;
  const bool need_pre = b.act != MOE_ACT_NONE;
  if (b.T > 0 && (!dy || (need_pre && !pre) || (dx && !w) || (dw && !x))) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(dy, x, w, pre, dx, dw, dbias, workspace)) return MOE_ERR_BAD_SHAPE;
  const BackwardLayout L = layout(b, dbias != nullptr);
  if (b.T > 0 && L.total > 0 && !workspace) return MOE_ERR_NULL_ARG;
  if (b.T > 0 && workspace_bytes < L.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();   // an error left by an earlier, unrelated HIP call is not ours
  if (b.T == 0) {
    if (dw) MOE_HIP_CHECK(launch_zero_bytes(dw, b.cols * b.K * (int64_t)esize(b.dtype), s));
    if (dbias) MOE_HIP_CHECK(launch_zero_bytes(dbias, b.cols * (int64_t)esize(b.dtype), s));
    return MOE_OK;
  }
  char* ws = static_cast<char*>(workspace);
  const bool direct = dz_is_dy(b), two = dz_in_two_parts(b);
  const int64_t rows = two ? 2 * b.T : b.T;
  const void* dz = direct ? dy : ws + L.dz;
  const int64_t lddz = direct ? b.ldy : dz_pitch(b);
  if (dbias || (!direct && (dx || dw))) {
    DzArgs a{};
    a.T = b.T;
    a.N = b.N;
    a.gated = b.gated;
    a.act = b.act;
    a.dy = dy;
    a.ldy = b.ldy;
    a.dy_f32 = b.dy_dtype == MOE_F32;
    a.pre = need_pre ? pre : nullptr;
    a.ldp = b.ldp;
    a.dz = !direct && (dx || dw) ? ws + L.dz : nullptr;
    a.ldz = dz_pitch(b);
    if (two && (dx || dw)) {
      a.x = x;
      a.ldx = b.ldx;
      a.x2 = ws + L.x2;
      a.K = dw ? b.K : 0;
    }
    a.part = dbias ? reinterpret_cast<float*>(ws + L.part) : nullptr;
    a.dbias = dbias;
    MOE_HIP_CHECK(launch_dz(a, f32, s));
  }
  auto product = [&](int r_kmajor, const void* c, int64_t ldc, int64_t M, int64_t K, void* out, int64_t ldo) {
    DenseGemm g{};
    g.r = dz;
    g.ldr = lddz;
    g.r_kmajor = r_kmajor;
    g.c = c;
    g.ldc = ldc;
    g.c_kmajor = 1;
    g.M = M;
    g.K = K;
    g.e.out = out;
    g.e.ldo = ldo;
    g.e.N = b.K;
    g.e.vec = 1;
    return g;
  };
  if (dx || dw) {
    const DenseGemm gx = product(0, w, b.K, rows, b.cols, dx, b.lddx),
                    gw = product(1, two ? ws + L.x2 : x, two ? b.K : b.ldx, b.cols, rows, dw, b.K);
    MOE_HIP_CHECK(launch_dense_gradients(dx ? &gx : nullptr, dw ? &gw : nullptr, ws + L.gemm, f32, two, s));
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_rms_norm(const moe_norm_problem* p, const void* x, const void* residual, const void* weight, void* y,
                        void* h, float* rstd, uint8_t* q, float* q_scale, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (q || q_scale) {
    if (p->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (p->H % 128 != 0) return MOE_ERR_BAD_SHAPE;
  }
  if (p->T == 0) return MOE_OK;
  if (!x || !weight || !rstd || (!y && !q) || !q != !q_scale || !residual != !h) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(x, residual, weight, y, h, q) || !aligned4(rstd) || !aligned4(q_scale)) return MOE_ERR_BAD_SHAPE;
  (void)hipGetLastError();
  NormArgs a{};
  a.T = p->T;
  a.H = p->H;
  a.eps = p->eps;
  a.ldx = pitch(p->ldx, p->H);
  a.ldr = pitch(p->ldr, p->H);
  a.ldh = pitch(p->ldh, p->H);
  a.ldy = pitch(p->ldy, p->H);
  a.x = x;
  a.res = residual;
  a.weight = weight;
  a.y = y;
  a.h = h;
  a.rstd = rstd;
  a.q = q;
  a.q_scale = q_scale;
  MOE_HIP_CHECK(launch_rms_norm(a, p->dtype == MOE_F32, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_rms_norm_workspace_size(const moe_norm_problem* p, size_t* bytes) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  *bytes = up256((size_t)norm_backward_parts(p->T, p->H) * p->H * 4);
  return MOE_OK;
}

moe_status moe_rms_norm_backward(const moe_norm_problem* p, const void* dy, const void* h, const void* weight,
                                 const float* rstd, const void* dh, void* dx, void* dweight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f32 = p->dtype == MOE_F32;
  if (!all_aligned16(dy, h, weight, dh, dx, dweight, workspace) || !aligned4(rstd)) return MOE_ERR_BAD_SHAPE;
  if (p->T == 0) {
    (void)hipGetLastError();
    if (dweight) MOE_HIP_CHECK(launch_zero_bytes(dweight, (int64_t)p->H * (int64_t)esize(p->dtype), s));
    return MOE_OK;
  }
  if (!dy || !h || !weight || !rstd || !dx || (dweight && !workspace)) return MOE_ERR_NULL_ARG;
  if (dweight && workspace_bytes < up256((size_t)norm_backward_parts(p->T, p->H) * p->H * 4))
    return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();
  NormArgs a{};
  a.T = p->T;
  a.H = p->H;
  a.ldx = pitch(p->ldx, p->H);
  a.ldr = pitch(p->ldr, p->H);
  a.ldh = pitch(p->ldh, p->H);
  a.ldy = pitch(p->ldy, p->H);
  a.dy = dy;
  a.hin = h;
  a.weight = weight;
  a.rstd_in = rstd;
  a.res = dh;
  a.dx = dx;
  a.dweight = dweight;
  a.part = dweight ? static_cast<float*>(workspace) : nullptr;
  MOE_HIP_CHECK(launch_rms_norm_backward(a, f32, s));
  return MOE_OK;
}

moe_status moe_linear_workspace_size(const moe_linear_problem* p, int backward, size_t* bytes) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  *bytes = backward ? layout(backward_of(*p), backward != MOE_BACKWARD_NO_BIAS).total : forward_bytes(*p);
  return MOE_OK;
}

moe_status moe_linear(const moe_linear_problem* p, const void* x, const void* w, const void* bias, const void* residual,
                      void* y, void* pre, void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  const bool f32 = p->dtype == MOE_F32;
  const size_t need = forward_bytes(*p);
  if (!x || !w || !y || (need && !workspace)) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(x, w, bias, residual, y, pre, workspace)) return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();
  DenseGemm g{};
  g.r = x;
  g.ldr = pitch(p->ldx, p->K);
  g.c = w;
  g.ldc = p->K;
  g.M = p->T;
  g.K = p->K;
  g.e.out = y;
  g.e.ldo = pitch(p->ldy, p->N);
  g.e.out_f32 = p->out_dtype == MOE_F32;
  g.e.bias = bias;
  g.e.res = residual;
  g.e.ldr = pitch(p->ldr, p->N);
  g.e.pre = pre;
  g.e.ldp = pitch(p->ldp, p->N);
  g.e.act = p->act;
  g.e.N = p->N;
  g.e.vec = stores_pieces(*p);
  MOE_HIP_CHECK(launch_dense_gemm(g, workspace, f32, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_linear_backward(const moe_linear_problem* p, const void* dy, const void* x, const void* w,
                               const void* pre, void* dx, void* dw, void* dbias, void* workspace,
                               size_t workspace_bytes, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  return run_backward(backward_of(*p), dy, x, w, pre, dx, dw, dbias, workspace, workspace_bytes,
                      static_cast<hipStream_t>(stream));
}

moe_status moe_gated_linear_workspace_size(const moe_gated_problem* p, int backward, size_t* bytes) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_NULL_ARG;
  *bytes = backward ? layout(backward_of(*p), backward != MOE_BACKWARD_NO_BIAS).total
                    : dense_gemm_workspace(p->T, p->I, p->H, 1, p->dtype == MOE_F32, 1);
  return MOE_OK;
}

moe_status moe_gated_linear(const moe_gated_problem* p, const void* x, const void* w_gate_up, const void* bias, void* a,
                            void* pre, void* workspace, size_t workspace_bytes, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  const bool f32 = p->dtype == MOE_F32;
  const size_t need = dense_gemm_workspace(p->T, p->I, p->H, 1, f32, 1);
  if (!x || !w_gate_up || !a || (need && !workspace)) return MOE_ERR_NULL_ARG;
  if (!all_aligned16(x, w_gate_up, bias, a, pre, workspace)) return MOE_ERR_BAD_SHAPE;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  (void)hipGetLastError();
  DenseGemm g{};
  g.r = x;
  g.ldr = pitch(p->ldx, p->H);
  g.c = w_gate_up;
  g.ldc = p->H;
  g.M = p->T;
  g.K = p->H;
  g.gated = 1;
  g.e.out = a;
  g.e.ldo = pitch(p->lda, p->I);
  g.e.out_f32 = f32;
  g.e.bias = bias;
  g.e.pre = pre;
  g.e.ldp = pitch(p->ldp, 2 * (int64_t)p->I);
  g.e.act = p->act;
  g.e.N = p->I;
  g.e.vec = 1;
  MOE_HIP_CHECK(launch_dense_gemm(g, workspace, f32, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

moe_status moe_gated_linear_backward(const moe_gated_problem* p, const void* da, const void* x, const void* w_gate_up,
                                     const void* pre, void* dx, void* dw, void* dbias, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const moe_status st = check(p);
  if (st != MOE_OK) return st;
  return run_backward(backward_of(*p), da, x, w_gate_up, pre, dx, dw, dbias, workspace, workspace_bytes,
                      static_cast<hipStream_t>(stream));
}

}  // extern "C"
