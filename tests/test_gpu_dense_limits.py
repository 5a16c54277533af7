"""The dense operators at the ends of what their entry points take: most rows, most outputs, longest contraction, widest
pitch, each subset of the gradients, and numbers near the ends of their type's range."""

import ctypes

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_dense import ACT, BF16, EPS, F32, rnd
from test_gpu_dense_layer import same

pytestmark = pytest.mark.gpu


def check_gradients(got, want, what):
    for g, (r, b), name in zip(got, want, ("dx", "dw", "db")):
        ref.check(g, r, b, f"{what} {name}")


def test_most_rows():
    T = 2 ** 22 - 1
    x, w, g = rnd("mx", (T, 8), BF16), rnd("mw", (3, 8), BF16), rnd("mg", (16, 8), BF16)
    y, pre = m.linear(x, w, act=m.ACT_SILU, save_pre=True)
    (ry, by), (rz, bz) = ref.linear(x, w, None, None, "silu", BF16, BF16)
    ref.check(y, ry, by, "y")
    ref.check(pre, rz, bz, "pre")
    dy = rnd("mdy", (T, 3), BF16)
    check_gradients(m.linear_backward(dy, x, w, pre=pre, act=m.ACT_SILU, need_bias=True),
                    ref.backward(*ref.dz_linear(dy, pre, "silu"), x, w, BF16), "linear")
    a, pre = m.gated_linear(x, g, save_pre=True)
    (ra, ba), _ = ref.gated(x, g, None, "silu", BF16)
    ref.check(a, ra, ba, "a")
    check_gradients(m.gated_linear_backward(x, x, g, pre, need_bias=True),
                    ref.backward(*ref.dz_gated(x, pre, "silu"), x, g, BF16), "gated")
    nw = rnd("mn", (8,), BF16, 0.2, 1.0)
    n, h, rstd = m.rms_norm(x, nw, EPS, residual=x)
    (rn, bn), rh, (rr, br), _ = ref.norm(x, nw, EPS, x, BF16)
    ref.check(n, rn, bn, "norm")
    ref.check(rstd, rr, br, "rstd")
    (rx, bx), (rw, bw) = ref.norm_backward(x, h, nw, rstd, n, BF16)
    dx, dw = m.rms_norm_backward(x, h, nw, rstd, dh=n)
    ref.check(dx, rx, bx, "norm dx")
    ref.check(dw, rw, bw, "norm dweight")


@pytest.mark.parametrize("T", [1, 20, 40])
def test_most_outputs(T):
    N = 2 ** 20
    x, w, dy, b = rnd("ox", (T, 16), BF16), rnd("ow", (N, 16), BF16, 0.25), rnd("ody", (T, N), F32), rnd("ob", (N,), BF16)
    y, pre = m.linear(x, w, b, act=m.ACT_GELU, out_dtype=F32, save_pre=True)
    (ry, by), (rz, bz) = ref.linear(x, w, b, None, "gelu", BF16, F32)
    ref.check(y, ry, by, "y")
    ref.check(pre, rz, bz, "pre")
    check_gradients(m.linear_backward(dy, x, w, pre=pre, act=m.ACT_GELU, need_bias=True),
                    ref.backward(*ref.dz_linear(dy, pre, "gelu"), x, w, BF16, two_parts=T <= 32), "linear")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 33])
def test_longest_contraction(T, dtype):
    K = 65536
    x, w, dy = rnd("kx", (T, K), dtype), rnd("kw", (16, K), dtype, K ** -0.5), rnd("kdy", (T, 16), dtype)
    y, pre = m.linear(x, w, act=m.ACT_SILU, save_pre=True)
    (ry, by), _ = ref.linear(x, w, None, None, "silu", dtype, dtype)
    ref.check(y, ry, by, "y")
    check_gradients(m.linear_backward(dy, x, w, pre=pre, act=m.ACT_SILU, need_bias=True),
                    ref.backward(*ref.dz_linear(dy, pre, "silu"), x, w, dtype, two_parts=T <= 32 and dtype is BF16), "linear")
    a, pre = m.gated_linear(x, w, save_pre=True)
    (ra, ba), _ = ref.gated(x, w, None, "silu", dtype)
    ref.check(a, ra, ba, "a")


def test_widest_pitch():
    """Rows 2^22 elements apart, beyond 2 GiB from the first to the last: x, dy, pre and the norm's rows."""
    T, K, N, ld = 300, 72, 272, 2 ** 22
    wide = torch.zeros((T, ld), dtype=BF16, device="cuda")
    x, dy, pre = wide[:, :K], wide[:, 128:128 + N], wide[:, 1024:1024 + N]
    x.copy_(rnd("px", (T, K), BF16))
    dy.copy_(rnd("pdy", (T, N), BF16))
    pre.copy_(rnd("pz", (T, N), BF16))
    w, nw = rnd("pw", (N, K), BF16, K ** -0.5), rnd("pn", (K,), BF16, 0.2, 1.0)
    c = [t.contiguous() for t in (x, dy, pre)]
    assert same(m.linear(x, w, residual=dy)[0], m.linear(c[0], w, residual=c[1])[0])
    for a, b in zip(m.linear_backward(dy, x, w, pre=pre, act=m.ACT_SILU, need_bias=True),
                    m.linear_backward(c[1], c[0], w, pre=c[2], act=m.ACT_SILU, need_bias=True)):
        assert same(a, b)
    half = dy[:, :N // 2]
    for a, b in zip(m.gated_linear_backward(half, x, w, pre, need_bias=True),
                    m.gated_linear_backward(half.contiguous(), c[0], w, c[2], need_bias=True)):
        assert same(a, b)
    for a, b in zip(m.rms_norm(x, nw, residual=dy[:, :K]), m.rms_norm(c[0], nw, residual=c[1][:, :K].contiguous())):
        assert same(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,N", [(20, 136, 264), (200, 264, 136), (1311, 544, 368)])
def test_each_subset_of_the_gradients(T, K, N, dtype):
    """dx, dw and dbias alone and in pairs, with the tensors that are then not read absent, linear and gated."""
    dt, code = (BF16, m.BF16) if dtype == "bf16" else (F32, m.F32)
    x, w = rnd("sx", (T, K), dt), rnd("sw", (2 * N, K), dt, K ** -0.5)
    dz, z, da = rnd("sd", (T, 2 * N), dt), rnd("sz", (T, 2 * N), dt, 1.5), rnd("sda", (T, N), dt)
    L = m.lib()
    forms = [(L.moe_linear_backward, L.moe_linear_workspace_size,
              m.LinearProblem(T, K, 2 * N, code, code, act, 0, 0, 0, 0, 0), dz, z if act else None,
              ref.dz_linear(dz, z, ("none", "silu", "gelu", "relu")[act])) for act in (m.ACT_NONE, m.ACT_GELU, m.ACT_RELU)]
    forms.append((L.moe_gated_linear_backward, L.moe_gated_linear_workspace_size,
                  m.GatedProblem(T, K, N, code, m.ACT_SILU, 0, 0, 0, 0), da, z, ref.dz_gated(da, z, "silu")))
    for k, (fn, size, p, dy, pre, (dzr, e)) in enumerate(forms):
        want = ref.backward(dzr, e, x, w, dt, two_parts=T <= 32 and dt is BF16 and k in (1, 3))
        for mask in range(1, 8):
            need_dx, need_dw, need_db = mask & 1, mask & 2, mask & 4
            n = ctypes.c_size_t(0)
            assert size(ctypes.byref(p), 1 if need_db else 2, ctypes.byref(n)) == 0
            ws = torch.full((n.value + 256,), 0xFF, dtype=torch.uint8, device="cuda")     # NaN in every type
            out = [torch.full(s, float("nan"), dtype=dt, device="cuda") if need else None
                   for s, need in (((T, K), need_dx), ((2 * N, K), need_dw), ((2 * N,), need_db))]
            at = [None if t is None else t.data_ptr()
                  for t in (dy, x if need_dw else None, w if need_dx else None, pre, *out)]
            assert fn(ctypes.byref(p), *at, ws.data_ptr(), n.value, torch.cuda.current_stream().cuda_stream) == 0
            assert bool((ws[n.value:] == 0xFF).all())
            for g, (r, b), name in zip(out, want, ("dx", "dw", "db")):
                if g is not None:
                    ref.check(g, r, b, f"form {k}, subset {mask}: {name}")


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("scale_x,scale_w", [(-126, 20), (-130, 60), (60, 60), (-60, -60)])
def test_far_exponents(T, scale_x, scale_w):
    """Operands near the ends of bf16's range, subnormal ones among them, whose products are ordinary numbers, or small ones."""
    K, N = 136, 72
    x = (rnd("ex", (T, K), F32).double() * 2.0 ** scale_x).to(BF16)
    w = (rnd("ew", (N, K), F32).double() * 2.0 ** scale_w).to(BF16)
    for odt in (BF16, F32):
        y, _ = m.linear(x, w, out_dtype=odt)
        (ry, by), _ = ref.linear(x, w, None, None, "none", BF16, odt)
        ref.check(y, ry, by, f"y {odt}")
