"""The dense operators on values that are not finite, or not of their result's usual range: where an output is
infinite, NaN or finite follows the formula in 64 bits, and finite values keep their bounds (dense_ref.py)."""

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_dense import ACT, BF16, F32, rnd

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def same(a, b):
    """torch.equal as a plain bool (a failure then prints no tensors)"""
    return bool(torch.equal(a, b))


def check_special(got, want, bound, what):
    """Infinities (by sign) and NaN in the same places as in `want`, the rest within `bound`."""
    got = got.double()
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        bad = (kind(got) != kind(want)).sum().item()
        assert bad == 0, f"{what}: {kind.__name__} differs in {bad} places"
    ok = torch.isfinite(want)
    ref.check(torch.where(ok, got, 0.0), torch.where(ok, want, 0.0), torch.where(ok, bound, 0.0), what)


# ----------------------------------------------------------------------------- gradients

def gradients(kind, T, K, N, name, odt, spoil):
    """Both gradients of a linear or gated projection with spoil(x, w, dy, pre) applied to the inputs, and
    the formula's.  At most 32 rows take dz in two bf16 parts unless it is dy itself."""
    cols = 2 * N if kind == "gated" else N
    x, w = rnd("x", (T, K), BF16), rnd("w", (cols, K), BF16, K ** -0.5)
    dy, pre = rnd("dy", (T, N), odt), rnd("z", (T, cols), BF16, 1.5)
    spoil(x, w, dy, pre)
    if kind == "gated":
        dz, e = ref.dz_gated(dy, pre, name)
        got = m.gated_linear_backward(dy, x, w, pre, ACT[name], need_bias=True)
    else:
        dz, e = ref.dz_linear(dy, pre, name)
        got = m.linear_backward(dy, x, w, pre=pre, act=ACT[name], need_bias=True)
    two = T <= 32 and (kind == "gated" or name not in ("none", "relu") or odt is F32)
    return got, ref.backward(dz, e, x, w, BF16, two_parts=two)


FORMS = [("linear", "silu", BF16), ("linear", "none", F32), ("linear", "gelu", F32), ("linear", "none", BF16),
         ("linear", "relu", F32), ("gated", "silu", BF16)]


@pytest.mark.parametrize("kind,name,odt", FORMS)
@pytest.mark.parametrize("T,K,N", [(1, 72, 40), (3, 264, 104), (16, 1032, 2056), (32, 520, 264), (33, 264, 104), (130, 136, 264)])
def test_gradients_with_infinite_operands(T, K, N, kind, name, odt):
    """An infinity or NaN in x spoils its column of dw, one in w its column of dx: as infinities where the sum has one
    sign, whatever the number of rows."""
    def spoil(x, w, dy, pre):
        x[T // 2, 5], x[0, K - 1], x[T - 1, 16] = INF, -INF, NAN
        w[1, 3], w[N // 2, 64], w[N - 1, K - 2] = INF, -INF, NAN
    got, want = gradients(kind, T, K, N, name, odt, spoil)
    for g, (r, b), what in zip(got, want, ("dx", "dw", "db")):
        check_special(g, r, b, f"{what} {name}")
    if name != "relu":     # (the case is what it says: one infinity in a column's sums leaves no NaN; relu's zeros do)
        assert not torch.isnan(want[0][0][:, 3]).any() and torch.isinf(want[0][0][:, 3]).all()
        assert not torch.isnan(want[1][0][:, 5]).any() and torch.isinf(want[1][0][:, 5]).all()


# ----------------------------------------------------------------------------- the norm's e4m3 codes

def rule(y):
    """moe_quantize_rows_fp8's rule on float32 values [T, H], evaluated on the host: (codes, scales)."""
    g = y.float().cpu().view(y.shape[0], -1, 128)
    amax = torch.where(torch.isnan(g), torch.zeros_like(g), g.abs()).amax(2, keepdim=True)
    s = amax / torch.tensor(448.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    v = g / s
    code = v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    code = torch.where(torch.isnan(v), torch.full_like(code, 0x7F), code)
    return code.view(y.shape).cuda(), s[:, :, 0].cuda()


@pytest.mark.parametrize("H", [256, 2176])
def test_norm_codes_of_groups_whose_scale_has_few_bits(H):
    """Channels so small beside their row's norm that amax / 448 keeps few of float32's bits, one bit or none: rounding
    the scale can put a value past 448 times it, which saturates, and a group whose scale would be zero has scale 1."""
    T = 150
    x, w = rnd("qx", (T, H), BF16, 2.0), torch.ones(H, dtype=BF16, device="cuda")
    x[:, :128] = rnd("qsmall", (T, 128), BF16) * 2.0 ** -4
    x[:, :128] *= (2.0 ** -(torch.arange(T, device="cuda") % 15)).to(BF16)[:, None]
    w[:128] = 2.0 ** -133                                 # bf16's smallest value
    x[7, :128], x[8, 3] = 0, 0
    q, s, _, h, rstd = m.rms_norm_fp8(x, w, 1e-6)
    y = (x.float().cpu() * rstd.cpu()[:, None]) * w.float().cpu()
    rq, rs = rule(y)
    few = (rs[:, 0] < 16 * 2.0 ** -149).sum().item()      # (the case is what it says)
    assert few > T // 4 and (rs[:, 0] == 1).sum().item() > T // 8
    assert same(s, rs) and same(q, rq)
    assert torch.isfinite(q.view(torch.float8_e4m3fn).float()).all()


def test_norm_codes_of_infinities_and_nan():
    """Rows of +-1 leave the weight itself as the norm's result: its codes are those of moe_quantize_rows_fp8, with
    infinities and NaN of either sign among them and in rows whose norm is not finite (a NaN's code is 0x7f or 0xff)."""
    def codes(q):
        return torch.where(q == 0xFF, 0x7F, q)
    T, H = 40, 512
    x = torch.where(rnd("ix", (T, H), F32) > 0, 1.0, -1.0).to(BF16)
    w = rnd("iw", (H,), BF16)
    w[5], w[130], w[131], w[300], w[301] = NAN, INF, 2.0, -NAN, -INF
    w[384:] = NAN
    q, s, y, *_ = m.rms_norm_fp8(x, w, 0.0, with_y=True)
    want, ws = m.quantize_rows_fp8((x * w).contiguous())
    assert same(s, ws) and same(codes(q), want)
    x[3, 9], x[4, 200], x[5, 500] = NAN, INF, -INF
    q, s, y, h, rstd = m.rms_norm_fp8(x, rnd("iw", (H,), BF16), 0.0, with_y=True)
    rq, rs = rule((x.float() * rstd[:, None]) * rnd("iw", (H,), BF16).float())
    assert same(s, rs) and same(codes(q), rq)
    assert not torch.isfinite(q[3].view(torch.float8_e4m3fn).float()).any()


# ----------------------------------------------------------------------------- activations

def relu(z):
    return torch.where(z <= 0, 0.0, z)


@pytest.mark.parametrize("T,K,N", [(3, 72, 41), (20, 2048, 264), (70, 200, 264), (300, 136, 521), (2100, 328, 1032)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", ref.ACTS)
def test_nan_rows_stay_nan(T, K, N, dtype, name):
    """A NaN in a row of x is in every output of that row, whatever the activation, and in no other row."""
    x, w, b = rnd("nx", (T, K), dtype), rnd("nw", (N, K), dtype, K ** -0.5), rnd("nb", (N,), dtype)
    clean = m.linear(x, w, b, act=ACT[name])[0]
    x[T // 2, K - 1] = NAN
    y, pre = m.linear(x, w, b, act=ACT[name], save_pre=True)
    rows = torch.arange(T, device="cuda") != T // 2
    assert torch.isnan(y[T // 2]).all() and torch.isnan(pre[T // 2]).all()
    assert torch.equal(y[rows], clean[rows])
    if name != "none" and N % 16 == 8:
        g = torch.cat([w, w])
        a, _ = m.gated_linear(x, g, act=ACT[name])
        assert torch.isnan(a[T // 2]).all() and torch.isfinite(a[rows]).all()


@pytest.mark.parametrize("dtype,odt", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("T,K,N", [(3, 72, 41), (40, 136, 264)])
def test_relu_gradient_of_special_values(T, K, N, dtype, odt):
    """dz is dy where pre > 0, 0 where pre <= 0 whatever dy is, and NaN where pre is NaN."""
    x, w = rnd("rx", (T, K), dtype), rnd("rw", (N, K), dtype, K ** -0.5)
    dy, pre = rnd("rdy", (T, N), odt), rnd("rz", (T, N), dtype)
    pre[0, 0], pre[0, 1], pre[0, 2], pre[1, 3], pre[1, 4] = -1.0, 0.0, -INF, 1.0, INF
    dy[0, 0], dy[0, 1], dy[0, 2], dy[1, 3] = INF, NAN, -INF, -INF
    dx, dw, db = m.linear_backward(dy, x, w, pre=pre, act=m.ACT_RELU, need_bias=True)
    dz = torch.where(pre.double() > 0, dy.double(), 0.0)
    for got, (r, b), what in zip((dx, dw, db), ref.backward(dz, torch.zeros_like(dz), x, w, dtype), ("dx", "dw", "db")):
        check_special(got, r, b, what)
    assert torch.isfinite(dx[0]).all() and torch.isfinite(dw[:3]).all() and not torch.isfinite(dx[1]).any()
    pre[2, 5] = NAN
    dx, dw, db = m.linear_backward(dy, x, w, pre=pre, act=m.ACT_RELU, need_bias=True)
    assert torch.isnan(dx[2]).all() and torch.isnan(dw[5]).all() and torch.isnan(db[5])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", [(3, 72, 40), (40, 136, 264)])
def test_gated_relu_gradient_of_special_values(T, H, I, dtype):
    x, w = rnd("gx", (T, H), dtype), rnd("gw", (2 * I, H), dtype, H ** -0.5)
    da, pre = rnd("gda", (T, I), dtype), rnd("gz", (T, 2 * I), dtype)
    pre[0, 0], pre[0, I] = -1.0, INF                 # up infinite behind a closed gate: no gradient for the gate
    pre[1, 1], pre[1, I + 1] = 2.0, -INF             # behind an open one an infinite one
    dx, dw, db = m.gated_linear_backward(da, x, w, pre, m.ACT_RELU, need_bias=True)
    g, u = pre.double().chunk(2, 1)
    dz = torch.cat([torch.where(g > 0, da.double() * u, 0.0), da.double() * relu(g)], 1)
    grads = ref.backward(dz, 4 * ref.U32 * dz.abs(), x, w, dtype, two_parts=T <= 32 and dtype is BF16)
    for got, (r, b), what in zip((dx, dw, db), grads, ("dx", "dw", "db")):
        check_special(got, r, b, what)
    assert torch.isfinite(dx[0]).all() and not torch.isfinite(dx[1]).any()


@pytest.mark.parametrize("T,N", [(3, 24), (20, 61), (200, 64), (333, 60), (2500, 1032)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_float32_outputs_have_float32_activations(name, T, N):
    """bf16 operands with a float32 output: each z is one bf16 value exactly, so the output's error is the
    activation's.  silu = z / (1 + exp(-z)): exp off by 2 u32 of itself, sum and quotient by one each: 4 u32.  gelu = z / 2
    erfc(-z / sqrt 2): an argument off by 2 u32 moves erfc by at most (z^2 + 1) times that, erfc is off by 8 u32 (4 units in the
    last place) and the products by 2."""
    z = torch.linspace(-24, 24, T * 8).view(8, T).t().contiguous() if T > 3 else torch.linspace(-9, 9, 24).view(3, 8)
    x = z.to(BF16).cuda()
    w = torch.zeros((N, 8), dtype=BF16, device="cuda")
    w[torch.arange(N), torch.arange(N) % 8] = 1
    y, _ = m.linear(x, w, act=ACT[name], out_dtype=F32)
    zd = x.double()[:, torch.arange(N) % 8]
    want = ref.act(name, zd) if name == "silu" else 0.5 * zd * torch.erfc(-zd * 0.5 ** 0.5)   # (erfc keeps the far tail)
    tol = 4.0 if name == "silu" else 12 + 2 * zd * zd
    ref.check(y, want, tol * ref.U32 * want.abs() + 2.0 ** -149, f"{name} of float32 outputs")
