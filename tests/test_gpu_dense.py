"""The dense operators around the routed experts (RMS norm, linear, gated projection) against
their 64-bit plain forms (dense_ref.py, whose bounds are derived there), forward and backward."""

import ctypes
import zlib

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACT = {"none": m.ACT_NONE, "silu": m.ACT_SILU, "gelu": m.ACT_GELU, "relu": m.ACT_RELU}
EPS = 1e-6


def rnd(name, shape, dtype, std=1.0, mean=0.0, pad=0):
    """Seeded normal values; pad > 0: rows inside a wider buffer whose other columns are NaN."""
    g = torch.Generator(device="cpu").manual_seed(zlib.crc32(repr((name, shape)).encode()))
    t = (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()
    if not pad:
        return t
    wide = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :shape[1]] = t
    return wide[:, :shape[1]]


# ----------------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 8), (3, 136), (16, 2048), (5, 2056), (130, 1024), (7, 4096), (33, 7168), (2, 8200), (3, 16384),
               (2, 65536), (1100, 512), (5000, 40)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm(T, H, residual, dtype):
    pad = 8 if T % 2 else 0
    x = rnd("x", (T, H), dtype, 2.0, pad=pad)
    w = rnd("w", (H,), dtype, 0.2, 1.0)
    res = rnd("res", (T, H), dtype, pad=2 * pad) if residual else None
    y, h, rstd = m.rms_norm(x, w, EPS, residual=res)
    (ry, by), rh, (rr, br), _ = ref.norm(x, w, EPS, res, dtype)
    assert torch.equal(h.double(), rh) and (residual or h is x)
    ref.check(rstd, rr, br, "rstd")
    ref.check(y, ry, by, "y")


@pytest.mark.parametrize("T,H", [(1, 128), (17, 2048), (9, 2176), (64, 7168), (3, 40960)])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_norm_fp8(T, H, residual):
    x = rnd("x", (T, H), BF16, 2.0)
    x[0, :min(H, 128)] = 0                    # a group of zeros: scale 1
    w = rnd("w", (H,), BF16, 0.2, 1.0)
    res = rnd("res", (T, H), BF16) if residual else None
    if residual:
        res[0, :min(H, 128)] = 0
    q, s, y, h, rstd = m.rms_norm_fp8(x, w, EPS, residual=res, with_y=True)
    (ry, by), rh, (rr, br), (fy, fe) = ref.norm(x, w, EPS, res, BF16)
    assert torch.equal(h.double(), rh)
    ref.check(rstd, rr, br, "rstd")
    ref.check(y, ry, by, "y")
    groups, eg = fy.view(T, -1, 128), fe.view(T, -1, 128)
    amax = groups.abs().amax(2)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    ref.check(s, want, eg.amax(2) / 448 + 2 * ref.U32 * want, "scale")
    # a code is the e4m3 value nearest to y / s: half a step is at most 2^-4 of it, or 2^-10 among the subnormal values
    val = q.view(torch.float8_e4m3fn).double().view(T, -1, 128)
    sd = s.double()[:, :, None]
    assert ((val * sd - groups).abs() <= (groups.abs() * 2.0 ** -4).clamp(min=2.0 ** -10 * sd) * (1 + 2.0 ** -20) + eg).all()
    assert (q.view(T, -1, 128)[0, 0] == 0).all() and s[0, 0] == 1
    q2, s2, y2, _, _ = m.rms_norm_fp8(x, w, EPS, residual=res)
    assert y2 is None and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("exponent", [-122, -110, 0, 110])
def test_norm_fp8_far_scales(exponent):
    """Weights that put the scales below, inside and above the range of a float32 reciprocal: the
    codes are those of the values at exponent 0, whose scales differ by the power of two alone."""
    x, w = rnd("fx", (9, 256), BF16), rnd("fw", (256,), BF16, 0.2, 1.0)
    q0, s0, *_ = m.rms_norm_fp8(x, w, EPS)
    q, s, *_ = m.rms_norm_fp8(x, (w.double() * 2.0 ** exponent).to(BF16), EPS)
    assert torch.equal(s.double(), (s0.double() * 2.0 ** exponent).float().double())
    if exponent > -122:                  # (there the scale has lost bits below the smallest normal value)
        assert torch.equal(q, q0)
    else:
        v, v0 = (t.view(torch.float8_e4m3fn).double() for t in (q, q0))
        assert torch.isfinite(v).all() and ((v - v0).abs() <= 2.0 ** -3 * v0.abs() + 2.0 ** -9).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("with_dh", [False, True], ids=["plain", "dh"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm_backward(T, H, with_dh, dtype):
    pad = 8 if T % 2 else 0
    h = rnd("h", (T, H), dtype, 2.0, pad=pad)
    w = rnd("w", (H,), dtype, 0.2, 1.0)
    dy = rnd("dy", (T, H), dtype, pad=pad)
    dh = rnd("dh", (T, H), dtype) if with_dh else None
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dx, dw = m.rms_norm_backward(dy, h, w, rstd, dh=dh)
    (rx, bx), (rw, bw) = ref.norm_backward(dy, h, w, rstd, dh, dtype)
    ref.check(dx, rx, bx, "dx")
    ref.check(dw, rw, bw, "dweight")


# ----------------------------------------------------------------------------- linear

# (T, K, N): single tokens, few tokens, every tile shape, ragged in each direction, long contractions
LINEAR_SHAPES = [(1, 8, 1), (1, 2048, 60), (2, 72, 16), (16, 1408, 2048), (17, 520, 257), (31, 7168, 256), (33, 64, 8),
                 (64, 264, 136), (65, 1032, 100), (127, 128, 384), (129, 2048, 60), (200, 4104, 520), (300, 136, 1000),
                 (512, 1000, 640), (700, 2048, 2050), (1111, 328, 2304), (2100, 512, 1030), (3000, 200, 24),
                 (4097, 64, 264)]


def linear_case(T, K, N, dtype, odt, bias, residual, pad=0):
    x = rnd("x", (T, K), dtype, pad=8 * pad)
    w = rnd("w", (N, K), dtype, K ** -0.5)
    b = rnd("b", (N,), dtype, 0.5) if bias else None
    r = rnd("r", (T, N), odt, pad=8 * pad) if residual else None
    return x, w, b, r


@pytest.mark.parametrize("dtype,odt", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("T,K,N", LINEAR_SHAPES)
def test_linear(T, K, N, dtype, odt):
    i = (T + N) % 4
    bias, residual, name = i != 0, i != 1, ref.ACTS[i]
    x, w, b, r = linear_case(T, K, N, dtype, odt, bias, residual, pad=T % 3)
    y, pre = m.linear(x, w, b, r, ACT[name], odt, save_pre=i >= 2)
    (ry, by), (rz, bz) = ref.linear(x, w, b, r, name, dtype, odt)
    ref.check(y, ry, by, "y")
    if i >= 2:
        ref.check(pre, rz, bz, "pre")
    else:
        assert pre is None


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("T", [3, 200, 1300])
def test_linear_every_epilogue(T, name):
    for bias in (False, True):
        for residual in (False, True):
            x, w, b, r = linear_case(T, 256, 264, BF16, BF16, bias, residual)
            y, pre = m.linear(x, w, b, r, ACT[name], save_pre=True)
            (ry, by), (rz, bz) = ref.linear(x, w, b, r, name, BF16, BF16)
            ref.check(y, ry, by, f"y bias={bias} residual={residual}")
            ref.check(pre, rz, bz, f"pre bias={bias} residual={residual}")


BACKWARD_SHAPES = [(1, 8, 1), (1, 2048, 60), (2, 72, 16), (16, 1408, 2048), (17, 520, 257), (33, 64, 8), (64, 264, 136),
                   (65, 1032, 100), (129, 2048, 60), (200, 4104, 520), (300, 136, 1000), (700, 2048, 2050),
                   (1111, 328, 2304), (2100, 512, 1030), (3000, 200, 24), (4097, 64, 264)]


@pytest.mark.parametrize("dtype,odt", [(BF16, BF16), (BF16, F32), (F32, F32)], ids=["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("T,K,N", BACKWARD_SHAPES)
def test_linear_backward(T, K, N, dtype, odt):
    i = (T + N) % 4
    name, bias = ref.ACTS[i], T % 2 == 1
    x = rnd("x", (T, K), dtype, pad=8 * (T % 3))
    w = rnd("w", (N, K), dtype, K ** -0.5)
    pre = rnd("z", (T, N), dtype, 1.5, pad=8 * (T % 2)) if i else None
    dy = rnd("dy", (T, N), odt, pad=8 * (T % 2))
    dx, dw, db = m.linear_backward(dy, x, w, pre=pre, act=ACT[name], need_bias=bias)
    grads = ref.backward(*ref.dz_linear(dy, pre, name), x, w, dtype)
    for got, (r, b), what in zip((dx, dw, db), grads, ("dx", "dw", "db")):
        if got is None:
            assert what == "db" and not bias
        else:
            ref.check(got, r, b, what)


# ----------------------------------------------------------------------------- gated

GATED_SHAPES = [(1, 8, 8), (1, 2048, 1408), (3, 72, 40), (16, 2048, 360), (40, 1032, 264), (64, 512, 128), (100, 136, 200),
                (130, 2048, 1408), (513, 264, 520), (1025, 640, 1032), (2100, 328, 136)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", GATED_SHAPES)
def test_gated(T, H, I, dtype):
    name, bias, save = ref.ACTS[1 + T % 3], I % 16 == 8, T % 4 != 1
    x = rnd("x", (T, H), dtype, pad=8 * (T % 2))
    w = rnd("w", (2 * I, H), dtype, H ** -0.5)
    b = rnd("b", (2 * I,), dtype, 0.5) if bias else None
    a, pre = m.gated_linear(x, w, b, ACT[name], save_pre=save)
    (ra, ba), (rz, bz) = ref.gated(x, w, b, name, dtype)
    ref.check(a, ra, ba, "a")
    if save:
        ref.check(pre, rz, bz, "pre")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", GATED_SHAPES)
def test_gated_backward(T, H, I, dtype):
    name, bias = ref.ACTS[1 + T % 3], T % 2 == 1
    x = rnd("x", (T, H), dtype, pad=8 * (T % 2))
    w = rnd("w", (2 * I, H), dtype, H ** -0.5)
    pre = rnd("z", (T, 2 * I), dtype, 1.5, pad=8 * (T % 2))
    da = rnd("da", (T, I), dtype, pad=8 * (T % 3))
    dx, dw, db = m.gated_linear_backward(da, x, w, pre, ACT[name], need_bias=bias)
    grads = ref.backward(*ref.dz_gated(da, pre, name), x, w, dtype)
    for got, (r, b), what in zip((dx, dw, db), grads, ("dx", "dw", "db")):
        if got is None:
            assert what == "db" and not bias
        else:
            ref.check(got, r, b, what)


# ----------------------------------------------------------------------------- gradients against differences

def directional(f, args, k, direction, step=1e-6):
    up, down = list(args), list(args)
    up[k], down[k] = args[k] + step * direction, args[k] - step * direction
    return ((f(*up) - f(*down)) / (2 * step)).item()


@pytest.mark.parametrize("name", ref.ACTS[:3])
def test_gradients_match_differences(name):
    """float32 kernels' gradients along random directions against central differences of the
    64-bit forward: off by the float32 bounds (1e-5 of the norms covers 40-long sums) and the
    differences' own step^2."""
    T, K, N = 11, 40, 32
    x, w, b = rnd("x", (T, K), F32), rnd("w", (N, K), F32, 0.2), rnd("b", (N,), F32)
    dy = rnd("dy", (T, N), F32)
    args = [t.double() for t in (x, w, b)]

    def lin(x, w, b):
        return (dy.double() * ref.act(name, x @ w.t() + b)).sum()

    _, pre = m.linear(x, w, b, act=ACT[name], save_pre=True)
    grads = m.linear_backward(dy, x, w, pre=pre, act=ACT[name], need_bias=True)
    for k, g in enumerate(grads):
        v = rnd(f"v{k}", tuple(g.shape), F32).double()
        assert abs(directional(lin, args, k, v) - (g.double() * v).sum().item()) <= 1e-5 * (g.norm() * v.norm()).item()

    if name == "none":
        nw, nx = rnd("nw", (K,), F32, 0.2, 1.0), x
        ndy, dh = rnd("ndy", (T, K), F32), rnd("dh", (T, K), F32)

        def nrm(x, w):
            return (ndy.double() * (x * (x.square().mean(1, keepdim=True) + EPS) ** -0.5 * w) + dh.double() * x).sum()

        _, h, rstd = m.rms_norm(nx, nw, EPS)
        for k, g in enumerate(m.rms_norm_backward(ndy, h, nw, rstd, dh=dh)):
            v = rnd(f"nv{k}", tuple(g.shape), F32).double()
            diff = directional(nrm, [nx.double(), nw.double()], k, v)
            assert abs(diff - (g.double() * v).sum().item()) <= 1e-5 * (g.norm() * v.norm()).item()
        return

    def gat(x, w, b):
        g, u = (x @ w.t() + b).chunk(2, 1)
        return (dy[:, :N // 2].double().contiguous() * ref.act(name, g) * u).sum()

    da = dy[:, :N // 2].contiguous()
    _, pre = m.gated_linear(x, w, b[:N].contiguous(), ACT[name], save_pre=True)
    for k, g in enumerate(m.gated_linear_backward(da, x, w, pre, ACT[name], need_bias=True)):
        v = rnd(f"gv{k}", tuple(g.shape), F32).double()
        assert abs(directional(gat, args, k, v) - (g.double() * v).sum().item()) <= 1e-5 * (g.norm() * v.norm()).item()


# ----------------------------------------------------------------------------- the largest tiles

def test_large_linear():
    T, K, N = 4000, 7176, 4096          # 256 tiles of 256 x 256, a contraction that ends 8 into a slice
    x, w, b, r = linear_case(T, K, N, BF16, BF16, True, True, pad=1)
    y, pre = m.linear(x, w, b, r, m.ACT_GELU, save_pre=True)
    (ry, by), (rz, bz) = ref.linear(x, w, b, r, "gelu", BF16, BF16)
    ref.check(y, ry, by, "y")
    ref.check(pre, rz, bz, "pre")


def test_large_gated():
    T, H, I = 3999, 7176, 2040
    x, w = rnd("bx", (T, H), BF16, pad=8), rnd("bw", (2 * I, H), BF16, H ** -0.5)
    b = rnd("bb", (2 * I,), BF16, 0.5)
    a, pre = m.gated_linear(x, w, b, save_pre=True)
    (ra, ba), (rz, bz) = ref.gated(x, w, b, "silu", BF16)
    ref.check(a, ra, ba, "a")
    ref.check(pre, rz, bz, "pre")


def test_large_gradients():
    T, K, N = 8187, 7168, 4104          # both gradients in 256 x 256 tiles, both contractions ragged
    x, w = rnd("lx", (T, K), BF16), rnd("lw", (N, K), BF16, K ** -0.5)
    dy = rnd("ldy", (T, N), BF16)
    dx, dw, db = m.linear_backward(dy, x, w, need_bias=True)
    grads = ref.backward(*ref.dz_linear(dy, None, "none"), x, w, BF16)
    for got, (r, b), what in zip((dx, dw, db), grads, ("dx", "dw", "db")):
        ref.check(got, r, b, what)


# Three whole rounds of 256 x 256 tiles and less than half a round, which runs as halves; the last tile row's
# lower halves have no rows, and the contraction ends 8 into a slice.

def test_half_tiles_linear():
    T, K, N = 7700, 2056, 7168
    x, w, b, r = linear_case(T, K, N, BF16, BF16, True, True, pad=1)
    y, pre = m.linear(x, w, b, r, m.ACT_RELU, save_pre=True)
    (ry, by), (rz, bz) = ref.linear(x, w, b, r, "relu", BF16, BF16)
    ref.check(y, ry, by, "y")
    ref.check(pre, rz, bz, "pre")


def test_half_tiles_gated():
    T, H, I = 3900, 2056, 7168
    x, w = rnd("hx", (T, H), BF16, pad=8), rnd("hw", (2 * I, H), BF16, H ** -0.5)
    b = rnd("hb", (2 * I,), BF16, 0.5)
    a, pre = m.gated_linear(x, w, b, save_pre=True)
    (ra, ba), (rz, bz) = ref.gated(x, w, b, "silu", BF16)
    ref.check(a, ra, ba, "a")
    ref.check(pre, rz, bz, "pre")


# ----------------------------------------------------------------------------- few rows: dz in two bf16 parts

@pytest.mark.parametrize("need", ["dx", "dw", "both"])
@pytest.mark.parametrize("T,K,N", [(1, 8, 1), (2, 2048, 104), (3, 520, 257), (7, 1032, 2056), (8, 4104, 40), (16, 1408, 2048),
                                   (32, 2048, 520)])
def test_few_rows_gradients_keep_dz(T, K, N, need):
    x, w = rnd("fx", (T, K), BF16, pad=8 * (T % 2)), rnd("fw", (N, K), BF16, K ** -0.5)
    for name, odt in (("silu", BF16), ("gelu", F32), ("none", F32)):
        dy, pre = rnd("fdy", (T, N), odt), rnd("fz", (T, N), BF16, 1.5) if name != "none" else None
        grads = ref.backward(*ref.dz_linear(dy, pre, name), x, w, BF16, two_parts=True)
        prob = m.LinearProblem(T, K, N, m.BF16, m.F32 if odt is F32 else m.BF16, ACT[name], x.stride(0), 0, 0, 0, 0)
        n = ctypes.c_size_t(0)
        assert m.lib().moe_linear_workspace_size(ctypes.byref(prob), 1, ctypes.byref(n)) == 0
        ws = torch.full((n.value,), 255, dtype=torch.uint8, device="cuda")      # NaN in every type
        dx = torch.empty((T, K), dtype=BF16, device="cuda") if need != "dw" else None
        dw = torch.empty((N, K), dtype=BF16, device="cuda") if need != "dx" else None
        at = lambda t: None if t is None else t.data_ptr()          # noqa: E731
        assert m.lib().moe_linear_backward(
            ctypes.byref(prob), dy.data_ptr(), x.data_ptr(), w.data_ptr(), at(pre), at(dx), at(dw), None, ws.data_ptr(),
            n.value, torch.cuda.current_stream().cuda_stream) == 0
        for got, (r, b), what in zip((dx, dw), grads, ("dx", "dw")):
            if got is not None:
                ref.check(got, r, b, f"{what} {name}")


@pytest.mark.parametrize("T,H,I", [(1, 64, 8), (2, 4760, 104), (9, 136, 1408), (32, 2048, 360)])
def test_few_rows_gated_gradients_keep_dz(T, H, I):
    x, w = rnd("gx", (T, H), BF16), rnd("gw", (2 * I, H), BF16, H ** -0.5)
    da, pre = rnd("gda", (T, I), BF16), rnd("gz", (T, 2 * I), BF16, 1.5)
    dx, dw, db = m.gated_linear_backward(da, x, w, pre, need_bias=True)
    grads = ref.backward(*ref.dz_gated(da, pre, "silu"), x, w, BF16, two_parts=True)
    for got, (r, b), what in zip((dx, dw, db), grads, ("dx", "dw", "db")):
        ref.check(got, r, b, what)


def test_few_rows_infinite_dz():
    """A dz that bf16 cannot hold is infinite, as with many rows, and no NaN comes of its second part."""
    T, K, N = 3, 64, 40
    x, w = torch.ones((T, K), dtype=BF16, device="cuda"), torch.ones((N, K), dtype=BF16, device="cuda")
    dy = torch.ones((T, N), dtype=F32, device="cuda")
    dy[1, 2] = 3.4e38          # finite in float32, past bf16's largest value
    dx, dw, _ = m.linear_backward(dy, x, w)
    assert torch.isposinf(dx[1]).all() and torch.isposinf(dw[2]).all()
    assert (dx[[0, 2]] == N).all() and (dw[[0, 1, 3, 39]] == T).all()
