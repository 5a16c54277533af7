"""The e4m3 products with block scales (moe_linear_fp8, moe_gated_linear_fp8), for one matrix and by expert, their gradients
and the weights' quantiser, against plain 64-bit forms on the same codes."""

import pytest
import torch

import fp8_ref as ref
import mixture_experts_routed_topk_amd as m

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ACT = {"none": m.ACT_NONE, "silu": m.ACT_SILU, "gelu": m.ACT_GELU, "relu": m.ACT_RELU}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(seed, shape, dtype=BF16, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def weights(seed, shape, ue8m0):
    return m.quantize_blocks_fp8(rnd(seed, shape, BF16, shape[-1] ** -0.5), ue8m0)


def rows(seed, T, K):
    x = rnd(seed, (T, K))
    x[:, seed % K] *= 30.0
    return m.quantize_rows_fp8(x) if T else (torch.empty((0, K), dtype=torch.uint8, device="cuda"),
                                             torch.empty((0, K // 128), device="cuda"))


def runs(seed, T, E, end=None):
    """Offsets of E runs over `end` of T rows, one of them empty where there are more than two."""
    share = torch.rand(E, generator=gen(seed), device="cuda") + 0.1
    if E > 2:
        share[E // 2] = 0.0
    ends = (torch.cumsum(share, 0) / share.sum() * (T if end is None else end)).round().to(torch.int32)
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), ends])


# ----------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(128, 128), (384, 256), (3, 256, 640), (1, 128, 65536), (65536, 128)])
def test_blocks_follow_the_rule_exactly(shape, dtype, ue8m0):
    w = rnd(1, shape, dtype)
    w.view(-1, shape[-1])[:128, :128] = 0.0                        # a block of zeros
    q, s = m.quantize_blocks_fp8(w, ue8m0)
    rq, rs = ref.block_groups(w, ue8m0)
    assert torch.equal(ref.scale_values(s), rs)
    if ue8m0:
        assert torch.equal(q.view(ref.E4M3).double(), rq)
    else:                                                          # the quotient is rounded to float32 before it is to e4m3
        g = w.double().view(*shape[:-2], shape[-2] // 128, 128, shape[-1] // 128, 128)
        quotient = (g / rs[..., :, None, :, None]).float()
        assert torch.equal(q.view(ref.E4M3).float(), quotient.to(ref.E4M3).float().view(shape))


def test_blocks_at_the_ends_of_the_range():
    tiny, huge = 2.0 ** -149, 3.0e38
    w = torch.zeros((128, 128 * 7), device="cuda")
    for b, v in enumerate((tiny, 5 * tiny, 2.0 ** -126, 448.0, 449.0, huge)):
        w[3, 128 * b + 5] = v
        w[4, 128 * b + 6] = -v / 2
    w[9, 128 * 6 + 1] = float("nan")
    w[10, 128 * 6 + 2] = 7.0
    q, s = m.quantize_blocks_fp8(w)
    v = ref.wide(q, s)
    assert v.isfinite().sum() == w.numel() - 1 and torch.isnan(v[9, 128 * 6 + 1]) and v[10, 128 * 6 + 2] == 7.0
    for b in (2, 3, 4, 5):
        # the largest lies on code 448, off by its scale's rounding: half a step, which below 2^-126 is 2^-150 (2^-126 / 448 has 15 bits)
        top = w[3, 128 * b + 5].item()
        assert abs(v[3, 128 * b + 5].item() / top - 1) <= max(2.0 ** -24, 2.0 ** -150 / (top / 448)) * 1.001
    q, s = m.quantize_blocks_fp8(w, ue8m0=True)
    assert s[0].tolist()[:6] == [1, 1, 1, 127, 128, 127 + 120]   # 3e38 = 1.763 * 2^127 passes 1.75 * 2^127
    v = ref.wide(q, s)
    assert v.isfinite().sum() == w.numel() - 1
    assert v[3, 128 * 3 + 5] == 448.0 and v[3, 128 * 4 + 5] == 448.0


# ----------------------------------------------------------------------------- forward

DENSE = [  # T, K, N
    (1, 128, 128), (2, 7168, 256), (16, 256, 384), (17, 4224, 128), (32, 2048, 384), (33, 128, 640), (40, 7168, 256), (127, 384, 256),
    (128, 1408, 512), (129, 256, 384), (257, 640, 896), (520, 1152, 1408), (2100, 512, 2048)]


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", DENSE)
def test_linear(T, K, N, ue8m0):
    q, s = rows(2, T, K)
    wq, ws = weights(3, (N, K), ue8m0)
    x, w = ref.wide_rows(q, s), ref.wide(wq, ws)
    y, pre = m.linear_fp8(q, s, wq, ws)
    assert pre is None
    ref.check(y, *ref.linear(x, w, None, None, "none")[0], "y")
    name = ("silu", "gelu", "relu")[(T + N) % 3]
    bias, res = rnd(4, (N,)), rnd(5, (T, N + 8))[:, :N]
    out = torch.empty((T, N + 16), dtype=BF16, device="cuda")[:, :N]
    wide_q = torch.zeros((T, K + 32), dtype=torch.uint8, device="cuda")
    wide_q[:, :K] = q
    got, pre = m.linear_fp8(wide_q[:, :K], s, wq.view(ref.E4M3), ws, bias=bias, residual=res, act=ACT[name], save_pre=True, out=out)
    want, wpre = ref.linear(x, w, bias, res, name)
    assert got is out
    ref.check(got, *want, f"{name} y")
    ref.check(pre, *wpre, f"{name} pre")


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", DENSE)
def test_gated(T, K, N, ue8m0):
    q, s = rows(6, T, K)
    wq, ws = weights(7, (2 * N, K), ue8m0)
    name = ("silu", "gelu", "relu")[(T + K // 128) % 3]
    a, pre = m.gated_linear_fp8(q, s, wq, ws, act=ACT[name], save_pre=True)
    want, wpre = ref.gated(ref.wide_rows(q, s), ref.wide(wq, ws), name)
    ref.check(a, *want, f"{name} a")
    ref.check(pre, *wpre, "pre")
    out = torch.empty((T, N + 8), dtype=BF16, device="cuda")[:, :N]
    b, none = m.gated_linear_fp8(q, s, wq, ws, act=ACT[name], out=out)
    assert b is out and none is None and torch.equal(b, a)


GROUPED = [  # T, K, N, E, rows that belong to experts
    (1, 128, 128, 1, 1), (7, 256, 128, 5, 7), (64, 384, 256, 64, 64), (300, 256, 384, 3, 290), (1000, 384, 256, 4, 1000),
    (1500, 256, 640, 3, 1490), (700, 128, 128, 1024, 650), (900, 512, 256, 1, 900)]


def by_expert(off):
    o = off.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N,E,end", GROUPED)
def test_experts(T, K, N, E, end, ue8m0):
    q, s = rows(8, T, K)
    off = runs(9, T, E, end)
    wq, ws = weights(10, (E, N, K), ue8m0)
    gq, gs = weights(11, (E, 2 * N, K), ue8m0)
    y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    a = torch.full((T, N), 6.0, dtype=BF16, device="cuda")
    assert m.linear_fp8(q, s, wq, ws, offsets=off, out=y)[0] is y
    _, pre = m.gated_linear_fp8(q, s, gq, gs, act=m.ACT_GELU, save_pre=True, offsets=off, out=a)
    last = int(off[-1])
    assert (y[last:] == 5.0).all() and (a[last:] == 6.0).all()
    for e, lo, hi in by_expert(off):
        x = ref.wide_rows(q[lo:hi], s[lo:hi])
        ref.check(y[lo:hi], *ref.linear(x, ref.wide(wq[e], ws[e]), None, None, "none")[0], f"expert {e}")
        want, wpre = ref.gated(x, ref.wide(gq[e], gs[e]), "gelu")
        ref.check(a[lo:hi], *want, f"expert {e} a")
        ref.check(pre[lo:hi], *wpre, f"expert {e} pre")


def test_offsets_that_do_not_fit_lead_nowhere():
    """Offsets outside [0, T] are taken into it, and ones that fall back do not lower a run: rows keep one owner."""
    T, K, N, E = 300, 256, 128, 4
    q, s = rows(12, T, K)
    wq, ws = weights(13, (E, N, K), False)
    bad = torch.tensor([-5, 100, 40, 2 ** 31 - 1, 7], dtype=torch.int32, device="cuda")
    good = torch.tensor([0, 100, 100, 300, 300], dtype=torch.int32, device="cuda")
    a, b = (m.linear_fp8(q, s, wq, ws, offsets=o)[0] for o in (bad, good))
    assert torch.equal(a, b)
    x, dy = rnd(14, (T, K)), rnd(15, (T, N))
    for u, v in zip(m.linear_fp8_backward(dy, x, wq, ws, offsets=bad)[:2], m.linear_fp8_backward(dy, x, wq, ws, offsets=good)[:2]):
        assert torch.equal(u, v)
    from_10 = torch.tensor([10, 10, 200, 250, 260], dtype=torch.int32, device="cuda")
    out = torch.full((T, N), 3.0, dtype=BF16, device="cuda")
    m.linear_fp8(q, s, wq, ws, offsets=from_10, out=out)
    assert (out[:10] == 3.0).all() and (out[260:] == 3.0).all() and not (out[10:260] == 3.0).all(1).any()


# ----------------------------------------------------------------------------- gradients

@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (31, 256, 384), (128, 384, 256), (129, 1152, 128), (300, 640, 896), (1100, 512, 1408), (5000, 256, 128)])
def test_linear_backward(T, K, N, ue8m0):
    wq, ws = weights(16, (N, K), ue8m0)
    w = ref.wide(wq, ws)
    x = rnd(17, (T, K + 16))[:, :K]
    dy = rnd(18, (T, N + 8), BF16, 1e-3)[:, :N]
    for name in ("none", ("silu", "gelu", "relu")[T % 3]):
        pre = rnd(19, (T, N)) if name != "none" else None
        out = torch.empty((T, K + 8), dtype=BF16, device="cuda")[:, :K]
        got = m.linear_fp8_backward(dy, x, wq, ws, pre=pre, act=ACT[name], need_bias=True, out=out)
        assert got[0] is out
        want = ref.backward(*ref.dz_linear(dy, pre, name), x, w, bias=True)
        for g, (r, b), what in zip(got, want, ("dx", "dw", "db")):
            ref.check(g, r, b, f"{name} {what}")
        assert m.linear_fp8_backward(dy, x, wq, ws, pre=pre, act=ACT[name])[2] is None


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (100, 384, 256), (300, 640, 384), (1030, 256, 1024)])
def test_gated_backward(T, K, N, ue8m0):
    wq, ws = weights(20, (2 * N, K), ue8m0)
    x, da, pre = rnd(21, (T, K)), rnd(22, (T, N), BF16, 1e-3), rnd(23, (T, 2 * N))
    for name in ("silu", "gelu", "relu"):
        got = m.gated_linear_fp8_backward(da, x, wq, ws, pre, act=ACT[name])
        want = ref.backward(*ref.dz_gated(da, pre, name), x, ref.wide(wq, ws))
        for g, (r, b), what in zip(got, want, ("dx", "dw")):
            ref.check(g, r, b, f"{name} {what}")


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N,E,end", GROUPED)
def test_experts_backward(T, K, N, E, end, ue8m0):
    off = runs(24, T, E, end)
    wq, ws = weights(25, (E, N, K), ue8m0)
    gq, gs = weights(26, (E, 2 * N, K), ue8m0)
    x, dy, pre = rnd(27, (T, K)), rnd(28, (T, N), BF16, 1e-3), rnd(29, (T, 2 * N))
    out = torch.full((T, K), 4.0, dtype=BF16, device="cuda")
    dx, dw, _ = m.linear_fp8_backward(dy, x, wq, ws, offsets=off, out=out)
    gx, gw = m.gated_linear_fp8_backward(dy, x, gq, gs, pre, act=m.ACT_SILU, offsets=off)
    assert (dx[int(off[-1]):] == 4.0).all()
    some = by_expert(off)
    for e in range(E):
        if e not in {r[0] for r in some}:
            assert (dw[e] == 0).all() and (gw[e] == 0).all()
    for e, lo, hi in some:
        for got, want in (((dx, dw), ref.backward(*ref.dz_linear(dy[lo:hi], None, "none"), x[lo:hi], ref.wide(wq[e], ws[e]))),
                          ((gx, gw), ref.backward(*ref.dz_gated(dy[lo:hi], pre[lo:hi], "silu"), x[lo:hi], ref.wide(gq[e], gs[e])))):
            ref.check(got[0][lo:hi], *want[0], f"expert {e} dx")
            ref.check(got[1][e], *want[1], f"expert {e} dw")


@pytest.mark.parametrize("E", [0, 3])
def test_gradients_against_differences(E):
    """Small whole numbers are e4m3 values and their sums float32 and bf16 ones: every step is exact, and <dy, y>, linear in x and in
    w, changes by exactly the gradient."""
    T, K, N = 200, 128, 128
    shape = (E, N, K) if E else (N, K)

    def whole(seed, shape, top):
        return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda").float()
    x, w, dy = whole(30, (T, K), 1), whole(31, shape, 1), whole(32, (T, N), 1)
    step_x, step_w = whole(33, (T, K), 1), whole(34, shape, 1)
    off = runs(35, T, E) if E else None
    one = torch.full(shape[:-2] + (N // 128, K // 128), 127, dtype=torch.uint8, device="cuda")

    def f(x, w):
        y, _ = m.linear_fp8(x.to(ref.E4M3), torch.ones((T, 1), device="cuda"), w.to(ref.E4M3), one, offsets=off)
        return (y.double() * dy.double()).sum().item()
    dx, dw, _ = m.linear_fp8_backward(dy.to(BF16), x.to(BF16), w.to(ref.E4M3), one, offsets=off)
    assert (f(x + step_x, w) - f(x - step_x, w)) / 2 == (dx.double() * step_x).sum().item()
    assert (f(x, w + step_w) - f(x, w - step_w)) / 2 == (dw.double() * step_w).sum().item()


def test_each_subset_of_the_gradients():
    import ctypes
    T, K, N = 300, 256, 384
    wq, ws = weights(36, (N, K), True)
    x, dy = rnd(37, (T, K)), rnd(38, (T, N))
    want = m.linear_fp8_backward(dy, x, wq, ws, need_bias=True)
    p = m.Fp8Problem(T, K, N, 0, m.SCALE_UE8M0, m.ACT_NONE, 0, 0, 0, 0, 0)
    n = ctypes.c_size_t(0)
    assert m.lib().moe_linear_fp8_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == 0
    w = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for which in range(8):
        got = [torch.full_like(t, 2.0) for t in want]
        at = [g.data_ptr() if which >> i & 1 else None for i, g in enumerate(got)]
        assert m.lib().moe_linear_fp8_backward(ctypes.byref(p), dy.data_ptr(), x.data_ptr() if which & 2 else None,
                                               wq.data_ptr() if which & 1 else None, ws.data_ptr() if which & 1 else None, None,
                                               None, *at, w.data_ptr(), n.value, stream) == 0
        torch.cuda.synchronize()
        for i in range(3):
            assert torch.equal(got[i], want[i] if which >> i & 1 else torch.full_like(want[i], 2.0)), (which, i)


# ----------------------------------------------------------------------------- special values

def test_values_that_are_not_finite_reach_what_they_enter():
    T, K, N = 300, 256, 256
    q, s = rows(39, T, K)
    wq, ws = weights(40, (N, K), False)
    clean, _ = m.linear_fp8(q, s, wq, ws)
    q2 = q.clone()
    q2[7, 3] = 0x7F                                       # a NaN code: its row alone
    y, _ = m.linear_fp8(q2, s, wq, ws)
    assert torch.isnan(y[7]).all()
    y[7] = clean[7]
    assert torch.equal(y, clean)
    w2 = wq.clone()
    w2[5, 200] = 0xFF                                     # in a weight: its column alone
    y, _ = m.linear_fp8(q, s, w2, ws)
    assert torch.isnan(y[:, 5]).all()
    y[:, 5] = clean[:, 5]
    assert torch.equal(y, clean)
    x, dy = rnd(41, (T, K)), rnd(42, (T, N))
    dx0, dw0, _ = m.linear_fp8_backward(dy, x, wq, ws)
    for v in (float("inf"), float("nan")):
        bad = dy.clone()
        bad[140, 9] = v                                   # its row of dx, its row of dw
        dx, dw, db = m.linear_fp8_backward(bad, x, wq, ws, need_bias=True)
        assert torch.isnan(dx[140]).all() and torch.isnan(dw[9]).all() and not torch.isfinite(db[9])
        dx[140], dw[9] = dx0[140], dw0[9]
        assert torch.equal(dx, dx0) and torch.equal(dw, dw0)
        bad = x.clone()
        bad[250, 17] = v                                  # x: its column of dw
        dx, dw, _ = m.linear_fp8_backward(dy, bad, wq, ws)
        assert torch.equal(dx, dx0) and torch.isnan(dw[:, 17]).all()
        dw[:, 17] = dw0[:, 17]
        assert torch.equal(dw, dw0)
    # behind a closed ReLU nothing arrives, whatever dy holds
    pre = rnd(43, (T, N))
    pre[140, 9] = -1.0
    bad = dy.clone()
    bad[140, 9] = float("inf")
    dx, dw, db = m.linear_fp8_backward(bad, x, wq, ws, pre=pre, act=m.ACT_RELU, need_bias=True)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()


def test_weights_that_are_nan_in_another_expert_do_not_matter():
    T, K, N, E = 200, 256, 128, 3
    q, s = rows(44, T, K)
    wq, ws = weights(45, (E, N, K), False)
    off = torch.tensor([0, 90, 90, 200], dtype=torch.int32, device="cuda")
    want, _ = m.linear_fp8(q, s, wq, ws, offsets=off)
    x, dy = rnd(46, (T, K)), rnd(47, (T, N))
    grads = m.linear_fp8_backward(dy, x, wq, ws, offsets=off)
    wq[1], ws[1] = 0x7F, float("nan")                     # the expert without rows
    assert torch.equal(m.linear_fp8(q, s, wq, ws, offsets=off)[0], want)
    for a, b in zip(m.linear_fp8_backward(dy, x, wq, ws, offsets=off)[:2], grads[:2]):
        assert torch.equal(a, b)
    # rows behind the last run, and a neighbour's, are not looked at
    off = torch.tensor([0, 90, 90, 150], dtype=torch.int32, device="cuda")
    dx, dw, _ = m.linear_fp8_backward(dy, x, wq, ws, offsets=off, out=torch.zeros_like(x))
    x2, dy2 = x.clone(), dy.clone()
    x2[150:], dy2[150:] = float("nan"), float("inf")
    dx2, dw2, _ = m.linear_fp8_backward(dy2, x2, wq, ws, offsets=off, out=torch.zeros_like(x))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("E", [0, 5])
def test_no_rows(E):
    K, N = 256, 128
    wq, ws = weights(48, (E, N, K) if E else (N, K), False)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda") if E else None
    q, s = rows(49, 0, K)
    assert m.linear_fp8(q, s, wq, ws, offsets=off)[0].shape == (0, N)
    none = torch.empty((0, K), dtype=BF16, device="cuda")
    dx, dw, db = m.linear_fp8_backward(torch.empty((0, N), dtype=BF16, device="cuda"), none, wq, ws, need_bias=not E, offsets=off)
    assert dx.shape == (0, K) and dw.shape == wq.shape and (dw == 0).all() and (E or (db == 0).all())
    if E:                                                 # rows, but none in a run
        q, s = rows(50, 40, K)
        out = torch.full((40, N), 2.0, dtype=BF16, device="cuda")
        m.linear_fp8(q, s, wq, ws, offsets=off, out=out)
        assert (out == 2.0).all()
        _, dw, _ = m.linear_fp8_backward(rnd(51, (40, N)), rnd(52, (40, K)), wq, ws, offsets=off)
        assert (dw == 0).all()


def test_matrices_past_32_bits():
    E, N, K = 40, 8192, 16384                             # 5.4 GB of codes
    wq = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    ws = torch.full((E, N // 128, K // 128), 127, dtype=torch.uint8, device="cuda")
    wq[-1] = torch.randint(0, 0x40, (N, K), generator=gen(53), device="cuda", dtype=torch.uint8)
    T = 300
    q, s = rows(54, T, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = T
    y, _ = m.linear_fp8(q, s, wq, ws, offsets=off)
    some = torch.tensor([0, 1, 300, 4095, 8191], device="cuda")
    ref.check(y[:, some], *ref.linear(ref.wide_rows(q, s), wq[-1][some].view(ref.E4M3).double(), None, None, "none")[0], "y")
    x, dy = rnd(55, (T, K)), rnd(56, (T, N))
    dx, dw, _ = m.linear_fp8_backward(dy, x, wq, ws, offsets=off)
    zr, _ = ref.quantised(dy.double(), torch.zeros((T, N), device="cuda", dtype=torch.float64), 1)
    r, b = ref.product(zr, wq[-1][:, -130:].view(ref.E4M3).double().t().contiguous(), chained=True)
    ref.check(dx[:, -130:], r, b + ref.HALF[BF16] * (r.abs() + b), "dx")
    zero = torch.zeros((T, 130), device="cuda", dtype=torch.float64)
    r, b = ref.product(ref.quantised(dy[:, -130:].double(), zero, 0)[0].t().contiguous(),
                       ref.quantised(x[:, -130:].double(), zero, 0)[0].t().contiguous(), chained=True)
    ref.check(dw[-1, -130:, -130:], r, b + ref.HALF[BF16] * (r.abs() + b), "dw")
    assert (dw[:-1, ::512, ::512] == 0).all()


def test_many_rows():
    T, K, N = 600_000, 8192, 128                          # 4.9 GB of codes
    q = torch.randint(0, 0x40, (T, K), generator=gen(57), device="cuda", dtype=torch.uint8)
    s = torch.ones((T, K // 128), device="cuda")
    wq, ws = weights(58, (N, K), True)
    y, _ = m.linear_fp8(q, s, wq, ws)
    some = torch.tensor([0, 255, 256, T // 2 + 1, T - 1], device="cuda")
    ref.check(y[some], *ref.linear(ref.wide_rows(q[some], s[some]), ref.wide(wq, ws), None, None, "none")[0], "y")
