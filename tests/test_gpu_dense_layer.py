"""The dense operators together, as a layer uses them around the routed experts; their calls
captured into graphs, on other streams and at once; rows and bytes they must not touch."""

import numpy as np
import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m
import synth
from moe_helpers import TOL, gpu_out_f64
from oracle.moe import ExpertWeights, forward, out_as_f64
from oracle.numerics import bf16_bits_to_f64
from synth.device import device_layer
from test_gpu_dense import ACT, BF16, EPS, F32, rnd

pytestmark = pytest.mark.gpu


def same(a, b):
    """Bitwise equality as a plain bool (a failure then prints no tensors)."""
    return (a.shape == b.shape and a.dtype == b.dtype
            and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)))


# ----------------------------------------------------------------------------- a layer

@pytest.mark.parametrize("T", [1, 48, 333])
def test_layer_forward(T):
    """norm -> router logits -> routed experts, and norm -> gated -> down with the routed output as its
    residual: every stage against the 64-bit form of that stage on the same inputs."""
    H, I, E, k = 256, 128, 6, 2
    spec = synth.Spec("dense_layer", T=T, H=H, I=I, E=E, k=k, act="bf16", weight="bf16", seed=4)
    L = synth.dense_layer(spec)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(BF16).cuda()

    wgu, wdn = dev(L["w_gate_up"]), dev(L["w_down"])
    x, res = rnd("lx", (T, H), BF16), rnd("lr", (T, H), BF16)
    nw, wr = rnd("lnw", (H,), BF16, 0.2, 1.0), rnd("lwr", (E, H), BF16, H ** -0.5)
    sgu, sdn = rnd("lsgu", (4 * I, H), BF16, H ** -0.5), rnd("lsdn", (H, 2 * I), BF16, (2 * I) ** -0.5)

    y, h, _ = m.rms_norm(x, nw, EPS, residual=res)
    logits, _ = m.linear(y, wr, out_dtype=F32)
    idx, w, *_ = m.route_logits(logits, k, True)
    routed = m.experts_forward(y, idx, w, wgu, wdn)
    a, _ = m.gated_linear(y, sgu)
    out, _ = m.linear(a, sdn, residual=routed)

    (ry, by), rh, _, _ = ref.norm(x, nw, EPS, res, BF16)
    ref.check(y, ry, by, "norm")
    assert torch.equal(h.double(), rh)
    (rl, bl), _ = ref.linear(y, wr, None, None, "none", BF16, F32)
    ref.check(logits, rl, bl, "logits")
    _, obits = forward(bf16_np(y), idx.cpu().numpy(), w.cpu().numpy(),
                       ExpertWeights("bf16", L["w_gate_up"], L["w_down"]), act="bf16")
    ro, (atol, rtol) = out_as_f64(obits, "bf16"), TOL["bf16"]
    assert (np.abs(gpu_out_f64(routed) - ro) <= atol + rtol * np.abs(ro)).all()
    (ra, ba), _ = ref.gated(y, sgu, None, "silu", BF16)
    ref.check(a, ra, ba, "gated")
    (rt, bt), _ = ref.linear(a, sdn, None, routed, "none", BF16, BF16)
    ref.check(out, rt, bt, "down")


def bf16_np(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("T", [1, 130])
def test_shared_expert_training_step(T):
    """Forward and backward of norm -> gated -> down + residual, stage by stage, the gradients
    chained as a training step chains them."""
    H, I = 264, 136
    x, nw = rnd("tx", (T, H), BF16), rnd("tn", (H,), BF16, 0.2, 1.0)
    wg, wd = rnd("tg", (2 * I, H), BF16, H ** -0.5), rnd("td", (H, I), BF16, I ** -0.5)
    y, h, rstd = m.rms_norm(x, nw, EPS)
    a, pre = m.gated_linear(y, wg, save_pre=True)
    out, _ = m.linear(a, wd, residual=h)
    dout = rnd("tdo", (T, H), BF16)
    da, dwd, _ = m.linear_backward(dout, a, wd)
    dy, dwg, _ = m.gated_linear_backward(da, y, wg, pre)
    dx, dnw = m.rms_norm_backward(dy, h, nw, rstd, dh=dout)      # the residual carries dout to h

    g1 = ref.backward(*ref.dz_linear(dout, None, "none"), a, wd, BF16)
    g2 = ref.backward(*ref.dz_gated(da, pre, "silu"), y, wg, BF16)
    g3 = ref.norm_backward(dy, h, nw, rstd, dout, BF16)
    for got, (r, b), what in ((da, g1[0], "da"), (dwd, g1[1], "dw_down"), (dy, g2[0], "dy"), (dwg, g2[1], "dw_gate_up"),
                              (dx, g3[0], "dx"), (dnw, g3[1], "dweight")):
        ref.check(got, r, b, what)

    # the whole step against automatic differentiation of the same step in 64 bits: ten bf16
    # roundings lie between dout and the furthest gradient, each at most 2^-8 of its tensor's norm
    leaves = [t.double().requires_grad_(True) for t in (x, nw, wg, wd)]
    X, NW, WG, WD = leaves
    N = X * (X.square().mean(1, keepdim=True) + EPS) ** -0.5 * NW
    G, U = (N @ WG.t()).chunk(2, 1)
    (((G * torch.sigmoid(G) * U) @ WD.t() + X) * dout.double()).sum().backward()
    for got, leaf, what in zip((dx, dnw, dwg, dwd), leaves, ("dx", "dweight", "dw_gate_up", "dw_down")):
        assert ((got.double() - leaf.grad).norm() <= 10 * 2.0 ** -8 * leaf.grad.norm()), what


@pytest.mark.parametrize("weight,scale", [("fp8", "f32"), ("fp8", "ue8m0"), ("fp4", "ue8m0")])
@pytest.mark.parametrize("T", [1, 200])
def test_experts_on_quantised_rows(weight, scale, T):
    spec = synth.Spec("dense_q", T=T, H=384, I=256, E=8, k=2, act="bf16", weight=weight, scale=scale, seed=9)
    D = device_layer(spec)
    experts = (D["idx"], D["w"], D["w_gate_up"], D["w_down"])
    kw = dict(w_gate_up_scale=D["w_gate_up_scale"], w_down_scale=D["w_down_scale"])
    q, s = m.quantize_rows_fp8(D["x"])
    want = m.experts_forward(D["x"], *experts, **kw)
    assert same(m.experts_forward_quantized(q, s, *experts, **kw), want)
    # the norm's 8-bit rows of an all-ones weight and the quantised norm agree with the experts on them
    nq, ns, _, _, _ = m.rms_norm_fp8(D["x"], rnd("qw", (spec.H,), BF16, 0.2, 1.0), EPS)
    out = m.experts_forward_quantized(nq.view(torch.float8_e4m3fn), ns, *experts, **kw)
    rows = (nq.view(torch.float8_e4m3fn).float().view(T, -1, 128) * ns[:, :, None]).view(T, -1)
    assert torch.isfinite(out).all()
    if T > 1:   # e4m3 rows are off by 2^-4 at most, 2^-5 in the mean: the experts on bf16 rows of their values are near
        near = m.experts_forward(rows.to(BF16), *experts, **kw)
        assert (out.float() - near.float()).norm() <= 2.0 ** -3 * near.float().norm()
    with pytest.raises(ValueError):
        m.experts_forward_quantized(q, s[:, :-1].contiguous(), *experts, **kw)
    with pytest.raises(ValueError):
        m.experts_forward_quantized(D["x"], s, *experts, **kw)


# ----------------------------------------------------------------------------- no rows

def test_no_rows():
    for dt in (BF16, F32):
        x, w = torch.empty((0, 64), dtype=dt, device="cuda"), rnd("e", (48, 64), dt)
        nw = rnd("en", (64,), dt)
        y, h, rstd = m.rms_norm(x, nw, EPS, residual=x)
        assert y.shape == h.shape == (0, 64) and rstd.shape == (0,)
        dx, dn = m.rms_norm_backward(x, x, nw, rstd)
        assert dx.shape == (0, 64) and (dn == 0).all()
        assert m.linear(x, w)[0].shape == (0, 48) and m.gated_linear(x, w)[0].shape == (0, 24)
        for dx, dw, db in (m.linear_backward(torch.empty((0, 48), dtype=dt, device="cuda"), x, w, need_bias=True),
                           m.gated_linear_backward(torch.empty((0, 24), dtype=dt, device="cuda"), x, w,
                                                   torch.empty((0, 48), dtype=dt, device="cuda"), need_bias=True)):
            assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


# ----------------------------------------------------------------------------- special values

def test_infinities_and_nan_stay_in_their_rows():
    """Rows of x with NaN or infinities spoil their own output rows alone, at the edges of tiles
    and where a contraction ends inside a slice."""
    for T, K, N in ((5, 72, 40), (70, 200, 264), (300, 136, 520), (2100, 328, 1032)):
        x, w = rnd("sx", (T, K), BF16), rnd("sw", (2 * N, K), BF16, K ** -0.5)
        bad = torch.zeros(T, dtype=torch.bool, device="cuda")
        clean = m.linear(x, w)[0], m.gated_linear(x, w)[0], m.rms_norm(x, w[0].contiguous(), EPS)[0]
        for i, v in ((0, float("nan")), (T // 2, float("inf")), (T - 1, -float("inf"))):
            x[i, i % K] = v
            bad[i] = True
        got = m.linear(x, w)[0], m.gated_linear(x, w)[0], m.rms_norm(x, w[0].contiguous(), EPS)[0]
        for g, c in zip(got, clean):
            assert same(g[~bad], c[~bad])
        assert not torch.isfinite(got[0][bad]).any()
        # dw: a NaN in row t of dy reaches only its own output's row of dw, and no row of dx but t
        dy = rnd("sdy", (T, 2 * N), BF16)
        x = rnd("sx", (T, K), BF16)
        dx0, dw0, _ = m.linear_backward(dy, x, w)
        dy[T - 1, 3] = float("nan")
        dx1, dw1, _ = m.linear_backward(dy, x, w)
        assert same(dx1[:-1], dx0[:-1]) and torch.isnan(dx1[-1]).all()
        keep = torch.arange(2 * N, device="cuda") != 3
        assert same(dw1[keep], dw0[keep]) and torch.isnan(dw1[3]).all()


# ----------------------------------------------------------------------------- what must not be touched

@pytest.mark.parametrize("T,K,N", [(5, 72, 41), (33, 200, 264), (130, 136, 60), (1030, 264, 520)])
def test_writes_stay_inside(T, K, N):
    """Outputs inside wider, longer buffers: what lies between rows and behind the last is left as it was."""
    import ctypes
    x, w = rnd("ix", (T, K), BF16), rnd("iw", (N, K), BF16, K ** -0.5)
    ld = (N + 7) // 8 * 8 + 8
    buf = torch.full((T + 3, ld), 7.0, dtype=BF16, device="cuda")
    pre = torch.full((T + 3, ld), 7.0, dtype=BF16, device="cuda")
    p = m.LinearProblem(T, K, N, m.BF16, m.BF16, m.ACT_SILU, 0, ld, 0, ld, 0)
    n = ctypes.c_size_t(0)
    assert m.lib().moe_linear_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert m.lib().moe_linear(ctypes.byref(p), x.data_ptr(), w.data_ptr(), None, None, buf.data_ptr(), pre.data_ptr(),
                              ws.data_ptr(), n.value, s) == 0
    y, z = m.linear(x, w, act=m.ACT_SILU, save_pre=True)
    assert same(buf[:T, :N], y) and same(pre[:T, :N], z)
    for b in (buf, pre):
        assert (b[:T, N:] == 7).all() and (b[T:] == 7).all()
    assert (ws[n.value:] == 0xA5).all()

    dy = rnd("idy", (T, N), BF16)
    p = m.LinearProblem(T, K, N, m.BF16, m.BF16, m.ACT_SILU, 0, 0, 0, ld, K + 16)
    assert m.lib().moe_linear_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    dx = torch.full((T + 3, K + 16), 7.0, dtype=BF16, device="cuda")
    dw = torch.full((N + 3, K), 7.0, dtype=BF16, device="cuda")
    assert m.lib().moe_linear_backward(ctypes.byref(p), dy.data_ptr(), x.data_ptr(), w.data_ptr(), pre.data_ptr(),
                                       dx.data_ptr(), dw.data_ptr(), None, ws.data_ptr(), n.value, s) == 0
    rx, rw, _ = m.linear_backward(dy, x, w, pre=z, act=m.ACT_SILU)
    assert same(dx[:T, :K], rx) and same(dw[:N], rw)
    assert (dx[:T, K:] == 7).all() and (dx[T:] == 7).all() and (dw[N:] == 7).all() and (ws[n.value:] == 0xA5).all()


def test_in_place_forms():
    import ctypes
    s = torch.cuda.current_stream().cuda_stream
    for T in (3, 200, 2000):
        x, res, w = rnd("px", (T, 256), BF16), rnd("pr", (T, 256), BF16), rnd("pw", (256,), BF16)
        y, h, _ = m.rms_norm(x, w, EPS, residual=res)
        for target in (0, 1):
            xr = [x.clone(), res.clone()]
            y2, rstd = torch.empty_like(y), torch.empty(T, device="cuda")
            p = m.NormProblem(T, 256, m.BF16, EPS, 0, 0, 0, 0)
            assert m.lib().moe_rms_norm(ctypes.byref(p), xr[0].data_ptr(), xr[1].data_ptr(), w.data_ptr(), y2.data_ptr(),
                                        xr[target].data_ptr(), rstd.data_ptr(), None, None, s) == 0
            assert same(y2, y) and same(xr[target], h)
        w2, acc = rnd("pw2", (264, 256), BF16, 0.06), rnd("pa", (T, 264), BF16)
        want, _ = m.linear(x, w2, residual=acc)
        pl = m.LinearProblem(T, 256, 264, m.BF16, m.BF16, 0, 0, 0, 0, 0, 0)
        n = ctypes.c_size_t(0)
        assert m.lib().moe_linear_workspace_size(ctypes.byref(pl), 0, ctypes.byref(n)) == 0
        ws = torch.empty(max(n.value, 16), dtype=torch.uint8, device="cuda")
        assert m.lib().moe_linear(ctypes.byref(pl), x.data_ptr(), w2.data_ptr(), None, acc.data_ptr(), acc.data_ptr(),
                                  None, ws.data_ptr(), n.value, s) == 0
        assert same(acc, want)


# ----------------------------------------------------------------------------- streams and graphs

def calls(T, K, N, seed=""):
    """One call of every entry point on its own inputs: (function of no arguments, ...) each returning its outputs."""
    x, w, b = rnd(f"gx{seed}", (T, K), BF16), rnd(f"gw{seed}", (2 * N, K), BF16, K ** -0.5), rnd(f"gb{seed}", (2 * N,), BF16)
    nw, res = rnd(f"gn{seed}", (K,), BF16), rnd(f"gr{seed}", (T, K), BF16)
    z, dz = rnd(f"gz{seed}", (T, 2 * N), BF16), rnd(f"gd{seed}", (T, 2 * N), BF16)
    da, rstd = rnd(f"ga{seed}", (T, N), BF16), torch.rand(T, device="cuda") + 0.5
    return [lambda: m.rms_norm(x, nw, EPS, residual=res), lambda: m.rms_norm_fp8(x, nw, EPS)[:2],
            lambda: m.rms_norm_backward(x, res, nw, rstd, dh=x),
            lambda: m.linear(x, w, b, residual=dz, act=m.ACT_GELU, save_pre=True),
            lambda: m.linear_backward(dz, x, w, pre=z, act=m.ACT_SILU, need_bias=True),
            lambda: m.linear_backward(dz, x, w),
            lambda: m.gated_linear(x, w, b, save_pre=True),
            lambda: m.gated_linear_backward(da, x, w, z, need_bias=True)]


def flat(out):
    return [t for t in out if isinstance(t, torch.Tensor)]


@pytest.mark.parametrize("T,K,N", [(1, 256, 128), (50, 1024, 264), (600, 2048, 1024)])
def test_captured_calls_replay_equal(T, K, N):
    fns = calls(T, K, N)
    want = [[t.clone() for t in flat(f())] for f in fns]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in fns:
            f()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [flat(f()) for f in fns]
    for _ in range(4):
        for out in got:
            for t in out:
                t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for out, ref_out in zip(got, want):
            for t, r in zip(out, ref_out):
                ok = same(t, r)
                assert ok
        eager = [flat(f()) for f in fns]       # the program's own work between replays
        for out, ref_out in zip(eager, want):
            for t, r in zip(out, ref_out):
                ok = same(t, r)
                assert ok


def test_calls_on_several_streams_at_once():
    sets = [calls(T, 512, 264, str(i)) for i, T in enumerate((3, 130, 700, 1500))]
    torch.cuda.synchronize()
    want = [[[t.clone() for t in flat(f())] for f in fns] for fns in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[] for _ in sets]
        for k in range(len(sets[0])):
            for i, (fns, st) in enumerate(zip(sets, streams)):
                with torch.cuda.stream(st):
                    got[i].append(flat(fns[k]()))
        torch.cuda.synchronize()
        for g, wnt in zip(got, want):
            for out, ref_out in zip(g, wnt):
                for t, r in zip(out, ref_out):
                    ok = same(t, r)
                assert ok


def test_calls_from_several_host_threads():
    import threading
    sets = [calls(T, 256, 136, f"t{i}") for i, T in enumerate((2, 65, 300))]
    want = [[[t.clone() for t in flat(f())] for f in fns] for fns in sets]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got = [flat(f()) for f in sets[i]]
                torch.cuda.current_stream().synchronize()
                if not all(same(t, r) for out, ref_out in zip(got, want[i]) for t, r in zip(out, ref_out)):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_results_do_not_depend_on_what_the_workspace_held():
    """The caller's workspace may hold anything, NaN among it, and may be larger than needed."""
    for T, K, N in ((20, 7168, 61), (200, 2048, 264), (8, 512, 512)):
        x, w = rnd("wx", (T, K), BF16), rnd("ww", (N, K), BF16, K ** -0.5)
        dy, z = rnd("wdy", (T, N), BF16), rnd("wz", (T, N), BF16)
        ws = torch.full((1 << 27,), 0xFF, dtype=torch.uint8, device="cuda")
        assert same(m.linear(x, w, workspace=ws)[0], m.linear(x, w)[0])
        ws.fill_(0xFF)
        got = m.linear_backward(dy, x, w, pre=z, act=m.ACT_SILU, need_bias=True, workspace=ws)
        for a, b in zip(got, m.linear_backward(dy, x, w, pre=z, act=m.ACT_SILU, need_bias=True)):
            assert same(a, b)


# ----------------------------------------------------------------------------- far offsets

@pytest.mark.parametrize("T", [3, 40, 700])
def test_gated_weights_beyond_32_bit_offsets(T):
    """The up projection's rows start more than 4 GiB behind the gate's; sampled columns against the
    64-bit form."""
    H, I = 65536, 32784
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty((2 * I, H), dtype=BF16, device="cuda").normal_(0, H ** -0.5, generator=g)
    x = rnd("ox", (T, H), BF16)
    a, pre = m.gated_linear(x, w, save_pre=True)
    cols = torch.tensor([0, 1, 63, 64, 127, 128, 8191, 32768, I - 1], device="cuda")
    ws = torch.cat([w[cols], w[I + cols]])
    (ra, ba), (rz, bz) = ref.gated(x, ws, None, "silu", BF16)
    ref.check(a[:, cols], ra, ba, "a")
    ref.check(pre[:, torch.cat([cols, I + cols])], rz, bz, "pre")


def test_rows_beyond_32_bit_offsets():
    """Activations of more than 4 GiB: the last rows of every output."""
    T, H = 70000, 32768
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.empty((T, H), dtype=BF16, device="cuda").normal_(generator=g)
    w, nw = rnd("ow", (24, H), BF16, H ** -0.5), rnd("onw", (H,), BF16, 0.2, 1.0)
    y, _ = m.linear(x, w)
    tail = x[-300:].clone()
    (ry, by), _ = ref.linear(tail, w, None, None, "none", BF16, BF16)
    ref.check(y[-300:], ry, by, "linear")
    n, _, rstd = m.rms_norm(x, nw, EPS)
    (rn, bn), _, (rr, br), _ = ref.norm(tail, nw, EPS, None, BF16)
    ref.check(n[-300:], rn, bn, "norm")
    ref.check(rstd[-300:], rr, br, "rstd")
    dy = rnd("ody", (T, 24), BF16)
    dx, dw, _ = m.linear_backward(dy, x, w)
    grads = ref.backward(*ref.dz_linear(dy[-300:], None, "none"), tail, w, BF16)
    ref.check(dx[-300:], *grads[0], "dx")
    part = torch.zeros((24, 64), dtype=torch.float64, device="cuda")      # dw's last columns, in pieces of rows
    mag = torch.zeros_like(part)
    for i in range(0, T, 10000):
        d, xs = dy[i:i + 10000].double(), x[i:i + 10000, -64:].double()
        part += d.t() @ xs
        mag += d.abs().t() @ xs.abs()
    ref.check(dw[:, -64:], part, (T + 1) * ref.U32 * mag + 2.0 ** -8 * part.abs() * 1.01, "dw")


# ----------------------------------------------------------------------------- refusals of the binding

def test_binding_refuses():
    x, w, b = rnd("rx", (4, 64), BF16), rnd("rw", (32, 64), BF16), rnd("rb", (32,), BF16)
    nw, z, dy = rnd("rn", (64,), BF16), rnd("rz", (4, 32), BF16), rnd("rdy", (4, 32), BF16)
    bad = [lambda: m.linear(x[0], w), lambda: m.linear(x, w[0]), lambda: m.linear(x, w[:, :56].contiguous()),
           lambda: m.linear(x, w.float()), lambda: m.linear(x, w, bias=b[:31]), lambda: m.linear(x, w, bias=b.float()),
           lambda: m.linear(x, w, residual=dy.float()), lambda: m.linear(x, w, residual=dy[:3]),
           lambda: m.linear(x, w, out_dtype=torch.float16), lambda: m.linear(x, w, act=4),
           lambda: m.linear(x.t().contiguous().t(), w), lambda: m.linear(x, w.t().contiguous().t()),
           lambda: m.linear(x[:1].expand(4, 64), w), lambda: m.linear(x[:, :60], w[:, :60].contiguous()),
           lambda: m.linear(torch.empty((4, 65), dtype=BF16, device="cuda")[:, :64], w),        # rows not 16-byte aligned
           lambda: m.linear(torch.empty((4, 72), dtype=BF16, device="cuda")[:, 4:68], w),       # nor the first
           lambda: m.linear(x.cpu(), w), lambda: m.linear(x, w.cpu()), lambda: m.linear(x, w, residual=dy.cpu()),
           lambda: m.linear(x, w, workspace=torch.empty(16, dtype=torch.uint8)),
           lambda: m.linear_backward(dy, x, w, act=m.ACT_GELU), lambda: m.linear_backward(dy[:, :31], x, w),
           lambda: m.linear_backward(dy, x, w, pre=z[:3], act=m.ACT_GELU),
           lambda: m.linear_backward(dy, x, w, pre=z, act=m.ACT_GELU,
                                     workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: m.gated_linear(x, w[:31].contiguous()), lambda: m.gated_linear(x, w, act=m.ACT_NONE),
           lambda: m.gated_linear(x, w[:24].contiguous()), lambda: m.gated_linear(x, w, bias=b[:16]),
           lambda: m.gated_linear_backward(dy, x, w, z), lambda: m.gated_linear_backward(dy[:, :16], x, w, z[:, :16]),
           lambda: m.rms_norm(x, nw[:63]), lambda: m.rms_norm(x, nw.float()), lambda: m.rms_norm(x, nw, residual=x[:3]),
           lambda: m.rms_norm(x, nw, -1.0), lambda: m.rms_norm(x, nw, float("nan")), lambda: m.rms_norm_fp8(x, nw),
           lambda: m.rms_norm_fp8(x.float(), nw.float()),
           lambda: m.rms_norm_backward(x, x, nw, torch.ones(3, device="cuda")),
           lambda: m.rms_norm_backward(x, x, nw, torch.ones(4, device="cuda").double()),
           lambda: m.rms_norm_backward(x, x, nw, torch.ones(4, device="cuda"),
                                       workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for i, f in enumerate(bad):
        try:
            f()
        except ValueError:
            continue
        raise AssertionError(f"call {i} was taken")
