"""Rows in expert order and the e4m3 products as a layer uses them: a routed layer's forward in separate calls against the fused
forward, a training step of it against 64 bits, captured graphs, several streams and threads, workspaces with old contents."""

import threading

import pytest
import torch

import fp8_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_fp8 import gen, rnd, rows, runs, weights

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
T, H, I, E, k = 200, 512, 256, 8, 2


def layer(ue8m0):
    gq, gs = weights(1, (E, 2 * I, H), ue8m0)
    dq, ds = weights(2, (E, H, I), ue8m0)
    x = rnd(3, (T, H))
    logits = torch.randn((T, E), generator=gen(4), device="cuda")
    return x, logits, (gq, gs), (dq, ds)


def forward(x, logits, up, down):
    q, s = m.quantize_rows_fp8(x)
    idx, w, counts, off, perm, inv = m.route_logits(logits, k, renorm=True)
    yq, ys = m.permute(q, inv, scale=s)
    a, pre = m.gated_linear_fp8(yq, ys, *up, save_pre=True, offsets=off)
    aq, as_ = m.quantize_rows_fp8(a)
    y, _ = m.linear_fp8(aq, as_, *down, offsets=off)
    return m.unpermute(y, inv, w), (q, s, idx, w, off, inv, a, pre, y)


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
def test_a_layer_in_separate_calls(ue8m0):
    """Against the fused forward on the same codes.  That one requantises the activation before its rounding to bf16 and adds rows
    it has weighted and rounded: an activation may take another code (a step is at most 2^-3 of its value, of which half is a rounding
    either forward makes) and every row of the sum another bf16 value."""
    x, logits, up, down = layer(ue8m0)
    out, (q, s, idx, w, off, inv, a, pre, y) = forward(x, logits, up, down)
    fused = m.experts_forward_quantized(q, s, idx, w, up[0], down[0], up[1], down[1])
    av = torch.zeros((T, E, I), device="cuda", dtype=torch.float64)
    bound = torch.zeros((T, H), device="cuda", dtype=torch.float64)
    want = torch.zeros((T, H), device="cuda", dtype=torch.float64)
    for e in range(E):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        (r, _), _ = ref.gated(ref.wide_rows(q[t], s[t]), ref.wide(up[0][e], up[1][e]), "silu")
        g = r.view(len(t), -1, 128)
        # e4m3: half a step is 2^-4 of a value, or 2^-10 of the scale (a group's largest over 448) below 2^-6
        step = (2.0 ** -4 * g.abs() + 2.0 ** -10 * g.abs().amax(2, keepdim=True) / 448).view_as(r) + 2.0 ** -8 * r.abs()
        dv = ref.wide(down[0][e], down[1][e])
        wt = w[t, j].double()[:, None]
        want.index_add_(0, t, wt * (r @ dv.t()))
        bound.index_add_(0, t, wt * (1.01 * step @ dv.abs().t() + 2.0 ** -7 * (r @ dv.t()).abs()))
    bound += 2.0 ** -8 * want.abs()
    for got, name in ((out, "separate"), (fused, "fused")):
        over = ((got.double() - want).abs() / bound).max().item()
        assert over <= 1.0, f"{name}: {over:.3g} of its bound"


def backward(x, saved, up, down, dout):
    q, s, idx, w, off, inv, a, pre, y = saved
    dy, dw = m.unpermute_backward(dout, y, inv, w)
    da, d_down, _ = m.linear_fp8_backward(dy, a, *down, offsets=off)
    xs, _ = m.permute(x, inv)
    dxs, d_up = m.gated_linear_fp8_backward(da, xs, *up, pre, offsets=off)
    return m.permute_backward(dxs, inv, T), dw, d_up, d_down, dy, da, dxs, xs


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
def test_a_training_step(ue8m0):
    """Every gradient of the chain against the formula on what the call before it left."""
    x, logits, up, down = layer(ue8m0)
    out, saved = forward(x, logits, up, down)
    q, s, idx, w, off, inv, a, pre, y = saved
    dout = rnd(5, (T, H))
    dx, dw, d_up, d_down, dy, da, dxs, xs = backward(x, saved, up, down, dout)
    at = inv.long().view(T, k)
    assert torch.equal(dy[at], (dout.float()[:, None, :] * w[:, :, None]).to(BF16))
    p = dout.double()[:, None, :] * y.double()[at]
    ref.check(dw, p.sum(2), (H + 2) * ref.U32 * p.abs().sum(2), "dw")
    o = off.tolist()
    for e in range(E):
        r = slice(o[e], o[e + 1])
        want = ref.backward(*ref.dz_linear(dy[r], None, "none"), a[r], ref.wide(down[0][e], down[1][e]))
        ref.check(da[r], *want[0], "da")
        ref.check(d_down[e], *want[1], "d_down")
        want = ref.backward(*ref.dz_gated(da[r], pre[r], "silu"), xs[r], ref.wide(up[0][e], up[1][e]))
        ref.check(dxs[r], *want[0], "dxs")
        ref.check(d_up[e], *want[1], "d_up")
    sums = dxs.double()[at]
    b = (k + 1) * ref.U32 * sums.abs().sum(1)
    ref.check(dx, sums.sum(1), b + 2.0 ** -8 * (sums.sum(1).abs() + b), "dx")
    # a step's weights in blocks again
    nq, ns = m.quantize_blocks_fp8((ref.wide(*up) - 0.01 * d_up.double()).float(), ue8m0)
    assert nq.shape == up[0].shape and ns.shape == up[1].shape and ns.dtype == up[1].dtype


def test_a_shared_expert_behind_the_norm():
    x, weight = rnd(6, (70, H)), rnd(7, (H,), BF16, 0.1) + 1
    q, s, _, _, _ = m.rms_norm_fp8(x, weight)
    (gq, gs), (dq, ds) = weights(8, (2 * I, H), False), weights(9, (H, I), False)
    routed = rnd(10, (70, H))
    a, _ = m.gated_linear_fp8(q, s, gq, gs)
    aq, as_ = m.quantize_rows_fp8(a)
    y, _ = m.linear_fp8(aq, as_, dq, ds, residual=routed)
    (ra, ba), _ = ref.gated(ref.wide_rows(q, s), ref.wide(gq, gs), "silu")
    ref.check(a, ra, ba, "a")
    ref.check(y, *ref.linear(ref.wide_rows(aq, as_), ref.wide(dq, ds), None, routed, "none")[0], "y")


def test_replays_in_a_graph():
    x, logits, up, down = layer(True)
    dout = rnd(11, (T, H))
    one_q, one_s = weights(12, (I, H), False)
    dyd = rnd(13, (T, I))

    def step():
        out, saved = forward(x, logits, up, down)
        dense = m.linear_fp8_backward(dyd, x, one_q, one_s, need_bias=True)
        return (out, *backward(x, saved, up, down, dout)[:4], *dense)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):                                    # two graphs in flight, each with its own buffers
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()
        graphs.append((g, held))
    for i in range(3):
        x.copy_(rnd(20 + i, (T, H)))
        logits.copy_(torch.randn((T, E), generator=gen(30 + i), device="cuda"))
        want = step()                                     # eager work between the replays
        for g, held in graphs:
            for t in held:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, held in graphs:
            for a, b in zip(held, want):
                assert torch.equal(a, b), f"replay {i}"


def test_streams_threads_and_workspaces():
    """Calls that overlap give what they give alone, also on workspaces that hold other values (NaN codes and bit patterns)."""
    import ctypes
    cases = []
    for n, (TT, K, N, EE) in enumerate(((300, 512, 256, 0), (20, 256, 128, 0), (400, 256, 384, 3), (90, 1024, 256, 0))):
        q, s = rows(40 + n, TT, K)
        wq, ws = weights(50 + n, (EE, N, K) if EE else (N, K), bool(n & 1))
        off = runs(60 + n, TT, EE) if EE else None
        x, dy = rnd(70 + n, (TT, K)), rnd(80 + n, (TT, N))
        p = m.Fp8Problem(TT, K, N, EE, m.SCALE_UE8M0 if n & 1 else m.SCALE_F32, m.ACT_NONE, 0, 0, 0, 0, 0)
        size = ctypes.c_size_t(0)
        need = 0
        for b in (0, 2):
            assert m.lib().moe_linear_fp8_workspace_size(ctypes.byref(p), b, ctypes.byref(size)) == 0
            need = max(need, size.value)
        cases.append((q, s, wq, ws, off, x, dy, torch.full((max(need, 1),), 0x7F, dtype=torch.uint8, device="cuda")))

    def call(c, ws=None):
        q, s, wq, sc, off, x, dy, _ = c
        return (m.linear_fp8(q, s, wq, sc, offsets=off, workspace=ws)[0],
                *m.linear_fp8_backward(dy, x, wq, sc, offsets=off, workspace=ws)[:2])
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    for fill in (0x7F, 0xFF):
        got = [None] * len(cases)
        for c in cases:
            c[-1].fill_(fill)
        torch.cuda.synchronize()

        def work(i):
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = call(cases[i], cases[i][-1])
                torch.cuda.current_stream().synchronize()
        threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_results_do_not_depend_on_timing():
    wq, ws = weights(90, (512, 1024), False)
    x, dy = rnd(91, (900, 1024)), rnd(92, (900, 512))
    first = m.linear_fp8_backward(dy, x, wq, ws, need_bias=True)
    for _ in range(3):
        for a, b in zip(m.linear_fp8_backward(dy, x, wq, ws, need_bias=True), first):
            assert torch.equal(a, b)
