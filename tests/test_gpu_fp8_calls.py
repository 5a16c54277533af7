"""Calls of the e4m3 products as programs make them: few rows by expert in captured graphs and on several streams, results in the residual's
place, the same call twice."""

import threading

import pytest
import torch

import mixture_experts_routed_topk_amd as m
from test_gpu_fp8 import BF16, rnd, rows, runs, weights

pytestmark = pytest.mark.gpu


def offsets(lengths):
    return torch.cat([torch.zeros(1, dtype=torch.int32), torch.tensor(lengths, dtype=torch.int32).cumsum(0, dtype=torch.int32)]).cuda()


@pytest.mark.parametrize("T,E", [(30, 100), (30, 3), (200, 100)])
def test_offsets_that_change_between_replays(T, E):
    """Runs grow, shrink, end before the last row and move past a wave's 64 experts; rows of no run keep what they held."""
    K, N = 512, 256
    q, s = rows(1, T, K)
    up, down = weights(2, (E, 2 * N, K), True), weights(3, (E, K, N), False)
    x, da = rnd(4, (T, K)), rnd(5, (T, N), BF16, 1e-3)
    off = runs(6, T, E)
    a = torch.empty((T, N), dtype=BF16, device="cuda")
    y = torch.empty((T, K), dtype=BF16, device="cuda")
    dx = torch.empty((T, K), dtype=BF16, device="cuda")

    def step(off, a, y, dx):
        a.fill_(2.0), y.fill_(3.0), dx.fill_(4.0)
        _, pre = m.gated_linear_fp8(q, s, *up, save_pre=True, offsets=off, out=a)
        aq, as_ = m.quantize_rows_fp8(a)
        m.linear_fp8(aq, as_, *down, offsets=off, out=y)
        _, dw = m.gated_linear_fp8_backward(da, x, *up, pre, offsets=off, out=dx)
        return a, y, dx, dw
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(off, a, y, dx)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step(off, a, y, dx)
    last = [0] * (E - 1)
    lengths = [[T] + last, last + [T], [1] * min(T, E) + [0] * (E - min(T, E)), last + [1], [0] * E,
               [0] + [T // 2] + [0] * (E - 3) + [T - T // 2 - 3]]
    for i, n in enumerate(lengths):
        new = offsets(n)
        off.copy_(new)
        rest = int(new[-1])
        q.copy_(rows(10 + i, T, K)[0])
        want = step(new, *(torch.empty_like(t) for t in (a, y, dx)))      # eager work between the replays
        for t in held:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(held, want):
            assert torch.equal(u, v), f"replay {i}"
        assert (a[rest:] == 2.0).all() and (y[rest:] == 3.0).all() and (dx[rest:] == 4.0).all()


def test_few_rows_by_expert_on_several_streams():
    cases = []
    for n, (T, K, N, E) in enumerate(((20, 256, 128, 4), (32, 1024, 256, 70), (1, 4224, 128, 8), (12, 512, 512, 2))):
        cases.append((*rows(20 + n, T, K), weights(30 + n, (E, N, K), bool(n & 1)), weights(40 + n, (E, 2 * N, K), not n & 1), runs(50 + n, T, E)))

    def call(c):
        q, s, w, gate, off = c
        return m.linear_fp8(q, s, *w, offsets=off)[0], m.gated_linear_fp8(q, s, *gate, offsets=off)[0]
    want = [call(c) for c in cases]
    torch.cuda.synchronize()
    got = [[] for _ in cases]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i].append(call(cases[i]))
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert len(a) == 5
        for pair in a:
            for u, v in zip(pair, b):
                assert torch.equal(u, v)


# few rows (a wave's columns and eight waves); tiles of 128 and of 256 rows; contractions in splits, which a second launch adds
@pytest.mark.parametrize("T,K,N", [(1, 256, 128), (16, 512, 256), (40, 4224, 128), (130, 256, 4096), (4099, 512, 2048), (100, 7168, 256), (700, 7168, 256)])
def test_results_in_the_residuals_place(T, K, N):
    q, s = rows(60, T, K)
    w = weights(61, (N, K), False)
    bias = rnd(62, (N,))
    for pitch in (N, N + 24):
        res = rnd(63, (T, pitch))
        for kw in ({}, dict(bias=bias, act=m.ACT_SILU)):
            want, _ = m.linear_fp8(q, s, *w, residual=res[:, :N], **kw)
            held = res.clone()
            got, _ = m.linear_fp8(q, s, *w, residual=held[:, :N], out=held[:, :N], **kw)
            assert torch.equal(got, want) and torch.equal(held[:, N:], res[:, N:])


@pytest.mark.parametrize("T,K,N,E", [(20, 512, 256, 0), (20, 512, 256, 6), (700, 7168, 256, 0), (3000, 256, 640, 5), (2731, 1024, 2816, 0)])
def test_the_same_call_twice(T, K, N, E):
    """No result depends on which workgroup comes first."""
    shape = (E,) if E else ()
    q, s = rows(70, T, K)
    off = runs(71, T, E) if E else None
    w, gate = weights(72, (*shape, N, K), False), weights(73, (*shape, 2 * N, K), True)
    x, dy, pre = rnd(74, (T, K)), rnd(75, (T, N), BF16, 1e-3), rnd(76, (T, 2 * N))

    def call():
        y, _ = m.linear_fp8(q, s, *w, offsets=off)
        a, p = m.gated_linear_fp8(q, s, *gate, save_pre=True, offsets=off)
        dx, dw, _ = m.linear_fp8_backward(dy, x, *w, offsets=off)
        return y, a, p, dx, dw, *m.gated_linear_fp8_backward(dy, x, *gate, pre, offsets=off)
    first = call()
    for _ in range(3):
        for u, v in zip(call(), first):
            assert torch.equal(u, v)
