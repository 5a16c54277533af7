"""Rows in expert order and back (moe_permute, moe_unpermute and its gradient) against plain 64-bit forms."""

import threading

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U32 = ref.U32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(seed, shape, dtype):
    return torch.randn(shape, generator=gen(seed), device="cuda").to(dtype)


def positions(seed, T, k, drop=0.0, spare=0):
    """inv [T*k] with some slots left out, and the rows of a sorted matrix with `spare` more than are named."""
    n = T * k
    keep = torch.rand(n, generator=gen(seed), device="cuda") >= drop
    order = torch.randperm(n + spare, generator=gen(seed + 1), device="cuda")[:n]
    inv = torch.where(keep, order, torch.full_like(order, -1)).to(torch.int32)
    return inv, n + spare


SHAPES = [  # T, k, H
    (1, 1, 8), (1, 8, 2048), (3, 9, 72), (16, 4, 2048), (65, 2, 264), (130, 8, 520), (33, 17, 1032), (257, 6, 7168), (5, 64, 65536)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_permute_moves_rows_and_leaves_the_others(T, k, H, dtype):
    for drop, spare in ((0.0, 0), (0.4, 5)):
        inv, rows = positions(T + k, T, k, drop, spare)
        x = rnd(1, (T, H + 8), dtype)[:, :H]                       # a pitch of its own
        out = torch.full((rows, H + 16), -7.0, device="cuda", dtype=dtype)[:, :H]
        want = out.clone()
        here = inv >= 0
        want[inv[here].long()] = x.repeat_interleave(k, 0)[here]
        y, scale = m.permute(x, inv, out=out)
        assert y is out and scale is None
        assert torch.equal(out, want)
        y, _ = m.permute(x.contiguous(), inv, rows=rows)
        named = inv[here].long()
        assert torch.equal(y[named], want[named])


@pytest.mark.parametrize("T,k,H", [(1, 1, 128), (37, 3, 256), (130, 8, 7168)])
def test_permute_moves_codes_with_their_scales(T, k, H):
    inv, rows = positions(T, T, k, 0.2, 3)
    q, s = m.quantize_rows_fp8(rnd(2, (T, H), BF16))
    for codes in (q, q.view(torch.float8_e4m3fn)):
        y, ys = m.permute(codes, inv, rows=rows, scale=s)
        here = inv >= 0
        named = inv[here].long()
        assert y.dtype == codes.dtype
        assert torch.equal(y.view(torch.uint8)[named], q.repeat_interleave(k, 0)[here])
        assert torch.equal(ys[named], s.repeat_interleave(k, 0)[here])
    y, ys = m.permute(q, inv, rows=rows)
    assert ys is None and torch.equal(y[named], q.repeat_interleave(k, 0)[here])


def combine(y, inv, w, T):
    """(sum, sum of absolute values) in 64 bits."""
    k = inv.numel() // T
    y = torch.cat([y.double(), torch.zeros((1, y.shape[1]), device="cuda", dtype=torch.float64)])
    at = torch.where(inv >= 0, inv, torch.full_like(inv, y.shape[0] - 1)).long().view(T, k)
    t = y[at]
    if w is not None:
        t = t * torch.where(inv.view(T, k) >= 0, w.double(), torch.zeros_like(w.double()))[:, :, None]
    return t.sum(1), t.abs().sum(1)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_unpermute_and_permute_backward(T, k, H, dtype):
    for drop, spare in ((0.0, 0), (0.5, 4)):
        inv, rows = positions(T + 2 * k, T, k, drop, spare)
        y = rnd(3, (rows, H + 8), dtype)[:, :H]
        w = torch.rand((T, k), generator=gen(4), device="cuda") - 0.3
        # k products and sums in float32, one rounding to the rows' type
        for got, ww in ((m.unpermute(y, inv, w), w), (m.permute_backward(y, inv, T), None)):
            s, a = combine(y, inv, ww, T)
            bound = (k + 1) * U32 * a
            ref.check(got, s, bound + ref.HALF[dtype] * (s.abs() + bound), f"{drop} {ww is not None}")
            empty = (inv.view(T, k) < 0).all(1)
            assert (got[empty] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_unpermute_backward(T, k, H, dtype):
    for drop, spare in ((0.0, 0), (0.5, 4)):
        inv, rows = positions(T + 3 * k, T, k, drop, spare)
        y = rnd(5, (rows, H + 8), dtype)[:, :H]
        dout = rnd(6, (T, H + 24), dtype)[:, :H]
        w = torch.rand((T, k), generator=gen(7), device="cuda") - 0.3
        here = inv >= 0
        named = inv[here].long()
        before = torch.full_like(y, 3.0)
        if before.stride() != y.stride():
            before = torch.empty_strided(y.shape, y.stride(), dtype=dtype, device="cuda").fill_(3.0)
        dy, dw = m.unpermute_backward(dout, y, inv, w, out=before)
        want = torch.full((rows, H), 3.0, device="cuda", dtype=dtype)
        # one float32 product, rounded: the same bits
        want[named] = (dout.float().repeat_interleave(k, 0) * w.view(-1, 1))[here].to(dtype)
        assert dy is before and torch.equal(dy, want)
        d, v = dout.double().repeat_interleave(k, 0)[here], y.double()[named]
        rw = torch.zeros(T * k, device="cuda", dtype=torch.float64)
        bw = torch.zeros_like(rw)
        rw[here] = (d * v).sum(1)
        bw[here] = (H + 2) * U32 * (d * v).abs().sum(1)
        ref.check(dw.view(-1), rw, bw, "dw")
        assert (dw.view(-1)[~here] == 0).all()
        # in y's place
        own = y.clone(memory_format=torch.contiguous_format)
        keep = own.clone()
        dy2, dw2 = m.unpermute_backward(dout, own, inv, w, out=own)
        assert dy2 is own and torch.equal(own[named], want[named]) and torch.equal(dw2, dw)
        rest = torch.ones(rows, dtype=torch.bool, device="cuda")
        rest[named] = False
        assert torch.equal(own[rest], keep[rest])


def test_gradients_against_differences():
    """Both are linear in y and in w: a difference is the gradient, up to the rounding of the sums it is taken of."""
    T, k, H = 12, 3, 64
    inv, rows = positions(8, T, k, 0.2, 2)
    y, dout = rnd(9, (rows, H), F32), rnd(10, (T, H), F32)
    w = torch.rand((T, k), generator=gen(11), device="cuda") + 0.1
    dy, dw = m.unpermute_backward(dout, y, inv, w, out=torch.zeros_like(y))

    def f(yy, ww):
        return (m.unpermute(yy, inv, ww).double() * dout.double()).sum().item()
    step_y, step_w = rnd(12, (rows, H), F32), rnd(13, (T, k), F32)
    noise = 4 * (k + 1) * U32 * (combine(y.abs() + step_y.abs(), inv, w.abs() + step_w.abs(), T)[1] * dout.abs()).sum().item()
    slope = (f(y + step_y, w) - f(y - step_y, w)) / 2
    # (y + step rounds in float32 too: half a step of every element)
    assert abs(slope - (dy.double() * step_y.double()).sum().item()) <= 2 * noise
    slope = (f(y, w + step_w) - f(y, w - step_w)) / 2
    assert abs(slope - (dw.double() * step_w.double()).sum().item()) <= 2 * noise
    x = rnd(14, (T, H), F32)
    dx = m.permute_backward(dy, inv, T)
    moved, _ = m.permute(x, inv, out=torch.zeros_like(y))
    assert abs((moved.double() * dy.double()).sum().item() - (dx.double() * x.double()).sum().item()) <= \
        noise + 4 * (k + 1) * U32 * (moved.double() * dy.double()).abs().sum().item()


def test_values_that_are_not_finite_stay_where_they_are():
    T, k, H = 6, 2, 128
    inv = torch.tensor([0, 1, 2, -1, 3, 4, -1, -1, 5, 6, 7, 8], dtype=torch.int32, device="cuda")
    y = rnd(15, (10, H), BF16)
    y[9] = float("nan")                                   # a row of no slot
    y[2, 5] = float("inf")
    w = torch.rand((T, k), generator=gen(16), device="cuda") + 0.1
    w.view(-1)[3] = float("nan")                          # a weight of no row
    w.view(-1)[6] = float("inf")
    out = m.unpermute(y, inv, w)
    assert torch.isinf(out[1, 5]) and torch.isfinite(out).sum() == T * H - 1
    assert (out[3] == 0).all()
    dout = rnd(17, (T, H), BF16)
    dout[3] = float("nan")                                # a token without rows
    dy, dw = m.unpermute_backward(dout, y, inv, w, out=torch.zeros_like(y))
    assert torch.isfinite(dy).all() and (dw.view(-1)[[3, 6, 7]] == 0).all()
    assert torch.isfinite(dw).sum() == T * k - 1          # (the slot of the infinite row)
    # the type's lowest value under a mask of -1 leaves no trace
    y[9] = torch.finfo(BF16).min
    assert torch.isfinite(m.unpermute(y, inv, w)).sum() == T * H - 1


def test_positions_outside_the_rows_are_left_out():
    inv = torch.tensor([0, 5, -1, -2147483648, 2147483647, 2], dtype=torch.int32, device="cuda")
    x = rnd(18, (3, 64), F32)
    out = torch.zeros((3, 64), device="cuda")
    m.permute(x, inv, out=out)
    assert torch.equal(out, torch.stack([x[0], torch.zeros_like(x[0]), x[2]]))
    w = torch.ones((3, 2), device="cuda")
    assert torch.equal(m.unpermute(out, inv, w), torch.stack([x[0], torch.zeros_like(x[0]), x[2]]))
    dy, dw = m.unpermute_backward(x, out, inv, w, out=torch.zeros_like(out))
    assert torch.equal(dy, torch.stack([x[0], torch.zeros_like(x[0]), x[2]]))
    assert (dw.view(-1)[1:5] == 0).all()


def test_no_tokens_and_no_rows():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    y, _ = m.permute(torch.empty((0, 64), device="cuda"), none)
    assert y.shape == (0, 64)
    assert m.unpermute(torch.empty((0, 64), device="cuda"), none, torch.empty((0, 2), device="cuda")).shape == (0, 64)
    inv = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    x = rnd(19, (3, 64), BF16)
    y, _ = m.permute(x, inv, rows=0)
    assert y.shape == (0, 64)
    assert (m.unpermute(y, inv, torch.ones((3, 2), device="cuda")) == 0).all()
    dy, dw = m.unpermute_backward(x, y, inv, torch.ones((3, 2), device="cuda"))
    assert dy.shape == (0, 64) and (dw == 0).all()


def test_offsets_past_32_bits():
    T, k, H = 70_000, 2, 16384                             # 4.6 GB of sorted rows in bf16
    inv = torch.arange(T * k - 1, -1, -1, dtype=torch.int32, device="cuda")
    x = torch.randint(-30, 30, (T, H), generator=gen(20), device="cuda", dtype=torch.int16).to(BF16)
    y, _ = m.permute(x, inv)
    for t in (0, 1, T // 2, T - 1):
        for j in range(k):
            assert torch.equal(y[T * k - 1 - (t * k + j)], x[t])
    w = torch.full((T, k), 0.5, device="cuda")
    assert torch.equal(m.unpermute(y, inv, w), x)
    dw = m.unpermute_backward(x, y, inv, w, out=y)[1]
    for t in (0, T // 2, T - 1):                           # (integers below 2^24: exact)
        assert (dw[t] == (x[t].float() ** 2).sum()).all()
    assert torch.equal(y[0], (x[T - 1].float() * 0.5).to(BF16))


def test_replays_in_a_graph_and_runs_on_another_stream():
    T, k, H = 50, 4, 512
    x, y, dout = rnd(21, (T, H), BF16), rnd(22, (T * k, H), BF16), rnd(23, (T, H), BF16)
    w = torch.rand((T, k), generator=gen(24), device="cuda")
    inv, _ = positions(25, T, k)
    other, _ = positions(26, T, k, 0.3)

    def calls():
        p, _ = m.permute(x, inv)
        o = m.unpermute(y, inv, w)
        dy, dw = m.unpermute_backward(dout, y, inv, w)
        return p, o, dy, dw
    calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = calls()
    for i in range(4):
        inv.copy_(other if i % 2 else positions(25, T, k)[0])
        for t in held:
            t.fill_(9.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        named = inv[inv >= 0].long()
        want = calls()
        for n, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a[named], b[named]) if n in (0, 2) else torch.equal(a, b)
    done = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            done[i] = calls()
            torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want = calls()
    torch.cuda.synchronize()
    named = inv[inv >= 0].long()
    for got in done:
        for n, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a[named], b[named]) if n in (0, 2) else torch.equal(a, b)


def test_goes_with_the_routing():
    """route's inv, an id that is out of range among them, moves every slot's row into its expert's run and back."""
    T, k, E, H = 100, 4, 12, 256
    idx = torch.stack([torch.randperm(E, generator=gen(27 + t), device="cuda")[:k] for t in range(T)]).to(torch.int32)
    idx[5, 2] = E + 3
    counts, offsets, perm, inv = m.route(idx, E)
    x = rnd(28, (T, H), F32)
    y, _ = m.permute(x, inv)
    n = int(offsets[-1])
    assert n == T * k - 1
    assert torch.equal(y[:n], x[(perm[:n] // k).long()])
    assert torch.equal(m.permute_backward(y, inv, T), (x * (inv.view(T, k) >= 0).sum(1, keepdim=True)))
