"""The e4m3 products where the choice of a kernel, a tile height or a split changes with the sizes: few rows and their scales in LDS, both
gradients of one launch with every pair of heights and with splits, runs in tiles of 256 rows."""

import ctypes

import pytest
import torch

import fp8_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_fp8 import ACT, BF16, by_expert, rnd, rows, runs, weights

pytestmark = pytest.mark.gpu


# rows to 8, 16, 32 and 64 to a kernel; four waves to 4096 inputs, eight beyond; rows x slices to 4096
FEW = [(8, 128, 128), (9, 512, 256), (16, 4096, 128), (16, 4224, 128), (31, 4096, 256), (33, 4096, 128), (47, 1152, 384), (64, 8192, 128),
       (64, 8320, 128), (65, 256, 128), (32, 16384, 128), (32, 16512, 128), (8, 65536, 128), (9, 65536, 128)]


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", FEW)
def test_few_rows(T, K, N, ue8m0):
    q, s = rows(60, T, K)
    x = ref.wide_rows(q, s)
    wq, ws = weights(61, (N, K), ue8m0)
    res = rnd(62, (T, N))
    y, _ = m.linear_fp8(q, s, wq, ws, residual=res)
    ref.check(y, *ref.linear(x, ref.wide(wq, ws), None, res, "none")[0], "y")
    gq, gs = weights(63, (2 * N, K), ue8m0)
    a, pre = m.gated_linear_fp8(q, s, gq, gs, save_pre=True)
    want, wpre = ref.gated(x, ref.wide(gq, gs), "silu")
    ref.check(a, *want, "a")
    ref.check(pre, *wpre, "pre")


def test_rows_that_are_not_there_hold_nothing():
    """What calls with NaN in every row left on the chip enters no row of a later call with fewer rows."""
    K, N = 2048, 512
    wq, ws = weights(64, (N, K), False)
    gq, gs = weights(65, (2 * N, K), False)
    bad = torch.full((64, K), 0x7f, dtype=torch.uint8, device="cuda")
    nan = torch.full((64, K // 128), float("nan"), device="cuda")
    for T in (1, 3, 9, 17, 33):
        q, s = rows(66 + T, T, K)
        for n in (8, 16, 32, 64):
            assert m.linear_fp8(bad[:n], nan[:n], wq, ws)[0].isnan().all()
        y, _ = m.linear_fp8(q, s, wq, ws)
        a, _ = m.gated_linear_fp8(q, s, gq, gs)
        x = ref.wide_rows(q, s)
        ref.check(y, *ref.linear(x, ref.wide(wq, ws), None, None, "none")[0], f"{T} rows y")
        ref.check(a, *ref.gated(x, ref.wide(gq, gs), "silu")[0], f"{T} rows a")


# contractions in splits, tiles of 128 and of 256 rows with a ragged end
TILED = [(100, 7168, 256), (257, 4096, 512), (700, 7168, 256), (2731, 1024, 2816), (4099, 512, 2048)]


@pytest.mark.parametrize("T,K,N", TILED)
def test_forward_splits_and_heights(T, K, N):
    q, s = rows(70, T, K)
    x = ref.wide_rows(q, s)
    wq, ws = weights(71, (N, K), False)
    w = ref.wide(wq, ws)
    bias = rnd(72, (N,))
    ref.check(m.linear_fp8(q, s, wq, ws)[0], *ref.linear(x, w, None, None, "none")[0], "y")
    ref.check(m.linear_fp8(q, s, wq, ws, bias=bias, act=ACT["gelu"])[0], *ref.linear(x, w, bias, None, "gelu")[0], "gelu y")
    a, pre = m.gated_linear_fp8(q, s, wq, ws, save_pre=True)
    want, wpre = ref.gated(x, w, "silu")
    ref.check(a, *want, "a")
    ref.check(pre, *wpre, "pre")


# dx and dw: both of 256 rows; 128 and 256; 256 and 128; 128 and 128; splits of one, the other and both
PAIRED = [(2000, 4096, 2048), (300, 5120, 1536), (4099, 1024, 1408), (1000, 2048, 1024), (136, 1024, 5632), (2983, 1024, 1024), (16384, 512, 512),
          (811, 512, 2048), (60, 512, 4096)]


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N", PAIRED)
def test_gradients_share_a_launch(T, K, N, ue8m0):
    wq, ws = weights(73, (N, K), ue8m0)
    x, dy = rnd(74, (T, K)), rnd(75, (T, N), BF16, 1e-3)
    got = m.linear_fp8_backward(dy, x, wq, ws, need_bias=True)
    want = ref.backward(*ref.dz_linear(dy, None, "none"), x, ref.wide(wq, ws), bias=True)
    for g, (r, b), what in zip(got, want, ("dx", "dw", "db")):
        ref.check(g, r, b, what)


def test_runs_in_tiles_of_256_rows():
    T, K, N, E = 9000, 128, 1280, 4
    q, s = rows(76, T, K)
    off = runs(77, T, E, 8900)
    wq, ws = weights(78, (E, N, K), False)
    gq, gs = weights(79, (E, 2 * N, K), True)
    y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    a = torch.full((T, N), 6.0, dtype=BF16, device="cuda")
    m.linear_fp8(q, s, wq, ws, offsets=off, out=y)
    m.gated_linear_fp8(q, s, gq, gs, offsets=off, out=a)
    last = int(off[-1])
    assert (y[last:] == 5.0).all() and (a[last:] == 6.0).all()
    for e, lo, hi in by_expert(off):
        x = ref.wide_rows(q[lo:hi], s[lo:hi])
        ref.check(y[lo:hi], *ref.linear(x, ref.wide(wq[e], ws[e]), None, None, "none")[0], f"expert {e}")
        ref.check(a[lo:hi], *ref.gated(x, ref.wide(gq[e], gs[e]), "silu")[0], f"expert {e} a")


@pytest.mark.parametrize("T,K,N,E", [(40, 4096, 128, 3), (64, 128, 256, 1024), (3000, 256, 128, 2)])
def test_one_expert_has_all_rows(T, K, N, E):
    """All rows in the last run, the others empty: also gradients, zeros for the experts without rows."""
    q, s = rows(80, T, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = T
    wq, ws = weights(81, (E, N, K), False)
    y, _ = m.linear_fp8(q, s, wq, ws, offsets=off)
    ref.check(y, *ref.linear(ref.wide_rows(q, s), ref.wide(wq[-1], ws[-1]), None, None, "none")[0], "y")
    x, dy = rnd(82, (T, K)), rnd(83, (T, N), BF16, 1e-3)
    dx, dw, _ = m.linear_fp8_backward(dy, x, wq, ws, offsets=off)
    want = ref.backward(*ref.dz_linear(dy, None, "none"), x, ref.wide(wq[-1], ws[-1]))
    ref.check(dx, *want[0], "dx")
    ref.check(dw[-1], *want[1], "dw")
    assert not dw[:-1].any()


@pytest.mark.parametrize("T,K,N,E", [(2983, 1024, 1024, 0), (811, 512, 2048, 0), (136, 1024, 5632, 0), (257, 4096, 512, 0), (1500, 256, 640, 3)])
def test_workspaces_of_exactly_the_size(T, K, N, E):
    """A workspace of the size asked for is enough for a call and each subset of its gradients, and what lies behind it stays."""
    shape = (E, N, K) if E else (N, K)
    off = runs(84, T, E) if E else None      # (all rows belong to experts)
    x, dy = rnd(85, (T, K)), rnd(86, (T, N), BF16, 1e-3)
    q, s = rows(87, T, K)
    stream = torch.cuda.current_stream().cuda_stream
    for ue8m0 in (False, True):
        wq, ws = weights(88, shape, ue8m0)
        p = m.Fp8Problem(T, K, N, E, m.SCALE_UE8M0 if ue8m0 else m.SCALE_F32, m.ACT_NONE, 0, 0, 0, 0, 0)
        addr = off.data_ptr() if E else None

        def space(kind):
            n = ctypes.c_size_t()
            assert getattr(m.lib(), "moe_linear_fp8_workspace_size")(ctypes.byref(p), kind, ctypes.byref(n)) == 0
            t = torch.full((n.value + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
            return t, n.value

        work, n = space(0)
        y = torch.empty((T, N), dtype=BF16, device="cuda")
        assert m.lib().moe_linear_fp8(ctypes.byref(p), q.data_ptr(), s.data_ptr(), wq.data_ptr(), ws.data_ptr(), addr, None, None,
                                      y.data_ptr(), None, work.data_ptr(), n, stream) == 0
        assert (work[n:] == 0xa5).all()
        assert torch.equal(y, m.linear_fp8(q, s, wq, ws, offsets=off)[0])
        want = m.linear_fp8_backward(dy, x, wq, ws, offsets=off)
        spans = by_expert(off) if E else [(0, 0, T)]
        w = ref.wide(wq, ws).reshape(-1, N, K)
        sizes = torch.zeros((T, K), dtype=torch.float64, device="cuda"), torch.zeros((max(E, 1), N, K), dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            sizes[0][lo:hi] = dy[lo:hi].double().abs() @ w[e].abs()
            sizes[1][e] = dy[lo:hi].double().abs().T @ x[lo:hi].double().abs()
        sizes = sizes[0], sizes[1].reshape(shape)
        work, n = space(2)
        for dx_too, dw_too in ((True, True), (True, False), (False, True)):
            dx = torch.empty((T, K), dtype=BF16, device="cuda") if dx_too else None
            dw = torch.empty(shape, dtype=BF16, device="cuda") if dw_too else None
            assert m.lib().moe_linear_fp8_backward(ctypes.byref(p), dy.data_ptr(), x.data_ptr(), wq.data_ptr(), ws.data_ptr(), addr, None,
                                                   dx.data_ptr() if dx_too else None, dw.data_ptr() if dw_too else None, None,
                                                   work.data_ptr(), n, stream) == 0
            assert (work[n:] == 0xa5).all()
            # A gradient alone may be split another way: the same at most 128 slices' results, each sum of them off by 2^-24 of
            # what has been added, then two roundings to bf16 of 2^-8 each.  (The codes' own rounding adds at most 2^-4 to each factor.)
            for got, full, size in ((dx, want[0], sizes[0]), (dw, want[1], sizes[1])):
                if got is not None:
                    bound = 2.0 ** -7 * full.double().abs() + 2 * 128 * 2.0 ** -24 * 1.13 * size
                    assert ((got.double() - full.double()).abs() <= bound).all()


def test_refusals_on_the_gpu():
    """Operands that do not fit are refused on the host, before and after a call whose sizes are known."""
    T, K, N, E = 5, 256, 128, 3
    q, s = rows(90, T, K)
    wq, ws = weights(91, (N, K), False)
    gq, gs = weights(92, (E, 2 * N, K), True)
    off = runs(93, T, E)
    half = torch.empty((T, 2 * K), dtype=torch.uint8, device="cuda")
    bad = [
        lambda: m.linear_fp8(q[:, :128], s, wq, ws),                                     # inputs
        lambda: m.linear_fp8(q[:4], s, wq, ws),                                          # rows
        lambda: m.linear_fp8(q.cpu(), s, wq, ws),
        lambda: m.linear_fp8(q, s.cpu(), wq, ws),
        lambda: m.linear_fp8(q, s, wq, ws.cpu()),
        lambda: m.linear_fp8(q, s.double(), wq, ws),
        lambda: m.linear_fp8(q, s, wq, ws.int()),
        lambda: m.linear_fp8(q, s, wq.float(), ws),
        lambda: m.linear_fp8(q.int(), s, wq, ws),
        lambda: m.linear_fp8(q, s, wq, ws.T),                                            # blocks the other way round
        lambda: m.linear_fp8(q, s, wq.T.contiguous().T, ws),
        lambda: m.linear_fp8(q.T.contiguous().T, s, wq, ws),
        lambda: m.linear_fp8(q[:1].expand(T, K), s, wq, ws),                             # rows that overlap
        lambda: m.linear_fp8(half[:, 1:K + 1], s, wq, ws),                               # not on 16 bytes
        lambda: m.linear_fp8(q, s, wq, ws, offsets=off),                                 # one matrix with offsets
        lambda: m.linear_fp8(q, s, wq[None], ws[None]),                                  # experts without
        lambda: m.linear_fp8(q, s, wq, ws, out=torch.empty((T, N), device="cuda")),
        lambda: m.linear_fp8(q, s, wq, ws, bias=rnd(94, (N + 8,))),
        lambda: m.linear_fp8(q, s, wq, ws, act=4),
        lambda: m.linear_fp8(q, s, wq, ws, residual=rnd(95, (T, N)), workspace=torch.empty(16)),
        lambda: m.gated_linear_fp8(q, s, wq, ws),                                        # 128 rows are no two halves
        lambda: m.gated_linear_fp8(q, s, gq, gs),
        lambda: m.gated_linear_fp8(q, s, gq, gs, offsets=off[:-1]),
        lambda: m.gated_linear_fp8(q, s, gq, gs, offsets=off.long()),
        lambda: m.gated_linear_fp8(q, s, gq, gs, offsets=off.cpu()),
        lambda: m.gated_linear_fp8(q, s, gq, gs, offsets=off, act=m.ACT_NONE),
        lambda: m.linear_fp8(None, s, wq, ws),
        lambda: m.linear_fp8(q, s, None, ws),
    ]
    for _ in range(2):
        for i, call in enumerate(bad):
            with pytest.raises(ValueError):
                call()
                print("not refused:", i)
        y, _ = m.linear_fp8(q, s, wq, ws)
        ref.check(y, *ref.linear(ref.wide_rows(q, s), ref.wide(wq, ws), None, None, "none")[0], "y")


# rows of experts in single-token steps: runs of more and fewer than eight rows, more experts than a wave has lanes
FEW_BY_EXPERT = [(1, 256, 128, 60), (5, 256, 128, 3), (17, 4224, 128, 2), (32, 65536, 128, 2), (33, 512, 256, 4), (40, 128, 128, 1024), (64, 4096, 128, 130),
                 (64, 384, 256, 1), (65, 384, 256, 5)]


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,N,E", FEW_BY_EXPERT)
def test_few_rows_by_expert(T, K, N, E, ue8m0):
    q, s = rows(100, T, K)
    off = runs(101, T, E, max(T - 2, 1))
    wq, ws = weights(102, (E, N, K), ue8m0)
    gq, gs = weights(103, (E, 2 * N, K), ue8m0)
    y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    a = torch.full((T, N), 6.0, dtype=BF16, device="cuda")
    m.linear_fp8(q, s, wq, ws, offsets=off, out=y)
    _, pre = m.gated_linear_fp8(q, s, gq, gs, act=m.ACT_GELU, save_pre=True, offsets=off, out=a)
    last = int(off[-1])
    assert (y[last:] == 5.0).all() and (a[last:] == 6.0).all()
    for e, lo, hi in by_expert(off):
        x = ref.wide_rows(q[lo:hi], s[lo:hi])
        ref.check(y[lo:hi], *ref.linear(x, ref.wide(wq[e], ws[e]), None, None, "none")[0], f"expert {e}")
        want, wpre = ref.gated(x, ref.wide(gq[e], gs[e]), "gelu")
        ref.check(a[lo:hi], *want, f"expert {e} a")
        ref.check(pre[lo:hi], *wpre, f"expert {e} pre")


@pytest.mark.parametrize("T", [30, 300])
def test_offsets_are_taken_into_the_rows_and_into_order(T):
    """Few rows and many read the same runs out of offsets that do not fit."""
    K, N, E = 256, 128, 70
    q, s = rows(104, T, K)
    wq, ws = weights(105, (E, N, K), False)
    off = torch.randint(-5, T + 40, (E + 1,), generator=torch.Generator().manual_seed(106)).tolist()
    off = sorted(off)[:50] + off[50:]                       # (in order at first, then not)
    off[0], off[3], off[40], off[E] = 4, -2 ** 31, T // 2, 2 ** 31 - 1
    start, spans = min(max(off[0], 0), T), []
    for e in range(E):
        end = max(start, min(max(off[e + 1], 0), T))
        if end > start:
            spans.append((e, start, end))
        start = end
    assert len(spans) > 5
    y = torch.full((T, N), 5.0, dtype=BF16, device="cuda")
    m.linear_fp8(q, s, wq, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out=y)
    assert (y[:4] == 5.0).all()
    for e, lo, hi in spans:
        x = ref.wide_rows(q[lo:hi], s[lo:hi])
        ref.check(y[lo:hi], *ref.linear(x, ref.wide(wq[e], ws[e]), None, None, "none")[0], f"expert {e}")
