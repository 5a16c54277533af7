"""The dense operators on values that are not finite, or not of their result's usual range: where an output is
infinite, NaN or finite follows the formula in 64 bits, and finite values keep their bounds (dense_ref.py)."""

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_dense import ACT, BF16, F32, rnd

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


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
