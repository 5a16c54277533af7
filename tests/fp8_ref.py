"""Plain 64-bit forms of the e4m3 products with block scales and of their quantisers, and the bounds their tests use.

A slice of 128 products is summed by one block-scaled MFMA: off by at most 2^-10 of its largest product
(test_gpu_mfma_bound.py), here bounded by the largest factors of either side.  Slices are scaled (two float32 roundings)
and added in float32, so a sum of n slices adds at most (n + 4) u32 of the sum of absolute values; where the MFMA
adds to its accumulator itself that addition is taken as four times as coarse.  Results are rounded once to bf16."""

import torch

import dense_ref as dense
from dense_ref import HALF, U32, act_err, check, dz_gated, dz_linear  # noqa: F401  (the tests' names)

E4M3 = torch.float8_e4m3fn
BLOCK = 2.0 ** -10
BF16 = torch.bfloat16


def codes(v):
    """e4m3 rounding of values in [-448, 448] (float64), saturating; NaN stays."""
    return v.clamp(-448, 448).float().to(E4M3).double()


def f32_scale(top):
    # (a float64 quotient of float32 values rounds to float32 as the exact one does: 53 >= 2 * 24 + 2)
    s = (top.double() / 448.0).float().double()
    return torch.where(s > 0, s, torch.ones_like(s))


def pow2_scale(top):
    """The smallest power of two s >= 2^-126 with top <= 448 s, 1 for 0."""
    m, e = torch.frexp(top.double())
    k = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.ldexp(torch.ones_like(m), torch.where(top > 0, k, torch.zeros_like(k)))


def row_groups(x, scale=f32_scale):
    """(codes as values, scales [R, C/128]) of groups of 128 columns, float64."""
    g = x.double().view(x.shape[0], -1, 128)
    s = scale(g.abs().amax(2))
    return codes(g / s[:, :, None]).view(x.shape), s


def block_groups(w, ue8m0):
    g = w.double().view(*w.shape[:-2], w.shape[-2] // 128, 128, w.shape[-1] // 128, 128)
    s = (pow2_scale if ue8m0 else f32_scale)(g.abs().amax(dim=(-3, -1)))
    return codes(g / s[..., :, None, :, None]).view(w.shape), s


def scale_values(s):
    return torch.exp2(s.double() - 127.0) if s.dtype == torch.uint8 else s.double()


def wide(q, s):
    """Codes [.., N, K] times block scales."""
    return q.view(E4M3).double() * scale_values(s).repeat_interleave(128, -2).repeat_interleave(128, -1)


def wide_rows(q, s):
    return q.view(E4M3).double() * s.double().repeat_interleave(128, 1)


def product(r, c, chained=False):
    """(r c^T, its bound) for r [M, K], c [N, K] dequantised, K padded to slices of 128 from its start."""
    K = r.shape[1]
    n = (K + 127) // 128
    pad = n * 128 - K
    top = [torch.nn.functional.pad(t.abs(), (0, pad)).view(t.shape[0], n, 128).amax(2) for t in (r, c)]
    err = BLOCK * top[0] @ top[1].t() + (n + 4) * (4 if chained else 1) * U32 * (r.abs() @ c.abs().t())
    return r @ c.t(), err


def linear(x, w, bias, res, name):
    """((y, bound), (pre, bound)) from dequantised x and w."""
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U32 * z.abs()
    y = dense.act(name, z)
    ey = dense.SLOPE[name] * ez + act_err(name, z)
    if res is not None:
        y = y + res.double()
        ey = ey + U32 * y.abs()
    h = HALF[BF16]
    return (y, ey + h * (y.abs() + ey)), (z, ez + h * (z.abs() + ez))


def gated(x, w, name):
    z, ez = product(x, w)
    (g, u), (eg, eu) = z.chunk(2, 1), ez.chunk(2, 1)
    a = dense.act(name, g)
    ea = dense.SLOPE[name] * eg + act_err(name, g)
    y = a * u
    ey = ea * (u.abs() + eu) + a.abs() * eu + U32 * y.abs()
    h = HALF[BF16]
    return (y, ey + h * (y.abs() + ey)), (z, ez + h * (z.abs() + ez))


def quantised(v, e, dim):
    """(dequantised, error) of v, known to within e, in groups of 128 along dim with power-of-two scales: where the rounding or
    the scale may fall either way, the error is what lies between."""
    n = v.shape[dim]
    pad = (-n) % 128
    spec = (0, pad) if dim == 1 else (0, 0, 0, pad)
    v, e = (torch.nn.functional.pad(t, spec) for t in (v, e))
    shape = (v.shape[0], -1, 128) if dim == 1 else (-1, 128, v.shape[1])
    k = 2 if dim == 1 else 1
    g, eg = v.reshape(shape), e.reshape(shape)

    def through(t, s):
        return (codes(t / s) * s).reshape(v.shape)
    top, most = g.abs().amax(k, keepdim=True), (g.abs() + eg).amax(k, keepdim=True)
    lo, hi = pow2_scale(torch.where(top > 0, top, most)), pow2_scale(most)
    mid = through(g, hi)
    err = torch.maximum((through(g + eg, hi) - mid).abs(), (through(g - eg, hi) - mid).abs())
    # a group whose largest value may lie on either side of a scale's end
    other = torch.maximum((through(g + eg, lo) - mid).abs(), (through(g - eg, lo) - mid).abs())
    err = torch.maximum(err, other)
    return (mid[:n], err[:n]) if dim == 0 else (mid[:, :n], err[:, :n])


def backward(dz, edz, x, w, bias=False):
    """((dx, bound), (dw, bound)[, (db, bound)]) over one run of rows; w dequantised [cols, K], x bf16 rows."""
    x = x.double()
    h = HALF[BF16]
    zr, er = quantised(dz, edz, 1)
    dx, ex = product(zr, w.t().contiguous(), chained=True)
    ex = ex + er @ w.abs() * (1 + BLOCK)
    zc, ec = quantised(dz, edz, 0)
    xc, _ = quantised(x, torch.zeros_like(x), 0)
    dw, ew = product(zc.t().contiguous(), xc.t().contiguous(), chained=True)
    ew = ew + ec.t() @ xc.abs() * (1 + BLOCK)
    out = [(dx, ex + h * (dx.abs() + ex)), (dw, ew + h * (dw.abs() + ew))]
    if bias:
        db = dz.sum(0)
        eb = edz.sum(0) + (dz.shape[0] + 1) * U32 * dz.abs().sum(0)
        out.append((db, eb + h * (db.abs() + eb)))
    return out
