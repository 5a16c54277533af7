"""Plain 64-bit forms of the dense operators and the error bounds their tests use.

u32 = 2^-24 and, by type, HALF = half a step relative to a value (bf16 2^-8, float32 2^-24).
A float32 sum of n products, in any order, is off by at most (n + 1) u32 sum|products|
(each product and each of at most n additions rounds once).  An activation adds a few
float32 roundings: ACT covers 16 of them and, for silu and gelu on exp, the |z| u32 by
which a rounded argument moves exp(z).  Each output is then rounded once to its type."""

import math

import torch

U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
ACTS = ("none", "silu", "gelu", "relu")
SLOPE = {"none": 1.0, "silu": 1.1, "gelu": 1.13, "relu": 1.0}   # largest |act'(z)|


def act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z.clamp(min=0.0) if name == "relu" else z


def slope(name, z):
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * torch.sigmoid(-z))
    if name == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return (z > 0).to(z.dtype) if name == "relu" else torch.ones_like(z)


def act_err(name, z):
    """|computed act(z) - act(z)| for an exact z, and the same bound for the slope."""
    return torch.zeros_like(z) if name in ("none", "relu") else (16 + 4 * z.abs()) * U32 * (1 + z.abs())


def product(r, c):
    """(r c^T, bound on a float32 evaluation's error) in 64 bits; r [M,K], c [N,K]."""
    return r @ c.t(), (r.shape[1] + 1) * U32 * (r.abs() @ c.abs().t())


def linear(x, w, bias, res, name, dtype, odt):
    x, w = x.double(), w.double()
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U32 * z.abs()
    y = act(name, z)
    ey = SLOPE[name] * ez + act_err(name, z)
    if res is not None:
        y = y + res.double()
        ey = ey + U32 * y.abs()
    return (y, ey + HALF[odt] * (y.abs() + ey)), (z, ez + HALF[dtype] * (z.abs() + ez))


def gated(x, w, bias, name, dtype):
    x, w = x.double(), w.double()
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + U32 * z.abs()
    g, u = z.chunk(2, 1)
    eg, eu = ez.chunk(2, 1)
    a = act(name, g)
    ea = SLOPE[name] * eg + act_err(name, g)
    y = a * u
    ey = ea * (u.abs() + eu) + a.abs() * eu + U32 * y.abs()
    return (y, ey + HALF[dtype] * (y.abs() + ey)), (z, ez + HALF[dtype] * (z.abs() + ez))


def dz_linear(dy, pre, name):
    dy = dy.double()
    if name == "none":
        return dy, torch.zeros_like(dy)
    z = pre.double()
    dz = dy * slope(name, z)
    return dz, dy.abs() * act_err(name, z) + 2 * U32 * dz.abs()


def dz_gated(da, pre, name):
    da = da.double()
    g, u = pre.double().chunk(2, 1)
    dg, du = da * u * slope(name, g), da * act(name, g)
    e = act_err(name, g)
    return (torch.cat([dg, du], 1),
            torch.cat([(da * u).abs() * e + 4 * U32 * dg.abs(), da.abs() * e + 4 * U32 * du.abs()], 1))


def backward(dz, edz, x, w, dtype, two_parts=False):
    """((dx, bound), (dw, bound), (db, bound)): the products take dz rounded to dtype, or in two_parts, the second
    being what that rounding took, rounded in its turn."""
    x, w = x.double(), w.double()
    er = edz + HALF[dtype] ** (2 if two_parts else 1) * (dz.abs() + edz)          # the rounded dz's error
    out = []
    for r, e, c in ((dz, er, w.t()), (dz.t(), er.t(), x.t())):
        p, ep = product(r, c)
        ep = ep * (1 + HALF[dtype]) * (2 if two_parts else 1) + e @ c.abs().t()      # (two parts: twice the terms)
        out.append((p, ep + HALF[dtype] * (p.abs() + ep)))
    db = dz.sum(0)
    eb = edz.sum(0) + (dz.shape[0] + 1) * U32 * dz.abs().sum(0)
    out.append((db, eb + HALF[dtype] * (db.abs() + eb)))
    return out


def norm(x, weight, eps, res, dtype):
    """((y, bound), h, (rstd, bound)); h is exact: one addition rounded once to dtype."""
    h = x.double()
    if res is not None:
        h = (h + res.double()).to(dtype).double()
    H = h.shape[1]
    ms = (h * h).mean(1, keepdim=True) + eps
    rstd = ms ** -0.5
    # the mean's relative error is (H + 3) u32, its root's half of that, and root and quotient round once each
    er = rstd * ((H + 3) / 2 + 4) * U32
    y = h * rstd * weight.double()
    ey = (h * weight.double()).abs() * er + 3 * U32 * y.abs()
    return (y, ey + HALF[dtype] * (y.abs() + ey)), h, (rstd[:, 0], er[:, 0]), (y, ey)


def norm_backward(dy, h, weight, rstd, dh, dtype):
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    H = h.shape[1]
    n, g = h * r, dy * w
    m = (g * n).mean(1, keepdim=True)
    em = (H + 4) * U32 * (g * n).abs().mean(1, keepdim=True)
    dx = r * (g - n * m)
    ex = r * (n.abs() * em + 4 * U32 * (g.abs() + (n * m).abs())) + 2 * U32 * dx.abs()
    if dh is not None:
        dx = dx + dh.double()
        ex = ex + U32 * dx.abs()
    dw = (dy * n).sum(0)
    ew = (h.shape[0] + 4) * U32 * (dy * n).abs().sum(0)
    return (dx, ex + HALF[dtype] * (dx.abs() + ex)), (dw, ew + HALF[dtype] * (dw.abs() + ew))


def check(got, ref, bound, what):
    got = got.double().to(ref.device)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {tuple(ref.shape)}"
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if got.numel():
        # (a result of exactly zero has bound zero: the smallest normal float32 stands in)
        over = ((got - ref).abs() / (bound + 2.0 ** -126)).max().item()
        assert over <= 1.0, f"{what}: {over:.3g} times its bound"
