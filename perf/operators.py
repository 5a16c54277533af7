"""The dense operators around the routed experts, as cases to be measured and compared.

Around the routed experts of a mixture-of-experts layer stand a root-mean-square norm in
front of the layer, the router's projection, and the experts that every token takes (the
shared experts: a gated projection and a down projection).  A case is one call of one of them:

  norm       y = h * rstd * weight, h = x + residual (stored in x's type), rstd = (mean h^2 + eps)^-1/2
  norm_fp8   the same, y as e4m3 codes with one float32 scale per row and 128 columns
  norm_bwd   gradients of x (= of residual) and of weight, from dy and the gradient that reaches h
  linear     y = act(x w^T + bias) + residual, y in x's type or float32
  linear_bwd gradients of x, w and bias, from dy and the saved x w^T + bias
  gated      a = act(x w_gate^T + bias_gate) * (x w_up^T + bias_up), w_gate_up = [w_gate; w_up]
  gated_bwd  gradients of x, w_gate_up and bias, from da and the saved projections

Types are bf16 or float32; every sum and statistic is held in float32.  Where `own` is true,
run() makes the package's calls; otherwise it evaluates the formulas with elementary torch
operations in float32.  exact() evaluates them in float64.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the norm of a decode step: one token each from 16 sequences
        dict(name="norm_decode", op="norm", T=16, H=2048, dtype="bf16", residual=True),
        # prefill in front of e4m3 experts: the norm hands them their codes and scales
        dict(name="norm_fp8_prefill", op="norm_fp8", T=4096, H=7168, dtype="bf16", residual=True),
        # a training step's norm, with the gradient of the residual stream added
        dict(name="norm_backward", op="norm_bwd", T=8192, H=7168, dtype="bf16", residual=True),
        # router logits of a prefill, 256 experts, kept in float32 for the top-k
        dict(name="linear_router", op="linear", T=4096, K=7168, N=256, dtype="bf16", out="f32", act="none",
             bias=False, residual=False),
        # a shared expert's down projection in a decode step, added to the routed experts' output
        dict(name="linear_down_decode", op="linear", T=16, K=1408, N=2048, dtype="bf16", out="same", act="none",
             bias=False, residual=True),
        # the same in a prefill of the wide layer
        dict(name="linear_down_prefill", op="linear", T=8192, K=2048, N=7168, dtype="bf16", out="same", act="none",
             bias=False, residual=True),
        # a float32 layer (used for checking), odd number of tokens
        dict(name="linear_f32", op="linear", T=333, K=1408, N=2048, dtype="f32", out="same", act="relu", bias=True,
             residual=False),
        # training a projection with bias and GELU on a ragged batch
        dict(name="linear_backward", op="linear_bwd", T=2731, K=2048, N=5632, dtype="bf16", out="same", act="gelu",
             bias=True),
        # one token through a shared expert as wide as four routed ones
        dict(name="gated_decode", op="gated", T=1, H=2048, I=5632, dtype="bf16", act="silu", bias=False, pre=False),
        # the wide layer's shared expert in training: projections saved for the backward pass
        dict(name="gated_train", op="gated", T=8192, H=7168, I=2048, dtype="bf16", act="silu", bias=False, pre=True),
        # a ragged training batch through a GeGLU expert with biases
        dict(name="gated_backward_ragged", op="gated_bwd", T=1999, H=2048, I=1408, dtype="bf16", act="gelu", bias=True),
        # the wide layer's shared expert, backward: the largest case
        dict(name="gated_backward", op="gated_bwd", T=8192, H=7168, I=2048, dtype="bf16", act="silu", bias=False),
    ]


def draw(rng):
    def size(lo, hi, step):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        return min(max(v, lo), hi // step * step)

    op = rng.choice(["norm", "norm_fp8", "norm_bwd", "linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd"])
    dtype = "f32" if op != "norm_fp8" and rng.random() < 0.15 else "bf16"
    c = dict(op=op, T=size(1, 8192, 1), dtype=dtype)
    if op.startswith("norm"):
        c.update(H=size(128, 7168, 128 if op == "norm_fp8" else 8), residual=rng.random() < 0.7)
    elif op.startswith("linear"):
        c.update(K=size(64, 7168, 8), N=size(16, 7168, rng.choice([1, 8, 128])), act=rng.choice(["none", "none", "silu", "gelu", "relu"]),
                 bias=rng.random() < 0.5, out="f32" if dtype == "f32" or rng.random() < 0.25 else "same")
        if op == "linear":
            c.update(residual=rng.random() < 0.5)
    else:
        c.update(H=size(64, 7168, 8), I=size(64, 5632, 8), act=rng.choice(["silu", "silu", "gelu", "relu"]),
                 bias=rng.random() < 0.3)
        if op == "gated":
            c.update(pre=rng.random() < 0.5)
    top = work(listed()[-1])
    scale = 16 if dtype == "f32" else 1
    while c["T"] > 1 and (work(c)["flops"] * scale > top["flops"] or work(c)["bytes"] > top["bytes"]):
        c["T"] = c["T"] * 3 // 4
    return c


# ----------------------------------------------------------------------------- inputs

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return t.mul_(std).add_(mean).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, T = case["op"], case["T"]
    s = dict(case)
    if op.startswith("norm"):
        H = case["H"]
        x = _normal(gen, (T, H), torch.float32)
        x[:, gen.initial_seed() % H] *= 30.0          # residual streams carry a few large channels
        s.update(x=x.to(dt), weight=_normal(gen, (H,), dt, 0.1, 1.0))
        if op == "norm_bwd":
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s.update(dy=_normal(gen, (T, H), dt), dh=_normal(gen, (T, H), dt) if case["residual"] else None)
        else:
            s["res"] = _normal(gen, (T, H), dt) if case["residual"] else None
    elif op.startswith("linear"):
        K, N = case["K"], case["N"]
        odt = torch.float32 if case["out"] == "f32" else dt
        s.update(x=_normal(gen, (T, K), dt), w=_normal(gen, (N, K), dt, 1.0 / math.sqrt(K)), odt=odt)
        if op == "linear_bwd":
            s["saved"] = _normal(gen, (T, N), dt) if case["act"] != "none" else None
            s["dy"] = _normal(gen, (T, N), odt)
        else:
            s["b"] = _normal(gen, (N,), dt, 0.1) if case["bias"] else None
            s["res"] = _normal(gen, (T, N), odt) if case["residual"] else None
    else:
        H, I = case["H"], case["I"]
        s.update(x=_normal(gen, (T, H), dt), w=_normal(gen, (2 * I, H), dt, 1.0 / math.sqrt(H)))
        if op == "gated_bwd":
            s.update(saved=_normal(gen, (T, 2 * I), dt), da=_normal(gen, (T, I), dt))
        else:
            s["b"] = _normal(gen, (2 * I,), dt, 0.1) if case["bias"] else None
    return s


def work(case):
    T, e = case["T"], 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op.startswith("norm"):
        H, r = case["H"], case["residual"]
        rows = {"norm": e * (2 + 2 * r), "norm_fp8": e * (1 + 2 * r) + 1 + 4 / 128, "norm_bwd": e * (3 + r)}[op]
        return {"bytes": int(T * H * rows + T * 4 + H * e * (2 if op == "norm_bwd" else 1)),
                "flops": T * H * (10 if op == "norm_bwd" else 6)}
    if op.startswith("linear"):
        K, N, o = case["K"], case["N"], 4 if case["out"] == "f32" else e
        if op == "linear":
            return {"bytes": T * K * e + N * K * e + T * N * o * (1 + case["residual"]) + N * e * case["bias"],
                    "flops": 2 * T * N * K}
        return {"bytes": 2 * T * K * e + 2 * N * K * e + T * N * (o + e * (case["act"] != "none")) + N * e * case["bias"],
                "flops": 4 * T * N * K}
    H, I = case["H"], case["I"]
    if op == "gated":
        return {"bytes": T * H * e + 2 * I * H * e + T * I * e * (1 + 2 * case["pre"]) + 2 * I * e * case["bias"],
                "flops": 4 * T * H * I}
    return {"bytes": 2 * T * H * e + 4 * I * H * e + 3 * T * I * e + 2 * I * e * case["bias"], "flops": 8 * T * H * I}


# ----------------------------------------------------------------------------- the calls

def run(s):
    if own:
        return _own(s)
    return _plain(s)


def _own(s):
    import mixture_experts_routed_topk_amd as m

    op = s["op"]
    if op == "norm":
        y, h, rstd = m.rms_norm(s["x"], s["weight"], EPS, residual=s["res"])
        return {"y": y, "h": h, "rstd": rstd}
    if op == "norm_fp8":
        q, scale, _, h, rstd = m.rms_norm_fp8(s["x"], s["weight"], EPS, residual=s["res"])
        return {"q": q.view(torch.float8_e4m3fn), "scale": scale, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dx, dweight = m.rms_norm_backward(s["dy"], s["x"], s["weight"], s["rstd"], dh=s["dh"])
        return {"dx": dx, "dweight": dweight}
    act = {"none": m.ACT_NONE, "silu": m.ACT_SILU, "gelu": m.ACT_GELU, "relu": m.ACT_RELU}[s["act"]]
    if op == "linear":
        y, _ = m.linear(s["x"], s["w"], bias=s["b"], residual=s["res"], act=act, out_dtype=s["odt"])
        return {"y": y}
    if op == "linear_bwd":
        dx, dw, db = m.linear_backward(s["dy"], s["x"], s["w"], pre=s["saved"], act=act, need_bias=s["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "gated":
        a, pre = m.gated_linear(s["x"], s["w"], bias=s["b"], act=act, save_pre=s["pre"])
        return {"a": a, "pre": pre}
    dx, dw, db = m.gated_linear_backward(s["da"], s["x"], s["w"], s["saved"], act=act, need_bias=s["bias"])
    return {"dx": dx, "dw": dw, "db": db}


def _act(name, z):
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    return z


def _slope(name, z):
    if name == "silu":
        g = 1.0 / (1.0 + torch.exp(-z))
        return g * (1.0 + z * (1.0 - g))
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "relu":
        return (z > 0).to(z.dtype)
    return torch.ones_like(z)


def _plain(s):
    op, x = s["op"], s["x"]
    dt = x.dtype
    if op == "norm" or op == "norm_fp8":
        h = x if s["res"] is None else (x.float() + s["res"].float()).to(dt)
        hf = h.float()
        rstd = 1.0 / torch.sqrt((hf * hf).mean(1) + EPS)
        y = hf * rstd[:, None] * s["weight"].float()
        if op == "norm":
            return {"y": y.to(dt), "h": h, "rstd": rstd}
        g = y.view(y.shape[0], -1, 128)
        top = g.abs().amax(2, keepdim=True)
        scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        return {"q": (g / scale).to(torch.float8_e4m3fn).view(y.shape), "scale": scale[:, :, 0], "h": h, "rstd": rstd}
    if op == "norm_bwd":
        dy, n = s["dy"].float(), x.float() * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(dt), "dweight": (dy * n).sum(0).to(dt)}
    xf, wf = x.float(), s["w"].float()
    if op == "linear":
        z = xf @ wf.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(s["act"], z)
        if s["res"] is not None:
            y = y + s["res"].float()
        return {"y": y.to(s["odt"])}
    if op == "linear_bwd":
        dz = s["dy"].float()
        if s["saved"] is not None:
            dz = dz * _slope(s["act"], s["saved"].float())
        return {"dx": (dz @ wf).to(dt), "dw": (dz.t() @ xf).to(dt), "db": dz.sum(0).to(dt) if s["bias"] else None}
    I = s["I"]
    if op == "gated":
        z = xf @ wf.t()
        if s["b"] is not None:
            z = z + s["b"].float()
        return {"a": (_act(s["act"], z[:, :I]) * z[:, I:]).to(dt), "pre": z.to(dt) if s["pre"] else None}
    gate, up, da = s["saved"][:, :I].float(), s["saved"][:, I:].float(), s["da"].float()
    dz = torch.cat([da * up * _slope(s["act"], gate), da * _act(s["act"], gate)], 1)
    return {"dx": (dz @ wf).to(dt), "dw": (dz.t() @ xf).to(dt), "db": dz.sum(0).to(dt) if s["bias"] else None}


# ----------------------------------------------------------------------------- float64

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op, x = case["op"], f["x"]
    if op in ("norm", "norm_fp8"):
        h = x
        if "res" in f:                                # h is held in x's type: what the norm reads
            h = (x + f["res"]).to(DTYPES[case["dtype"]]).double()
        rstd = (torch.sum(h ** 2, dim=1) / case["H"] + EPS) ** -0.5
        y = torch.einsum("th,t,h->th", h, rstd, f["weight"])
        if op == "norm":
            return {"y": y, "h": h, "rstd": rstd}
        scale = y.reshape(-1, 128).abs().max(dim=1).values / 448.0
        scale[scale == 0] = 1.0
        scale = scale.reshape(case["T"], -1)
        return {"q": y / scale.repeat_interleave(128, dim=1), "scale": scale, "h": h, "rstd": rstd}
    if op == "norm_bwd":
        # dx_j = rstd w_j dy_j - rstd^3 h_j <dy w, h> / H + dh_j
        r, H = f["rstd"][:, None], case["H"]
        along = torch.sum(f["dy"] * f["weight"] * x, dim=1, keepdim=True) / H
        dx = r * f["weight"] * f["dy"] - r ** 3 * x * along
        return {"dx": dx + f["dh"] if "dh" in f else dx, "dweight": torch.sum(f["dy"] * x * r, dim=0)}

    def gate(z):
        if case["act"] == "silu":
            return z * torch.sigmoid(z)
        if case["act"] == "gelu":
            return z * torch.special.ndtr(z)
        return z.clamp(min=0.0) if case["act"] == "relu" else z

    def slope(z):
        if case["act"] == "silu":
            p = torch.sigmoid(z)
            return p + z * p * torch.sigmoid(-z)
        if case["act"] == "gelu":
            return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        return torch.heaviside(z, torch.zeros_like(z[:1, :1])) if case["act"] == "relu" else torch.ones_like(z)

    w = f["w"]
    if op in ("linear", "gated"):
        z = torch.mm(x, w.T) + (f["b"] if "b" in f else 0.0)
        if op == "linear":
            return {"y": gate(z) + (f["res"] if "res" in f else 0.0)}
        g, u = z.chunk(2, dim=1)
        return {"a": gate(g) * u, "pre": z if case["pre"] else None}
    if op == "linear_bwd":
        dz = f["dy"] * slope(f["saved"]) if "saved" in f else f["dy"]
    else:
        g, u = f["saved"].chunk(2, dim=1)
        dz = torch.hstack((f["da"] * u * slope(g), f["da"] * gate(g)))
    return {"dx": torch.mm(dz, w), "dw": torch.mm(dz.T, x), "db": torch.sum(dz, dim=0) if case["bias"] else None}
