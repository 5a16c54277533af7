"""Every tile kernel of the dense operators (dense_tiles.py) against the 64-bit plain forms: with bias, activation,
residual and saved projections, on rows inside wider buffers; and every tensor of calls made on several streams at once."""

import ctypes

import pytest
import torch

import dense_ref as ref
import mixture_experts_routed_topk_amd as m
import synth
from dense_tiles import GATED, GRADIENTS, LINEAR
from synth.device import device_layer
from test_gpu_dense import ACT, BF16, F32, linear_case, rnd
from test_gpu_dense_layer import calls, flat, same

pytestmark = pytest.mark.gpu

TYPE = {"bf16": BF16, "f32": F32}


@pytest.mark.parametrize("dtype,T,K,N,tile,split", LINEAR)
def test_linear_tiles(dtype, T, K, N, tile, split):
    dt = TYPE[dtype]
    for odt in dict.fromkeys((dt, F32)):
        for name in ("gelu", "relu", "silu", "none"):
            x, w, b, r = linear_case(T, K, N, dt, odt, True, True, pad=1)
            y, pre = m.linear(x, w, b, r, ACT[name], odt, save_pre=True)
            (ry, by), (rz, bz) = ref.linear(x, w, b, r, name, dt, odt)
            ref.check(y, ry, by, f"y {name} {odt}")
            ref.check(pre, rz, bz, f"pre {name} {odt}")
    y, pre = m.linear(x, w)                            # and with none of them
    assert pre is None
    (ry, by), _ = ref.linear(x, w, None, None, "none", dt, dt)
    ref.check(y, ry, by, "y plain")


@pytest.mark.parametrize("dtype,T,H,I,tile,split", GATED)
def test_gated_tiles(dtype, T, H, I, tile, split):
    dt = TYPE[dtype]
    x, w, b = rnd("x", (T, H), dt, pad=8), rnd("w", (2 * I, H), dt, H ** -0.5), rnd("b", (2 * I,), dt, 0.5)
    for name in ref.ACTS[1:]:
        a, pre = m.gated_linear(x, w, b, ACT[name], save_pre=True)
        (ra, ba), (rz, bz) = ref.gated(x, w, b, name, dt)
        ref.check(a, ra, ba, f"a {name}")
        ref.check(pre, rz, bz, f"pre {name}")
    a, pre = m.gated_linear(x, w, None, ACT[name])
    assert pre is None
    ref.check(a, *ref.gated(x, w, None, name, dt)[0], "a plain")


@pytest.mark.parametrize("dtype,T,K,cols,rx,rw,sx,sw", GRADIENTS)
def test_gradient_tiles(dtype, T, K, cols, rx, rw, sx, sw):
    dt, I = TYPE[dtype], cols // 2
    x, w = rnd("x", (T, K), dt, pad=8), rnd("w", (cols, K), dt, K ** -0.5)
    pre = rnd("z", (T, cols), dt, 1.5, pad=8)
    forms = [("linear gelu", *ref.dz_linear(dy := rnd("dy", (T, cols), dt, pad=8), pre, "gelu"),
              lambda: m.linear_backward(dy, x, w, pre=pre, act=m.ACT_GELU, need_bias=True)),
             ("linear", *ref.dz_linear(dy, None, "none"), lambda: m.linear_backward(dy, x, w, need_bias=True)),
             ("gated silu", *ref.dz_gated(da := rnd("da", (T, I), dt), pre, "silu"),
              lambda: m.gated_linear_backward(da, x, w, pre, need_bias=True))]
    for what, dz, e, call in forms:
        for got, (r, b), name in zip(call(), ref.backward(dz, e, x, w, dt), ("dx", "dw", "db")):
            ref.check(got, r, b, f"{what} {name}")


@pytest.mark.parametrize("dtype,odt", [(BF16, F32), (F32, F32)], ids=["bf16_f32", "f32"])
@pytest.mark.parametrize("T,K,N", [(300, 136, 1000), (3479, 360, 2050)])
def test_linear_outputs_that_are_not_stored_in_pieces(T, K, N, dtype, odt):
    """Rows of y, residual and pre whose pitches are odd, and a float32 residual under an activation."""
    x, w, b, _ = linear_case(T, K, N, dtype, odt, True, False)
    wide = rnd("odd", (T, N + 3), odt)
    for name in ref.ACTS:
        y, pre = m.linear(x, w, b, wide[:, :N], ACT[name], odt, save_pre=True)
        (ry, by), (rz, bz) = ref.linear(x, w, b, wide[:, :N], name, dtype, odt)
        ref.check(y, ry, by, f"y {name}")
        ref.check(pre, rz, bz, f"pre {name}")


def test_every_tensor_of_calls_on_several_streams():
    sets = [calls(T, 512, 264, f"every{i}") for i, T in enumerate((3, 130, 700, 1500))]
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
        bad = [(i, k, j) for i, (g, wnt) in enumerate(zip(got, want)) for k, (out, ref_out) in enumerate(zip(g, wnt))
               for j, (t, r) in enumerate(zip(out, ref_out)) if not same(t, r)]
        assert not bad, f"(set, call, tensor) {bad}"


@pytest.mark.parametrize("T,K,N", [(5, 72, 40), (33, 200, 264), (1030, 264, 520)])
def test_gradients_without_bias_in_their_own_workspace(T, K, N):
    """The workspace of a call without dbias is what it says: the call stays inside, and gives the same gradients."""
    x, w = rnd("x", (T, K), BF16), rnd("w", (N, K), BF16, K ** -0.5)
    dy, pre = rnd("dy", (T, N), BF16), rnd("z", (T, N), BF16)
    p = m.LinearProblem(T, K, N, m.BF16, m.BF16, m.ACT_SILU, 0, 0, 0, 0, 0)
    n = ctypes.c_size_t(0)
    assert m.lib().moe_linear_workspace_size(ctypes.byref(p), 2, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    assert m.lib().moe_linear_backward(ctypes.byref(p), dy.data_ptr(), x.data_ptr(), w.data_ptr(), pre.data_ptr(), dx.data_ptr(),
                                       dw.data_ptr(), None, ws.data_ptr(), n.value,
                                       torch.cuda.current_stream().cuda_stream) == 0
    full = m.linear_backward(dy, x, w, pre=pre, act=m.ACT_SILU, need_bias=True)
    assert same(dx, full[0]) and same(dw, full[1]) and bool((ws[n.value:] == 0xA5).all())
    for a, b in zip(m.linear_backward(dy, x, w, pre=pre, act=m.ACT_SILU)[:2], full):
        assert same(a, b)


@pytest.mark.parametrize("T", [1, 200])
def test_stage_events_of_the_quantised_forward(T):
    """moe_experts_forward_quantized records the events of the stages it runs, and leaves the row quantisation's as they were."""
    D = device_layer(synth.Spec("stages", T=T, H=384, I=256, E=8, k=2, act="bf16", weight="fp8", scale="f32", seed=9))
    args = (D["idx"], D["w"], D["w_gate_up"], D["w_down"], D["w_gate_up_scale"], D["w_down_scale"])
    q, s = m.quantize_rows_fp8(D["x"])
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2 * len(m.STAGES))]
    recorded = {}
    for name, call in (("forward", lambda: m.experts_forward(D["x"], *args)),
                       ("quantized", lambda: m.experts_forward_quantized(q, s, *args))):
        for e in events:
            e.record()
        torch.cuda.synchronize()
        mid = torch.cuda.Event(enable_timing=True)
        mid.record()
        m.set_stage_events([e.cuda_event for e in events])
        try:
            call()
        finally:
            m.set_stage_events(None)
        torch.cuda.synchronize()
        again = [mid.elapsed_time(e) > 0 for e in events]
        assert again[::2] == again[1::2]
        recorded[name] = {stage for stage, a in zip(m.STAGES, again[::2]) if a}
    assert {"gate_up", "down", "finalize"} < recorded["forward"]
    assert recorded["forward"] - recorded["quantized"] == {"quant_x"} and recorded["quantized"] < recorded["forward"]
