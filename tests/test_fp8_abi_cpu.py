"""Host-side checks of the C entry points for rows in expert order and e4m3 products (no HIP call is reached), and the binding's
refusals."""

import ctypes

import pytest
import torch

import mixture_experts_routed_topk_amd as m
from test_dense_host_cpu import on

A = 1 << 20          # a 16-byte aligned address that is never dereferenced
BIG = 1 << 50
L = m.lib()


def perm(**kw):
    d = dict(T=4, rows=8, H=64, k=2, dtype=m.BF16, ldt=0, ldy=0)
    d.update(kw)
    return m.PermuteProblem(**d)


def fp8(**kw):
    d = dict(T=4, K=256, N=128, E=0, scale_fmt=m.SCALE_F32, act=0, ldx=0, ldy=0, ldr=0, ldp=0, lddx=0)
    d.update(kw)
    return m.Fp8Problem(**d)


BAD_PERM = [(dict(T=-1), 2), (dict(T=2 ** 22), 2), (dict(rows=-1), 2), (dict(rows=2 ** 31), 2), (dict(H=0), 2), (dict(H=12), 2),
            (dict(H=65544), 2), (dict(k=0), 2), (dict(k=1025), 2), (dict(ldt=56), 2), (dict(ldt=68), 2), (dict(ldy=60), 2),
            (dict(ldy=2 ** 22 + 8), 2), (dict(dtype=m.FP4_E2M1), 3), (dict(dtype=7), 3)]


@pytest.mark.parametrize("kw,status", BAD_PERM)
def test_permute_refuses(kw, status):
    r = ctypes.byref(perm(**kw))
    assert L.moe_permute(r, A, None, A, A, None, None) == status
    assert L.moe_unpermute(r, A, A, A, A, None) == status
    assert L.moe_unpermute_backward(r, A, A, A, A, A, A, None) == status


def test_permute_pointers():
    r = ctypes.byref(perm())
    assert L.moe_permute(None, A, None, A, A, None, None) == 1
    assert L.moe_unpermute(None, A, A, A, A, None) == 1
    assert L.moe_unpermute_backward(None, A, A, A, A, A, A, None) == 1
    for hole in (0, 2, 3):
        a = [A, None, A, A, None]
        a[hole] = None
        assert L.moe_permute(r, *a, None) == 1
        a[hole] = A + (8 if hole != 2 else 2)
        assert L.moe_permute(r, *a, None) == 2
    assert L.moe_permute(r, A, A, A, A, None, None) == 1                       # scales of one side
    assert L.moe_permute(r, A, A, A, A, A, None) == 3                          # scales of bf16 rows
    codes = perm(dtype=m.FP8_E4M3, H=256)
    assert L.moe_permute(ctypes.byref(codes), A, A + 2, A, A, A, None) == 2
    for bad in (dict(H=192), dict(ldt=264), dict(ldy=264)):
        assert L.moe_permute(ctypes.byref(perm(**{**dict(dtype=m.FP8_E4M3, H=256), **bad})), A, A, A, A, A, None) == 2
    assert L.moe_unpermute(ctypes.byref(codes), A, A, A, A, None) == 3         # codes are not summed
    assert L.moe_unpermute_backward(ctypes.byref(codes), A, A, A, A, A, A, None) == 3
    for hole in (0, 1, 3):
        a = [A, A, A, A]
        a[hole] = None
        assert L.moe_unpermute(r, *a, None) == 1
        a[hole] = A + (8 if hole != 1 else 2)
        assert L.moe_unpermute(r, *a, None) == 2
    for hole in (0, 1, 2):
        a = [A] * 6
        a[hole] = None
        assert L.moe_unpermute_backward(r, *a, None) == 1
    for hole in range(6):
        a = [A] * 6
        a[hole] = A + 2
        assert L.moe_unpermute_backward(r, *a, None) == 2
    zero = ctypes.byref(perm(T=0))
    assert L.moe_permute(zero, *[None] * 6) == 0 and L.moe_unpermute(zero, *[None] * 5) == 0
    assert L.moe_unpermute_backward(zero, *[None] * 7) == 0


BAD_FP8 = [(dict(T=-1), 2), (dict(T=2 ** 22), 2), (dict(K=0), 2), (dict(K=64), 2), (dict(K=200), 2), (dict(K=65664), 2), (dict(N=0), 2),
           (dict(N=192), 2), (dict(N=65664), 2), (dict(E=-1), 2), (dict(E=1025), 2), (dict(ldx=264), 2), (dict(ldx=128), 2),
           (dict(ldy=132), 2), (dict(ldy=120), 2), (dict(ldr=8), 2), (dict(ldp=100), 2), (dict(lddx=260), 2),
           (dict(ldx=2 ** 22 + 16), 2), (dict(T=2 ** 20, K=65536), 2), (dict(T=2 ** 20, N=65536), 2),
           (dict(E=512, K=65536, N=65536), 2), (dict(scale_fmt=0), 3), (dict(scale_fmt=3), 3)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw,status", BAD_FP8 + [(dict(act=4), 3), (dict(act=-1), 3)])
def test_fp8_refuses(kw, status, gated):
    p = ctypes.byref(fp8(**{**dict(act=m.ACT_SILU if gated else 0), **kw}))
    n = ctypes.c_size_t(0)
    if gated:
        assert L.moe_gated_linear_fp8_workspace_size(p, 0, ctypes.byref(n)) == status
        assert L.moe_gated_linear_fp8_workspace_size(p, 1, ctypes.byref(n)) == status
        assert L.moe_gated_linear_fp8(p, A, A, A, A, A, A, None, A, BIG, None) == status
        assert L.moe_gated_linear_fp8_backward(p, A, A, A, A, A, A, A, A, A, BIG, None) == status
    else:
        assert L.moe_linear_fp8_workspace_size(p, 0, ctypes.byref(n)) == status
        assert L.moe_linear_fp8_workspace_size(p, 2, ctypes.byref(n)) == status
        assert L.moe_linear_fp8(p, A, A, A, A, A, None, None, A, None, A, BIG, None) == status
        assert L.moe_linear_fp8_backward(p, A, A, A, A, A, A, A, A, None, A, BIG, None) == status


def test_what_goes_with_experts_alone_or_without_them():
    n = ctypes.c_size_t(0)
    assert L.moe_linear_fp8_workspace_size(ctypes.byref(fp8(E=2, act=m.ACT_GELU)), 0, ctypes.byref(n)) == 3
    assert L.moe_gated_linear_fp8_workspace_size(ctypes.byref(fp8(act=0)), 0, ctypes.byref(n)) == 3
    e = ctypes.byref(fp8(E=2))
    assert L.moe_linear_fp8(e, A, A, A, A, A, A, None, A, None, A, BIG, None) == 3           # bias
    assert L.moe_linear_fp8(e, A, A, A, A, A, None, A, A, None, A, BIG, None) == 3           # residual
    assert L.moe_linear_fp8(e, A, A, A, A, A, None, None, A, A, A, BIG, None) == 3           # pre
    assert L.moe_linear_fp8_backward(e, A, A, A, A, A, None, A, A, A, A, BIG, None) == 3     # dbias
    assert L.moe_linear_fp8(e, A, A, A, A, None, None, None, A, None, A, BIG, None) == 1     # no offsets
    assert L.moe_linear_fp8_backward(e, A, A, A, A, None, None, A, A, None, A, BIG, None) == 1


def test_fp8_pointers():
    p, g = ctypes.byref(fp8(T=200)), ctypes.byref(fp8(T=200, act=m.ACT_SILU))
    for hole in (0, 1, 2, 3, 7):                     # x_q, x_scale, w_q, w_scale, y
        a = [A, A, A, A, None, None, None, A, None]  # (x_q .. w_scale, offsets, bias, residual, y, pre)
        a = a[:4] + [None] + a[5:]
        a[hole] = None
        assert L.moe_linear_fp8(p, *a, A, BIG, None) == 1
        a[hole] = A + 2
        assert L.moe_linear_fp8(p, *a, A, BIG, None) == 2
    for hole in (0, 1, 2, 3, 5):
        a = [A, A, A, A, None, A, None]
        a[hole] = None
        assert L.moe_gated_linear_fp8(g, *a, A, BIG, None) == 1
        a[hole] = A + 2
        assert L.moe_gated_linear_fp8(g, *a, A, BIG, None) == 2
    for hole in (0, 1, 2, 3, 5, 8):                  # da, x, w, w_scale, pre, workspace
        a = [A, A, A, A, None, A, A, A, A]
        a[hole] = None
        assert L.moe_gated_linear_fp8_backward(g, *a, BIG, None) == 1
        a[hole] = A + 2
        assert L.moe_gated_linear_fp8_backward(g, *a, BIG, None) == 2
    n = ctypes.c_size_t(0)
    assert L.moe_linear_fp8_workspace_size(p, 1, None) == 1 and L.moe_gated_linear_fp8_workspace_size(None, 1, ctypes.byref(n)) == 1
    assert L.moe_linear_fp8_workspace_size(p, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert L.moe_linear_fp8_backward(p, A, A, A, A, None, None, A, A, A, A, n.value - 1, None) == 4
    less = ctypes.c_size_t(0)
    assert L.moe_linear_fp8_workspace_size(p, 2, ctypes.byref(less)) == 0 and less.value < n.value
    e = ctypes.byref(fp8(T=200, E=3))
    assert L.moe_linear_fp8_workspace_size(e, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert L.moe_linear_fp8(e, A, A, A, A, A, None, None, A, None, A, n.value - 1, None) == 4
    none = ctypes.byref(fp8(T=0))
    assert L.moe_linear_fp8(none, *[None] * 10, 0, None) == 0
    assert L.moe_linear_fp8_backward(none, *[None] * 10, 0, None) == 0


def test_blocks_refuse():
    def call(w=A, dtype=m.BF16, count=1, N=128, K=128, fmt=m.SCALE_F32, q=A, s=A):
        return L.moe_quantize_blocks_fp8(w, dtype, count, N, K, fmt, q, s, None)
    for kw, status in ((dict(w=None), 1), (dict(q=None), 1), (dict(s=None), 1), (dict(w=A + 8), 2), (dict(q=A + 4), 2), (dict(s=A + 2), 2),
                       (dict(dtype=m.FP8_E4M3), 3), (dict(fmt=0), 3), (dict(count=-1), 2), (dict(count=1025), 2), (dict(N=64), 2),
                       (dict(K=130), 2), (dict(N=65664), 2), (dict(count=1024, N=65536, K=65536), 2)):
        assert call(**kw) == status, kw
    assert call(count=0, w=None, q=None, s=None) == 0


def test_binding_refuses():
    u8, f32, bf = torch.uint8, torch.float32, torch.bfloat16
    x, s = on(0, 4, 256), on(0, 4, 2, dtype=f32)
    w, ws = on(0, 128, 256), on(0, 1, 2, dtype=f32)
    off = on(0, 3, dtype=torch.int32)
    we, wes = on(0, 2, 128, 256), on(0, 2, 1, 2, dtype=f32)
    bad = [(torch.zeros((4, 256), dtype=u8), s, w, ws, {}, "GPU"), (x.view(bf), s, w, ws, {}, "codes"), (x, on(0, 4, 1, dtype=f32), w, ws, {}, "x_scale"),
           (x, s, on(0, 128, 128), on(0, 1, 1, dtype=f32), {}, "inputs"), (x, s, on(0, 100, 256), ws, {}, "multiples of 128"),
           (x, s, w, on(0, 1, 1, dtype=f32), {}, "w_scale"), (x, s, w, on(0, 1, 2, dtype=bf), {}, "w_scale"), (x, s, we, wes, {}, "w_q"),
           (x, s, w, ws, dict(offsets=off), "w_q"), (x, s, we, wes, dict(offsets=on(0, 2, dtype=torch.int32)), "offsets"),
           (x, s, on(1, 128, 256), ws, {}, "cuda:"), (x, s, w, on(1, 1, 2, dtype=f32), {}, "cuda:"), (x, on(1, 4, 2, dtype=f32), w, ws, {}, "cuda:"),
           (x, s, we, wes, dict(offsets=on(1, 3, dtype=torch.int32)), "cuda:"), (x, s, w, ws, dict(out=on(0, 4, 128, dtype=f32)), "out"),
           (x, s, w, ws, dict(out=on(1, 4, 128, dtype=bf)), "cuda:"), (x, s, w, ws, dict(bias=on(0, 64, dtype=bf)), "bias"),
           (x, s, w, ws, dict(residual=on(0, 4, 64, dtype=bf)), "residual"), (x, s, w, ws, dict(workspace=on(1, 64)), "cuda:|range"),
           (x, s, we, wes, dict(offsets=off, act=m.ACT_GELU), "unsupported|status 3")]
    for a, b, c, d, kw, match in bad:
        with pytest.raises(ValueError, match=match):
            m.linear_fp8(a, b, c, d, **kw)
    with pytest.raises(ValueError, match="multiples of 128"):
        m.gated_linear_fp8(x, s, w, ws)                                         # 128 rows are not two of 128
    y = on(0, 4, 256, dtype=bf)
    with pytest.raises(ValueError, match="bf16"):
        m.linear_fp8_backward(on(0, 4, 128, dtype=bf), on(0, 4, 256, dtype=f32), w, ws)
    with pytest.raises(ValueError, match="dy"):
        m.linear_fp8_backward(on(0, 4, 120, dtype=bf), y, w, ws)
    with pytest.raises(ValueError, match="pre"):
        m.linear_fp8_backward(on(0, 4, 128, dtype=bf), y, w, ws, act=m.ACT_SILU)
    with pytest.raises(ValueError, match="status 2"):                           # x's pitch
        m.linear_fp8_backward(on(0, 4, 128, dtype=bf), on(0, 4, 264, dtype=bf)[:, :256].as_subclass(type(y)), w, ws)
    inv = on(0, 8, dtype=torch.int32)
    for args, kw, match in (((on(0, 4, 64, dtype=bf), on(0, 7, dtype=torch.int32)), {}, "entries"),
                            ((on(0, 4, 64, dtype=bf), on(0, 8, dtype=torch.int64)), {}, "int32"),
                            ((on(0, 4, 64, dtype=bf), on(1, 8, dtype=torch.int32)), {}, "cuda:"),
                            ((on(0, 4, 64, dtype=torch.float16), inv), {}, "bf16 or float32"),
                            ((on(0, 4, 64, dtype=bf), inv), dict(scale=on(0, 4, 1, dtype=f32)), "e4m3"),
                            ((on(0, 4, 256), inv), dict(scale=on(0, 4, 1, dtype=f32)), "scale"),
                            ((on(0, 4, 64, dtype=bf), inv), dict(out=on(0, 8, 64, dtype=f32)), "out"),
                            ((torch.zeros((4, 64), dtype=bf), inv), {}, "GPU")):
        with pytest.raises(ValueError, match=match):
            m.permute(*args, **kw)
    with pytest.raises(ValueError, match="topk_w"):
        m.unpermute(on(0, 8, 64, dtype=bf), inv, on(0, 4, 3, dtype=f32))
    with pytest.raises(ValueError, match="bf16 or float32"):
        m.unpermute(on(0, 8, 64), inv, on(0, 4, 2, dtype=f32))
    with pytest.raises(ValueError, match="y must be"):
        m.unpermute_backward(on(0, 4, 64, dtype=bf), on(0, 8, 64, dtype=f32), inv, on(0, 4, 2, dtype=f32))
    with pytest.raises(ValueError, match="multiples of 128"):
        m.quantize_blocks_fp8(on(0, 128, 100, dtype=bf))
    with pytest.raises(ValueError, match="bf16 or float32"):
        m.quantize_blocks_fp8(on(0, 128, 128))


def test_sizes_that_wrap_are_refused():
    for kind, fields in ((m.PermuteProblem, (4, 8, 2 ** 32 + 64, 2, m.BF16, 0, 0)),
                         (m.Fp8Problem, (4, 2 ** 32 + 128, 128, 0, m.SCALE_F32, 0, 0, 0, 0, 0, 0))):
        with pytest.raises(ValueError):
            m._problem(kind, fields)
