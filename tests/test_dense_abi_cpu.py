"""Host-side checks of the dense operators' C entry points (no HIP call is reached) and of the
Python binding's refusals."""

import ctypes

import pytest
import torch

import mixture_experts_routed_topk_amd as m

A = 1 << 20          # a 16-byte aligned address that is never dereferenced
L = m.lib()


def norm(**kw):
    d = dict(T=4, H=256, dtype=m.BF16, eps=1e-6, ldx=0, ldr=0, ldh=0, ldy=0)
    d.update(kw)
    return m.NormProblem(**d)


def linear(**kw):
    d = dict(T=4, K=64, N=60, dtype=m.BF16, out_dtype=m.BF16, act=0, ldx=0, ldy=0, ldr=0, ldp=0, lddx=0)
    d.update(kw)
    return m.LinearProblem(**d)


def gated(**kw):
    d = dict(T=4, H=64, I=64, dtype=m.BF16, act=m.ACT_SILU, ldx=0, lda=0, ldp=0, lddx=0)
    d.update(kw)
    return m.GatedProblem(**d)


def size(fn, p, *args):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(p), *args, ctypes.byref(n)), n.value


BAD_NORM = [(dict(T=-1), 2), (dict(T=2**22), 2), (dict(H=0), 2), (dict(H=4), 2), (dict(H=12), 2), (dict(H=65544), 2),
            (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2), (dict(ldx=248), 2),
            (dict(ldx=260), 2), (dict(ldr=8), 2), (dict(ldh=2**22 + 8), 2), (dict(ldy=-8), 2),
            (dict(dtype=m.FP8_E4M3), 3), (dict(dtype=9), 3)]
BAD_LINEAR = [(dict(T=-1), 2), (dict(T=2**22), 2), (dict(K=0), 2), (dict(K=60), 2), (dict(K=65544), 2), (dict(N=0), 2),
              (dict(N=2**20 + 1), 2), (dict(T=2**15, N=2**20), 2), (dict(T=2**20, K=65536), 2),
              (dict(K=65536, N=2**20), 2), (dict(ldx=68), 2), (dict(ldx=56), 2), (dict(ldy=59), 2), (dict(ldr=2**22 + 1), 2),
              (dict(ldp=-1), 2), (dict(lddx=60), 2), (dict(act=4), 3), (dict(act=-1), 3), (dict(dtype=m.FP4_E2M1), 3),
              (dict(dtype=m.F32), 3), (dict(out_dtype=m.FP8_E4M3), 3)]
BAD_GATED = [(dict(T=-1), 2), (dict(H=60), 2), (dict(I=60), 2), (dict(I=0), 2), (dict(I=65544), 2), (dict(T=2**20, H=65536), 2), (dict(T=2**18, I=65536), 2), (dict(ldx=56), 2),
             (dict(lda=60), 2), (dict(ldp=64), 2), (dict(ldp=132), 2), (dict(lddx=68), 2), (dict(act=0), 3),
             (dict(act=4), 3), (dict(dtype=m.FP8_E4M3), 3)]


@pytest.mark.parametrize("kw,status", BAD_NORM)
def test_norm_refuses(kw, status):
    p = norm(**kw)
    assert size(L.moe_rms_norm_workspace_size, p)[0] == status
    assert L.moe_rms_norm(ctypes.byref(p), A, None, A, A, None, A, None, None, None) == status
    assert L.moe_rms_norm_backward(ctypes.byref(p), A, A, A, A, None, A, A, A, 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", BAD_LINEAR)
def test_linear_refuses(kw, status):
    p = linear(**kw)
    assert size(L.moe_linear_workspace_size, p, 0)[0] == status
    assert size(L.moe_linear_workspace_size, p, 1)[0] == status
    assert L.moe_linear(ctypes.byref(p), A, A, None, None, A, None, A, 1 << 40, None) == status
    assert L.moe_linear_backward(ctypes.byref(p), A, A, A, A, A, A, A, A, 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", BAD_GATED)
def test_gated_refuses(kw, status):
    p = gated(**kw)
    assert size(L.moe_gated_linear_workspace_size, p, 0)[0] == status
    assert L.moe_gated_linear(ctypes.byref(p), A, A, None, A, None, A, 1 << 40, None) == status
    assert L.moe_gated_linear_backward(ctypes.byref(p), A, A, A, A, A, A, A, A, 1 << 40, None) == status


def test_null_and_misaligned_pointers():
    n, l, g = norm(), linear(), gated()
    big = 1 << 40

    def fwd(p, *a):
        return L.moe_rms_norm(ctypes.byref(p), *a, None)

    assert L.moe_rms_norm(None, A, None, A, A, None, A, None, None, None) == 1
    for hole in (0, 2, 3, 5):                                        # x, weight, y (without q), rstd
        a = [A, None, A, A, None, A, None, None]
        a[hole] = None
        assert fwd(n, *a) == 1
    assert fwd(n, A, A, A, A, None, A, None, None) == 1              # a residual without h
    assert fwd(n, A, None, A, A, A, A, None, None) == 1              # h without a residual
    assert fwd(n, A, None, A, A, None, A, A, None) == 1              # codes without scales
    assert fwd(n, A, None, A, A, None, A, None, A) == 1
    assert fwd(norm(H=264), A, None, A, A, None, A, A, A) == 2       # codes need whole 128-column groups
    assert fwd(norm(dtype=m.F32), A, None, A, A, None, A, A, A) == 3
    for hole in (0, 2, 3):
        a = [A, None, A, A, None, A, None, None]
        a[hole] = A + 8
        assert fwd(n, *a) == 2
    assert fwd(n, A, None, A, A, None, A + 2, None, None) == 2

    def bwd(fn, p, *a):
        return fn(ctypes.byref(p), *a, None)

    for hole in (0, 1, 2, 3, 5, 7):                                  # dy, h, weight, rstd, dx, workspace
        a = [A, A, A, A, None, A, A, A, big]
        a[hole] = None
        assert bwd(L.moe_rms_norm_backward, n, *a) == 1
    need = size(L.moe_rms_norm_workspace_size, n)[1]
    assert need > 0
    assert bwd(L.moe_rms_norm_backward, n, A, A, A, A, None, A, A, A, need - 1) == 4

    for hole in (0, 1, 4):                                           # x, w, y
        a = [A, A, None, None, A, None, A, big]
        a[hole] = None
        assert bwd(L.moe_linear, l, *a) == 1
        a[hole] = A + 4
        assert bwd(L.moe_linear, l, *a) == 2
    for hole in (0, 1, 3):                                           # x, w_gate_up, a
        a = [A, A, None, A, None, A, big]
        a[hole] = None
        assert bwd(L.moe_gated_linear, g, *a) == 1
        a[hole] = A + 4
        assert bwd(L.moe_gated_linear, g, *a) == 2
    for fn, p, sz in ((L.moe_linear_backward, linear(act=m.ACT_GELU), L.moe_linear_workspace_size),
                      (L.moe_gated_linear_backward, g, L.moe_gated_linear_workspace_size)):
        for hole in (0, 1, 2, 3, 7):                                 # dy, x, w, pre, workspace
            a = [A, A, A, A, A, A, A, A, big]
            a[hole] = None
            assert bwd(fn, p, *a) == 1
            a[hole] = A + 8
            assert bwd(fn, p, *a) == 2
        need = size(sz, p, 1)[1]
        assert bwd(fn, p, A, A, A, A, A, A, A, A, need - 1) == 4
    assert L.moe_linear_workspace_size(ctypes.byref(l), 0, None) == 1
    assert L.moe_gated_linear_workspace_size(ctypes.byref(g), 1, None) == 1
    assert L.moe_rms_norm_workspace_size(ctypes.byref(n), None) == 1


def test_no_rows_need_no_pointers():
    assert L.moe_rms_norm(ctypes.byref(norm(T=0)), *[None] * 9) == 0
    assert L.moe_linear(ctypes.byref(linear(T=0)), *[None] * 7, 0, None) == 0
    assert L.moe_gated_linear(ctypes.byref(gated(T=0)), *[None] * 6, 0, None) == 0
    assert L.moe_rms_norm_backward(ctypes.byref(norm(T=0)), *[None] * 8, 0, None) == 0
    assert L.moe_linear_backward(ctypes.byref(linear(T=0)), *[None] * 8, 0, None) == 0


def test_quantized_forward_refuses():
    p = m.Problem(4, 128, 128, 4, 2, m.BF16, m.BF16, m.SCALE_NONE, 0)
    call = [A, A, A, A, A, A, A, A, A, A, 1 << 40, None]
    assert L.moe_experts_forward_quantized(ctypes.byref(p), *call) == 3     # bf16 weights
    p = m.Problem(4, 128, 128, 4, 2, m.BF16, m.FP8_E4M3, m.SCALE_F32, 0)
    for hole in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):
        a = list(call)
        a[hole] = None
        assert L.moe_experts_forward_quantized(ctypes.byref(p), *a) == 1
    a = list(call)
    a[1] = A + 4                                                            # scales 16-byte aligned
    assert L.moe_experts_forward_quantized(ctypes.byref(p), *a) == 2
    a = list(call)
    a[10] = 16
    assert L.moe_experts_forward_quantized(ctypes.byref(p), *a) == 4


def test_workspace_grows_with_the_problem_not_with_earlier_calls():
    small, big = linear(T=8), linear(T=4096, act=m.ACT_GELU)
    assert size(L.moe_linear_workspace_size, small, 1) == size(L.moe_linear_workspace_size, small, 1)
    assert size(L.moe_linear_workspace_size, big, 1)[1] > 4096 * 60 * 2


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        m.linear(x, w)
    with pytest.raises(ValueError, match="GPU"):
        m.gated_linear(x, w)
    with pytest.raises(ValueError, match="GPU"):
        m.rms_norm(x, w[0])
    with pytest.raises(ValueError, match="bf16 or float32"):
        m.rms_norm(x.half(), w[0])
    with pytest.raises(ValueError, match="bf16 or float32"):
        m.linear(x.half(), w)
    with pytest.raises(ValueError, match="torch tensor|bf16"):
        m.linear([[1.0]], w)
