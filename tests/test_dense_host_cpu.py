"""Host-side behaviour of the dense operators: workspaces, plans and the binding's conversions (no HIP call is reached)."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_routed_topk_amd as m
from test_dense_abi_cpu import A, L, gated, linear, size

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T", [1, 16, 32])
def test_few_rows_take_a_second_part_only_where_dz_has_one(T):
    """At most 32 bf16 rows take dz in two parts, and x twice, unless dz is a bf16 value exactly: dy itself,
    or what relu keeps of a bf16 dy."""
    K, N = 2048, 64

    def need(**kw):
        return size(L.moe_linear_workspace_size, linear(T=T, K=K, N=N, **kw), 1)[1]

    x2 = 2 * T * K * 2                                     # x's copies
    two = need(act=m.ACT_SILU)
    assert need(act=m.ACT_RELU) + x2 <= two and need(act=m.ACT_NONE) + x2 <= two
    assert need(act=m.ACT_RELU, out_dtype=m.F32) == need(act=m.ACT_NONE, out_dtype=m.F32) == two
    assert size(L.moe_gated_linear_workspace_size, gated(T=T, H=K, I=N, act=m.ACT_RELU), 1)[1] > x2


def test_package_imports_on_a_torch_without_gpu_support():
    """Host-only calls (workspace sizes, plans) need no GPU entry points of torch."""
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda_')]: delattr(torch._C, n)\n"
            "import mixture_experts_routed_topk_amd as m\n"
            "p = m.make_problem(4, 128, 128, 4, 2, m.BF16, m.BF16)\n"
            "assert m.workspace_size(p) > 0 and m.plan_describe(p)\n"
            "try: m.linear(torch.zeros(1, 8, dtype=torch.bfloat16), torch.zeros(8, 8, dtype=torch.bfloat16))\n"
            "except ValueError: print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]


@pytest.mark.parametrize("kind,fields", [
    (m.NormProblem, (1, 2 ** 32 + 128, m.BF16, 1e-6, 0, 0, 0, 0)),
    (m.LinearProblem, (1, 64, 2 ** 32 + 8, m.BF16, m.BF16, 0, 0, 0, 0, 0, 0)),
    (m.LinearProblem, (1, 2 ** 32 + 64, 8, m.BF16, m.BF16, 0, 0, 0, 0, 0, 0)),
    (m.LinearProblem, (1, 64, 8, m.BF16, m.BF16, 2 ** 32, 0, 0, 0, 0, 0)),
    (m.GatedProblem, (1, 64, 2 ** 32 + 8, m.BF16, m.ACT_SILU, 0, 0, 0, 0)),
    (m.NormProblem, (2 ** 64 + 4, 128, m.BF16, 1e-6, 0, 0, 0, 0))])
def test_sizes_that_wrap_are_refused(kind, fields):
    """A C struct's fields keep the low bits of what is put in: a row of 2^32 + 128 elements is not one of 128."""
    with pytest.raises(ValueError):
        m._problem(kind, fields)


@pytest.mark.parametrize("T", [3, 700, 100_000])
def test_workspace_without_a_bias_gradient(T):
    """The partial sums of dbias, eight rows each, are taken only where dbias is asked for."""
    for fn, call, p, cols in ((L.moe_linear_workspace_size, L.moe_linear_backward, linear(T=T, N=64, act=m.ACT_SILU), 64),
                              (L.moe_gated_linear_workspace_size, L.moe_gated_linear_backward, gated(T=T), 128)):
        full, less = size(fn, p, 1)[1], size(fn, p, 2)[1]
        assert 0 < less <= full - (T + 7) // 8 * cols * 4
        args = [A] * 6 + [None, A]                                   # dy, x, w, pre, dx, dw, dbias, workspace
        assert call(ctypes.byref(p), *args, less - 1, None) == 4
        args[6] = A
        assert call(ctypes.byref(p), *args, less, None) == 4


class Elsewhere(torch.Tensor):
    """A host tensor that says it is on a GPU: enough for the checks that come before any GPU call."""
    gpu = 0
    device = property(lambda self: torch.device("cuda", self.gpu))

    def get_device(self):
        return self.gpu


def on(gpu, *shape, dtype=torch.uint8):
    t = torch.zeros(shape, dtype=dtype).as_subclass(Elsewhere)
    t.gpu = gpu
    return t


@pytest.mark.parametrize("which", range(10))
def test_quantized_forward_refuses_tensors_of_several_gpus(which):
    """Every tensor of a call on one GPU (that of hidden_q), the caller's out and workspace among them."""
    T, H, I, E, k = 4, 128, 128, 2, 2
    f32, i32 = torch.float32, torch.int32
    spec = [((T, H), torch.uint8), ((T, 1), f32), ((T, k), i32), ((T, k), f32), ((E, 2 * I, H), torch.uint8),
            ((E, H, I), torch.uint8), ((E, 2, 1), f32), ((E, 1, 1), f32), ((T, H), torch.bfloat16), ((1 << 20,), torch.uint8)]
    if which == 0:                                            # all but hidden_q
        args = [on(int(i > 0), *s, dtype=d) for i, (s, d) in enumerate(spec)]
    else:
        args = [on(int(i == which), *s, dtype=d) for i, (s, d) in enumerate(spec)]
    with pytest.raises(ValueError, match="cuda:"):
        m.experts_forward_quantized(*args[:8], out=args[8], workspace=args[9])
