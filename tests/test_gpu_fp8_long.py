"""Gradients of gated e4m3 products whose dz is so wide that dx's contraction has more than 704 slices: the float32 scales of two tiles' blocks
do not fit in LDS beside the slices of 128-row tiles.  The blocks' scales are small but for the last slices', which differ from tile to tile.
And such a gate's weights to e4m3 blocks."""

import ctypes

import pytest
import torch

import fp8_ref as ref
import mixture_experts_routed_topk_amd as m
from test_gpu_fp8 import BF16, gen, rnd

pytestmark = pytest.mark.gpu


def dx_alone(da, x, wq, ws, off, pre, E, I):
    T, K = x.shape
    p = m.Fp8Problem(T, K, I, E, m.SCALE_UE8M0 if ws.dtype == torch.uint8 else m.SCALE_F32, m.ACT_SILU, 0, 0, 0, 0, 0)
    n = ctypes.c_size_t(0)
    assert m.lib().moe_gated_linear_fp8_workspace_size(ctypes.byref(p), 1, ctypes.byref(n)) == 0
    work = torch.full((n.value + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    dx = torch.empty((T, K), dtype=BF16, device="cuda")
    assert m.lib().moe_gated_linear_fp8_backward(ctypes.byref(p), da.data_ptr(), None, wq.data_ptr(), ws.data_ptr(),
                                                 None if off is None else off.data_ptr(), pre.data_ptr(), dx.data_ptr(), None,
                                                 work.data_ptr(), n.value, torch.cuda.current_stream().cuda_stream) == 0
    assert (work[n.value:] == 0xa5).all()
    return dx


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("T,K,I,E", [(300, 65536, 45184, 0), (300, 65536, 45056, 0), (160, 512, 45184, 150), (160, 512, 65536, 150), (300, 32768, 65536, 0)])
def test_dx_of_a_wide_gate(T, K, I, E, ue8m0):
    shape = ((E,) if E else ()) + (2 * I, K)
    wq = torch.randint(0, 0x7f, shape, generator=gen(1), device="cuda", dtype=torch.uint8)
    k = torch.randint(-3, 4, (*shape[:-2], 2 * I // 128, K // 128), generator=gen(2), device="cuda")
    k[..., :-4, :] -= 16                                  # (a scale for each 128 of the contraction and 128 columns of dx)
    ws = (k + 120).to(torch.uint8) if ue8m0 else torch.ldexp(torch.full((1,), 1.25, device="cuda"), k - 7)
    da, pre = rnd(3, (T, I)), rnd(4, (T, 2 * I))
    x = torch.empty((T, K), dtype=BF16, device="cuda")
    off = None
    if E:                                                 # a row for each, the last has what is left
        off = torch.arange(E + 1, dtype=torch.int32, device="cuda")
        off[-1] = T
    dx = dx_alone(da, x, wq, ws, off, pre, E, I)
    dz, edz = ref.dz_gated(da, pre, "silu")
    i = torch.arange(64, device="cuda")                   # columns of both halves of the tiles
    some = (i * (K // 64) + 130 * (i & 1)) % K
    o = off.tolist() if E else [0, T]
    for e in range(len(o) - 1):
        if E and 40 <= e < E - 2:
            continue
        q, s = (wq[e], ws[e]) if E else (wq, ws)
        w = q[:, some].view(ref.E4M3).double() * ref.scale_values(s)[:, some // 128].repeat_interleave(128, 0)
        rows = slice(o[e], o[e + 1])
        zr, er = ref.quantised(dz[rows], edz[rows], 1)
        want, err = ref.product(zr, w.t().contiguous(), chained=True)
        err = err + er @ w.abs() * (1 + ref.BLOCK)
        ref.check(dx[rows][:, some], want, err + ref.HALF[BF16] * (want.abs() + err), f"expert {e}")


@pytest.mark.parametrize("ue8m0", [False, True], ids=["f32", "ue8m0"])
@pytest.mark.parametrize("shape", [(131072, 128), (2, 65792, 256)])
def test_weights_of_a_wide_gate_to_blocks(shape, ue8m0):
    w = rnd(5, shape)
    q, s = m.quantize_blocks_fp8(w, ue8m0)
    g = w.double().view(*shape[:-2], shape[-2] // 128, 128, shape[-1] // 128, 128)
    _, scales = ref.block_groups(w, ue8m0)
    assert torch.equal(ref.scale_values(s), scales)
    quotient = (g / scales[..., :, None, :, None]).float()          # (rounded to float32 before it is to e4m3)
    assert torch.equal(q.view(ref.E4M3).float(), quotient.to(ref.E4M3).float().view(shape))
