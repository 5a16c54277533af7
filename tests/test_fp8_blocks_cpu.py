"""The weights' quantiser takes every matrix that the e4m3 products take: their host-side checks side by side (no HIP call is reached)."""

import ctypes

import pytest

import mixture_experts_routed_topk_amd as m

L = m.lib()


def blocks(N, K, count=1):
    """Whether the sizes pass: the pointers, which are missing, are looked at behind them."""
    status = L.moe_quantize_blocks_fp8(None, m.BF16, count, N, K, m.SCALE_F32, None, None, None)
    assert status in (1, 2)
    return status == 1


def product(N, K, E, gated):
    p = m.Fp8Problem(1, K, N, E, m.SCALE_F32, m.ACT_SILU if gated else 0, 0, 0, 0, 0, 0)
    size = L.moe_gated_linear_fp8_workspace_size if gated else L.moe_linear_fp8_workspace_size
    return size(ctypes.byref(p), 0, ctypes.byref(ctypes.c_size_t(0))) == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("K", [128, 65536, 65664])
@pytest.mark.parametrize("E", [0, 1, 2, 40, 1024, 1025])
def test_the_products_matrices_are_quantised(E, K, gated):
    for N in (128, 32768, 32896, 65408, 65536, 65664):
        if product(N, K, E, gated):
            assert blocks(2 * N if gated else N, K, max(E, 1)), (N, K, E)


def test_sizes_past_the_widest_gate():
    assert blocks(131072, 128) and blocks(65792, 128) and blocks(65536, 65536)
    for N, K in ((131200, 128), (131328, 128), (65664, 128), (131072 + 64, 128), (128, 65664)):
        assert not blocks(N, K), (N, K)
    assert blocks(131072, 65536, 2) and not blocks(131072, 65536, 3)     # 2^34 elements
