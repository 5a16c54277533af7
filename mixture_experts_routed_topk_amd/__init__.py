"""Routed top-k MoE experts forward on MI355X (gfx950): Python binding.

A thin ctypes layer over libmoe_experts.so (declared in include/moe_experts.h).
It only marshals arguments: torch tensors provide device pointers, the current
HIP stream and workspace memory; every step of the forward runs in the library's
HIP kernels.  There is no fallback: if the library is not built, or a tensor is
not on the GPU, the call raises.  Results carry no autograd history, also of tensors
that require gradients: a training loop calls the *_backward functions itself.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional

import torch

__all__ = [
    "experts_forward", "experts_forward_noalloc", "check_scales", "check_mfma_blocks", "route", "route_logits", "quantize_rows_fp8", "workspace_size", "plan_describe",
    "experts_forward_quantized", "rms_norm", "rms_norm_fp8", "rms_norm_backward", "linear", "linear_backward",
    "gated_linear", "gated_linear_backward", "ACT_NONE", "ACT_SILU", "ACT_GELU", "ACT_RELU",
    "Problem", "NormProblem", "LinearProblem", "GatedProblem", "MoeError", "lib", "FLAG_CHECK_INDICES", "FLAG_DETERMINISTIC", "FLAG_ATOMIC_COMBINE", "FLAG_ACT_GELU", "FLAG_ACT_RELU",
    "FLAG_FORCE_GROUPED", "FLAG_FORCE_DECODE", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_experts.so")

# moe_status
OK, ERR_NULL_ARG, ERR_BAD_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_BAD_INDEX, ERR_HIP = range(7)
# moe_dtype
F32, BF16, FP8_E4M3, FP4_E2M1 = 0, 1, 2, 3
# moe_scale_fmt
SCALE_NONE, SCALE_F32, SCALE_UE8M0 = 0, 1, 2
# flags
FLAG_CHECK_INDICES = 1
FLAG_DETERMINISTIC = 2
FLAG_FORCE_GROUPED = 4
FLAG_FORCE_DECODE = 8
FLAG_ATOMIC_COMBINE = 16
FLAG_ACT_GELU = 32
FLAG_ACT_RELU = 64
# moe_act
ACT_NONE, ACT_SILU, ACT_GELU, ACT_RELU = range(4)

EXPORTS = ["moe_abi_version", "moe_status_str", "moe_workspace_size", "moe_experts_forward",
           "moe_route", "moe_route_logits", "moe_quantize_rows_fp8", "moe_plan_describe",
           "moe_set_stage_events", "moe_check_mfma_blocks", "moe_experts_forward_noalloc",
           "moe_noalloc_scratch_bytes", "moe_experts_forward_quantized",
           "moe_rms_norm", "moe_rms_norm_workspace_size", "moe_rms_norm_backward",
           "moe_linear", "moe_linear_workspace_size", "moe_linear_backward",
           "moe_gated_linear", "moe_gated_linear_workspace_size", "moe_gated_linear_backward"]

# stage ids (moe_set_stage_events)
STAGES = ["zero", "route", "quant_x", "gate_up", "quant_act", "down", "finalize"]


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("scale_fmt", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class NormProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldh", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class LinearProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("ldx", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldp", ctypes.c_int64), ("lddx", ctypes.c_int64)]


class GatedProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("lda", ctypes.c_int64), ("ldp", ctypes.c_int64),
                ("lddx", ctypes.c_int64)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"moe status {status}: {msg}")
        self.status = status


_lib = None


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                           "`python -m mixture_experts_routed_topk_amd.build_lib`")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(Problem)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    L.moe_abi_version.restype = ctypes.c_int
    L.moe_abi_version.argtypes = []
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_status_str.argtypes = [ctypes.c_int]
    L.moe_workspace_size.restype = ctypes.c_int
    L.moe_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_experts_forward.restype = ctypes.c_int
    L.moe_experts_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_experts_forward_noalloc.restype = ctypes.c_int
    L.moe_experts_forward_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_noalloc_scratch_bytes.restype = ctypes.c_size_t
    L.moe_noalloc_scratch_bytes.argtypes = []
    L.moe_route.restype = ctypes.c_int
    L.moe_route.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route_logits.restype = ctypes.c_int
    L.moe_route_logits.argtypes = [P, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_quantize_rows_fp8.restype = ctypes.c_int
    L.moe_quantize_rows_fp8.argtypes = [vp, ctypes.c_int64, ctypes.c_int32, vp, vp, vp]
    L.moe_plan_describe.restype = ctypes.c_int
    L.moe_plan_describe.argtypes = [P, ctypes.c_char_p, sz]
    L.moe_check_mfma_blocks.restype = ctypes.c_int
    L.moe_check_mfma_blocks.argtypes = [ctypes.c_int, vp, vp, vp, vp, ctypes.c_int, vp]
    L.moe_experts_forward_quantized.restype = ctypes.c_int
    L.moe_experts_forward_quantized.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    PN, PL, PG = (ctypes.POINTER(c) for c in (NormProblem, LinearProblem, GatedProblem))
    pz = ctypes.POINTER(sz)
    for fn, args in ((L.moe_rms_norm, [PN] + [vp] * 9), (L.moe_rms_norm_workspace_size, [PN, pz]),
                     (L.moe_rms_norm_backward, [PN] + [vp] * 8 + [sz, vp]),
                     (L.moe_linear, [PL] + [vp] * 7 + [sz, vp]),
                     (L.moe_linear_workspace_size, [PL, ctypes.c_int, pz]),
                     (L.moe_linear_backward, [PL] + [vp] * 8 + [sz, vp]),
                     (L.moe_gated_linear, [PG] + [vp] * 6 + [sz, vp]),
                     (L.moe_gated_linear_workspace_size, [PG, ctypes.c_int, pz]),
                     (L.moe_gated_linear_backward, [PG] + [vp] * 8 + [sz, vp])):
        fn.restype = ctypes.c_int
        fn.argtypes = args
    L.moe_set_stage_events.restype = ctypes.c_int
    L.moe_set_stage_events.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
    _lib = L
    return L


def _check(status: int):
    if status == OK:
        return
    msg = lib().moe_status_str(status).decode()
    if status in (ERR_NULL_ARG, ERR_BAD_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE):
        raise ValueError(f"moe status {status}: {msg}")
    if status == ERR_BAD_INDEX:
        raise IndexError(f"moe status {status}: {msg}")
    raise MoeError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


_ACT = {torch.float32: F32, torch.bfloat16: BF16}
_WGT = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: FP8_E4M3, torch.uint8: FP8_E4M3}
_FP4_DTYPES = (torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ()


def make_problem(T, H, I, E, k, act, weight, scale=SCALE_NONE, flags=0) -> Problem:
    return Problem(T, H, I, E, k, act, weight, scale, flags)


def workspace_size(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return n.value


def plan_describe(problem: Problem) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(lib().moe_plan_describe(ctypes.byref(problem), buf, len(buf)))
    return buf.value.decode()


def _need_gpu(name: str, t: torch.Tensor):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def problem_for(hidden, topk_idx, w_gate_up, w_down, w_gate_up_scale=None, flags=0) -> Problem:
    T, H = hidden.shape
    E, twoI, H2 = w_gate_up.shape
    k = topk_idx.shape[1]
    # fp4 weights: packed bytes (uint8 or float4_e2m1fn_x2) with half as many columns
    fp4 = (w_gate_up.dtype in _FP4_DTYPES or w_gate_up.dtype == torch.uint8) and 2 * H2 == H
    cols = 2 if fp4 else 1
    if (H2 * cols != H or twoI % 2 or tuple(w_down.shape) != (E, H, twoI // 2 // cols)
            or topk_idx.shape[0] != T):
        raise ValueError("inconsistent shapes: hidden [T,H], topk_idx [T,k], "
                         "w_gate_up [E,2I,H], w_down [E,H,I] (fp4: [E,2I,H/2], [E,H,I/2])")
    if hidden.dtype not in _ACT or w_down.dtype != w_gate_up.dtype or not (fp4 or w_gate_up.dtype in _WGT):
        raise ValueError("unsupported dtypes")
    weight = FP4_E2M1 if fp4 else _WGT[w_gate_up.dtype]
    scale = SCALE_NONE
    if weight in (FP8_E4M3, FP4_E2M1):
        if w_gate_up_scale is None:
            raise ValueError("fp8 and fp4 weights need scales")
        scale = SCALE_UE8M0 if w_gate_up_scale.dtype == torch.uint8 else SCALE_F32
    return Problem(T, H, twoI // 2, E, k, _ACT[hidden.dtype], weight, scale, flags)


def check_scales(prob: Problem, w_gate_up_scale: Optional[torch.Tensor],
                 w_down_scale: Optional[torch.Tensor]) -> None:
    """Block scales must match the weight format exactly, since the kernels read them by index.

    e4m3 weights: [E, 2I/128, H/128] and [E, H/128, I/128], both float32 or both uint8 (UE8M0);
    fp4 weights: [E, 2I, H/32] and [E, H, I/32] uint8 (UE8M0); other weights take none.
    Raises ValueError on a missing, extra, mismatched or wrongly shaped scale tensor.
    """
    E, H, I = prob.E, prob.H, prob.I
    if prob.weight_dtype not in (FP8_E4M3, FP4_E2M1):
        if w_gate_up_scale is not None or w_down_scale is not None:
            raise ValueError("block scales are only taken with e4m3 or fp4 weights")
        return
    if w_gate_up_scale is None or w_down_scale is None:
        raise ValueError("e4m3 and fp4 weights need both w_gate_up_scale and w_down_scale")
    if w_gate_up_scale.dtype != w_down_scale.dtype:
        raise ValueError(f"scale dtypes differ: {w_gate_up_scale.dtype} and {w_down_scale.dtype}")
    if prob.weight_dtype == FP4_E2M1:
        if w_gate_up_scale.dtype != torch.uint8:
            raise ValueError("fp4 weights take UE8M0 (uint8) scales")
        want = ((E, 2 * I, H // 32), (E, H, I // 32))
    else:
        if w_gate_up_scale.dtype not in (torch.float32, torch.uint8):
            raise ValueError("e4m3 block scales must be float32 or uint8 (UE8M0)")
        want = ((E, 2 * I // 128, H // 128), (E, H // 128, I // 128))
    for name, t, shape in (("w_gate_up_scale", w_gate_up_scale, want[0]),
                           ("w_down_scale", w_down_scale, want[1])):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def experts_forward(hidden: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                    w_gate_up: torch.Tensor, w_down: torch.Tensor,
                    w_gate_up_scale: Optional[torch.Tensor] = None,
                    w_down_scale: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, flags: int = 0,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[T,H] = sum_j topk_w[:,j] * SwiGLU-MLP_{topk_idx[:,j]}(hidden) on the GPU.

    hidden [T,H] f32|bf16; topk_idx [T,k] int32; topk_w [T,k] f32;
    w_gate_up [E,2I,H] and w_down [E,H,I] in f32 | bf16 | e4m3 (float8_e4m3fn or
    uint8 codes) with block scales [E,2I/128,H/128] / [E,H/128,I/128]
    (float32, or uint8 UE8M0 exponents); or fp4: w_gate_up [E,2I,H/2] and
    w_down [E,H,I/2] packed e2m1 bytes (uint8 or float4_e2m1fn_x2, element 2j in the low
    nibble of byte j) with UE8M0 scales [E,2I,H/32] / [E,H,I/32] (uint8).
    """
    for name, t in (("hidden", hidden), ("topk_idx", topk_idx), ("topk_w", topk_w),
                    ("w_gate_up", w_gate_up), ("w_down", w_down)):
        _need_gpu(name, t)
    if topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32:
        raise ValueError("topk_idx must be int32 and topk_w float32")
    if topk_w.shape != topk_idx.shape:
        raise ValueError("topk_w and topk_idx shapes differ")
    prob = problem_for(hidden, topk_idx, w_gate_up, w_down, w_gate_up_scale, flags)
    check_scales(prob, w_gate_up_scale, w_down_scale)
    for name, t in (("w_gate_up_scale", w_gate_up_scale), ("w_down_scale", w_down_scale)):
        if t is not None:
            _need_gpu(name, t)
    if out is None:
        out = torch.empty_like(hidden)
    else:
        _need_gpu("out", out)
        if out.shape != hidden.shape or out.dtype != hidden.dtype:
            raise ValueError("out must match hidden in shape and dtype")
    nbytes = workspace_size(prob)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=hidden.device)
    else:
        _need_gpu("workspace", workspace)
    _check(lib().moe_experts_forward(
        ctypes.byref(prob), _ptr(hidden), _ptr(topk_idx), _ptr(topk_w), _ptr(w_gate_up),
        _ptr(w_down), _ptr(w_gate_up_scale), _ptr(w_down_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(hidden.device)))
    return out


def experts_forward_quantized(hidden_q: torch.Tensor, hidden_scale: torch.Tensor, topk_idx: torch.Tensor,
                              topk_w: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                              w_gate_up_scale: torch.Tensor, w_down_scale: torch.Tensor,
                              out: Optional[torch.Tensor] = None, flags: int = 0,
                              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """experts_forward of e4m3 or fp4 experts on rows that are quantised already
    (moe_experts_forward_quantized): hidden_q [T,H] e4m3 codes (uint8 or float8_e4m3fn) and
    hidden_scale [T,H/128] float32, as rms_norm_fp8 and quantize_rows_fp8 return them.  The
    output is bf16."""
    given = [("hidden_q", hidden_q), ("hidden_scale", hidden_scale), ("topk_idx", topk_idx), ("topk_w", topk_w),
             ("w_gate_up", w_gate_up), ("w_down", w_down), ("w_gate_up_scale", w_gate_up_scale),
             ("w_down_scale", w_down_scale)]
    given += [(name, t) for name, t in (("out", out), ("workspace", workspace)) if t is not None]
    for name, t in given:
        _need_gpu(name, t)
    dev = hidden_q.get_device()
    for name, t in given:
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, hidden_q on cuda:{dev}")
    if hidden_q.dtype not in (torch.uint8, torch.float8_e4m3fn) or hidden_q.dim() != 2:
        raise ValueError("hidden_q must be a 2-D tensor of e4m3 codes (uint8 or float8_e4m3fn)")
    T, H = hidden_q.shape
    if hidden_scale.dtype != torch.float32 or H % 128 or tuple(hidden_scale.shape) != (T, H // 128):
        raise ValueError("hidden_scale must be float32 [T, H/128]")
    if topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32:
        raise ValueError("topk_idx must be int32 and topk_w float32")
    if topk_w.shape != topk_idx.shape:
        raise ValueError("topk_w and topk_idx shapes differ")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=hidden_q.device)
    elif tuple(out.shape) != (T, H) or out.dtype != torch.bfloat16:
        raise ValueError("out must be bf16 [T, H]")
    prob = problem_for(out, topk_idx, w_gate_up, w_down, w_gate_up_scale, flags)
    check_scales(prob, w_gate_up_scale, w_down_scale)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(prob), 1), dtype=torch.uint8, device=hidden_q.device)
    _run(lib().moe_experts_forward_quantized, dev, ctypes.byref(prob), _ptr(hidden_q), _ptr(hidden_scale), _ptr(topk_idx),
         _ptr(topk_w), _ptr(w_gate_up), _ptr(w_down), _ptr(w_gate_up_scale), _ptr(w_down_scale), _ptr(out), _ptr(workspace),
         workspace.numel() * workspace.element_size())
    return out


def experts_forward_noalloc(hidden: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                            w_gate_up: torch.Tensor, w_down: torch.Tensor,
                            w_gate_up_scale: Optional[torch.Tensor] = None,
                            w_down_scale: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, flags: int = 0) -> torch.Tensor:
    """experts_forward on the library's own device array instead of a workspace
    (moe_experts_forward_noalloc): allocates nothing when `out` is given."""
    for name, t in (("hidden", hidden), ("topk_idx", topk_idx), ("topk_w", topk_w),
                    ("w_gate_up", w_gate_up), ("w_down", w_down)):
        _need_gpu(name, t)
    if topk_idx.dtype != torch.int32 or topk_w.dtype != torch.float32:
        raise ValueError("topk_idx must be int32 and topk_w float32")
    if topk_w.shape != topk_idx.shape:
        raise ValueError("topk_w and topk_idx shapes differ")
    prob = problem_for(hidden, topk_idx, w_gate_up, w_down, w_gate_up_scale, flags)
    check_scales(prob, w_gate_up_scale, w_down_scale)
    for name, t in (("w_gate_up_scale", w_gate_up_scale), ("w_down_scale", w_down_scale)):
        if t is not None:
            _need_gpu(name, t)
    if out is None:
        out = torch.empty_like(hidden)
    else:
        _need_gpu("out", out)
        if out.shape != hidden.shape or out.dtype != hidden.dtype:
            raise ValueError("out must match hidden in shape and dtype")
    _check(lib().moe_experts_forward_noalloc(
        ctypes.byref(prob), _ptr(hidden), _ptr(topk_idx), _ptr(topk_w), _ptr(w_gate_up), _ptr(w_down),
        _ptr(w_gate_up_scale), _ptr(w_down_scale), _ptr(out), _stream(hidden.device)))
    return out


def route(topk_idx: torch.Tensor, E: int, flags: int = 0, workspace=None):
    """(counts[E], offsets[E+1], perm[T*k], inv[T*k]) int32: the stable sort of slots by expert."""
    _need_gpu("topk_idx", topk_idx)
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise ValueError("topk_idx must be a 2-D int32 tensor")
    T, k = topk_idx.shape
    dev = topk_idx.device
    # the bookkeeping does not depend on H, I or the dtypes; any valid problem sizes it
    prob = Problem(T, 128, 128, E, k, BF16, BF16, SCALE_NONE, flags)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(workspace_size(prob), dtype=torch.uint8, device=dev)
    _check(lib().moe_route(ctypes.byref(prob), _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                           _ptr(perm), _ptr(inv), _ptr(workspace), workspace.numel(), _stream(dev)))
    return counts, offsets, perm[: T * k], inv[: T * k]


def route_logits(logits: torch.Tensor, k: int, renorm: bool = False, workspace=None):
    """Router + bookkeeping from float32 logits [T, E]: (topk_idx[T,k] int32, topk_w[T,k] float32,
    counts[E], offsets[E+1], perm[T*k], inv[T*k]); see moe_route_logits."""
    _need_gpu("logits", logits)
    if logits.dtype != torch.float32 or logits.dim() != 2 or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous 2-D float32 tensor")
    T, E = logits.shape
    dev = logits.device
    prob = Problem(T, 128, 128, E, k, BF16, BF16, SCALE_NONE, 0)
    idx = torch.empty((max(T, 1), k), dtype=torch.int32, device=dev)
    w = torch.empty((max(T, 1), k), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    inv = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = torch.empty(workspace_size(prob), dtype=torch.uint8, device=dev)
    _check(lib().moe_route_logits(ctypes.byref(prob), _ptr(logits), int(bool(renorm)), _ptr(idx), _ptr(w),
                                  _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(inv), _ptr(workspace),
                                  workspace.numel(), _stream(dev)))
    return idx[:T], w[:T], counts, offsets, perm[: T * k], inv[: T * k]


def set_stage_events(handles):
    """Install per-stage hipEvent_t handles (a list of 2*len(STAGES) ints or None) on this thread;
    None clears the hook."""
    if handles is None:
        _check(lib().moe_set_stage_events(None, 0))
        return
    arr = (ctypes.c_void_p * len(handles))(*[h or None for h in handles])
    _check(lib().moe_set_stage_events(arr, len(handles)))


def quantize_rows_fp8(x: torch.Tensor):
    """Per-row, per-128-column e4m3 quantisation of a bf16 matrix -> (codes uint8, scales f32)."""
    _need_gpu("x", x)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    R, C = x.shape
    if C % 128:
        raise ValueError("columns must be a multiple of 128")
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    s = torch.empty((R, C // 128), dtype=torch.float32, device=x.device)
    _check(lib().moe_quantize_rows_fp8(_ptr(x), R, C, _ptr(q), _ptr(s), _stream(x.device)))
    return q, s


def check_mfma_blocks(a: torch.Tensor, b: torch.Tensor, b_scale: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Block products on the kernels' block-scaled MFMA (moe_check_mfma_blocks): a uint8
    [n,16,128] e4m3 codes; b uint8 [n,16,128] e4m3 codes (with an optional b_scale), or
    [n,16,64] packed e2m1 with b_scale; b_scale uint8 [n,16,4] UE8M0.  Returns float32
    [n,16,16]."""
    fmt = 0 if b_scale is None else (2 if b.dim() == 3 and b.shape[-1] == 128 else 1)
    for name, t in (("a", a), ("b", b)) + ((("b_scale", b_scale),) if fmt else ()):
        _need_gpu(name, t)
        if t.dtype != torch.uint8:
            raise ValueError(f"{name} must be uint8")
    n = a.shape[0]
    want_b = (n, 16, 64) if fmt == 1 else (n, 16, 128)
    if tuple(a.shape) != (n, 16, 128) or tuple(b.shape) != want_b or (fmt and tuple(b_scale.shape) != (n, 16, 4)):
        raise ValueError("shapes: a [n,16,128], b [n,16,128] (e4m3, b_scale optional) or [n,16,64] with "
                         "b_scale [n,16,4] (e2m1)")
    d = torch.empty((n, 16, 16), dtype=torch.float32, device=a.device)
    _check(lib().moe_check_mfma_blocks(fmt, _ptr(a), _ptr(b), _ptr(b_scale), _ptr(d), n, _stream(a.device)))
    return d


# ----------------------------------------------------------------------------- dense operators
# (Decode steps make these calls by the thousand, each a few microseconds of GPU time: the checks
# below take the common case in one comparison and say what is wrong only after it fails.)
# `workspace`, where a call takes one, is any contiguous tensor of at least the bytes that lib()'s moe_*_workspace_size
# gives for the NormProblem, LinearProblem or GatedProblem; calls that may overlap take different ones.  Without
# it each call takes its own from torch's allocator.


def _rows(name: str, t: torch.Tensor, T: int, cols: int, dtype: torch.dtype, dev: int) -> int:
    """Checks a [T, cols] activation matrix on GPU `dev`; returns its row pitch in elements."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.shape != (T, cols) or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, (T, cols), dtype, dev)
    ld, inner = t.stride()
    if T <= 1:
        ld = cols
    if (inner != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have unit stride along its rows and rows that do not overlap")
    return ld


def _packed(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, dev: int) -> None:
    """Checks a packed tensor on GPU `dev`."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _refuse(name, t, shape, dtype, dev):
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
    raise ValueError(f"{name} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")


def _matrix(name: str, t: torch.Tensor):
    """(moe_dtype, GPU index) of the 2-D bf16 or float32 GPU tensor that a call's types follow."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _ACT:
        raise ValueError(f"{name} must be a bf16 or float32 tensor")
    dev = t.get_device() if t.device.type == "cuda" else -1
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {list(t.shape)}")
    return _ACT[t.dtype], dev


def _outputs(name: str, w: torch.Tensor) -> int:
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError(f"{name} must be a tensor of two dimensions")
    return w.shape[0]


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _run(fn, dev: int, *args) -> None:
    """Calls fn(*args, current stream of GPU `dev`) with that GPU current."""
    C = torch._C             # (looked up here: a torch without GPU support has neither name, and imports the package)
    if C._cuda_getDevice() == dev:
        status = fn(*args, C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


def _scratch(workspace: Optional[torch.Tensor], need: int, x: torch.Tensor, dev: int):
    """(tensor or None, bytes): the caller's workspace, or one of `need` bytes next to x."""
    if workspace is not None:
        _need_gpu("workspace", workspace)
        if workspace.get_device() != dev:
            raise ValueError(f"workspace is on {workspace.device}, the call's other tensors on cuda:{dev}")
        return workspace, workspace.numel() * workspace.element_size()
    if need == 0:
        return None, 0
    return x.new_empty(need, dtype=torch.uint8), need


@functools.lru_cache(maxsize=4096)
def _problem(kind, fields: tuple, size_fn: Optional[str] = None, *args):
    """(reference to the C problem, its workspace bytes): both follow from the fields alone, so
    they are made once per problem.  The library only reads the struct."""
    prob = kind(*fields)
    for (name, _), given in zip(kind._fields_, fields):      # (ctypes keeps an integer's low bits without a word)
        if isinstance(given, int) and getattr(prob, name) != given:
            raise ValueError(f"{name} = {given} is out of range")
    ref = ctypes.byref(prob)
    n = ctypes.c_size_t(0)
    if size_fn is not None:
        _check(getattr(lib(), size_fn)(ref, *args, ctypes.byref(n)))
    return ref, n.value


def _rms_norm(x, weight, eps, residual, fp8, with_y):
    dt, dev = _matrix("x", x)
    T, H = x.shape
    dtype = x.dtype
    ldr = 0
    _packed("weight", weight, (H,), dtype, dev)
    if residual is None:
        h = x
    else:
        ldr = _rows("residual", residual, T, H, dtype, dev)
        h = torch.empty_like(x)
    prob, _ = _problem(NormProblem, (T, H, dt, float(eps), _rows("x", x, T, H, dtype, dev), ldr, 0, 0))
    y = torch.empty_like(x) if with_y else None
    rstd = x.new_empty(T, dtype=torch.float32)
    q = scale = None
    if fp8:
        if dtype is not torch.bfloat16 or H % 128:
            raise ValueError("the 8-bit output takes bf16 rows with H a multiple of 128")
        q = x.new_empty((T, H), dtype=torch.uint8)
        scale = x.new_empty((T, H // 128), dtype=torch.float32)
    _run(lib().moe_rms_norm, dev, prob, x.data_ptr(), _addr(residual), weight.data_ptr(), _addr(y),
         None if residual is None else h.data_ptr(), rstd.data_ptr(), _addr(q), _addr(scale))
    return q, scale, y, h, rstd


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None):
    """(y, h, rstd): h = x + residual (x itself without one), rstd = (mean h^2 + eps)^-1/2 [T]
    float32, y = h * rstd * weight; see moe_rms_norm.  x, residual [T,H], weight [H], bf16 or float32."""
    _, _, y, h, rstd = _rms_norm(x, weight, eps, residual, False, True)
    return y, h, rstd


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 residual: Optional[torch.Tensor] = None, with_y: bool = False):
    """(q, scales, y, h, rstd): rms_norm with its result as e4m3 codes (uint8 [T,H]) and float32
    scales [T,H/128], the rows experts_forward_quantized takes, and y in bf16 as well when
    with_y (else None)."""
    return _rms_norm(x, weight, eps, residual, True, with_y)


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      dh: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """(dx, dweight) of rms_norm, from dy and dh, the gradient that reaches h along the residual
    stream; dx is the gradient of x and of the residual.  See moe_rms_norm_backward."""
    dt, dev = _matrix("h", h)
    T, H = h.shape
    dtype = h.dtype
    ldr = 0 if dh is None else _rows("dh", dh, T, H, dtype, dev)
    fields = (T, H, dt, 0.0, 0, ldr, _rows("h", h, T, H, dtype, dev), _rows("dy", dy, T, H, dtype, dev))
    _packed("weight", weight, (H,), dtype, dev)
    _packed("rstd", rstd, (T,), torch.float32, dev)
    prob, need = _problem(NormProblem, fields, "moe_rms_norm_workspace_size")
    ws, n = _scratch(workspace, need, h, dev)
    dx = torch.empty_like(h)
    dweight = torch.empty_like(weight)
    _run(lib().moe_rms_norm_backward, dev, prob, dy.data_ptr(), h.data_ptr(),
         weight.data_ptr(), rstd.data_ptr(), _addr(dh), dx.data_ptr(), dweight.data_ptr(), _addr(ws), n)
    return dx, dweight


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
           residual: Optional[torch.Tensor] = None, act: int = ACT_NONE, out_dtype: Optional[torch.dtype] = None,
           save_pre: bool = False, workspace: Optional[torch.Tensor] = None):
    """(y, pre): y = act(x w^T + bias) + residual in out_dtype (x's, or float32), and pre = x w^T +
    bias when save_pre (else None).  x [T,K], w [N,K], bias [N], residual [T,N] in
    out_dtype; see moe_linear."""
    dt, dev = _matrix("x", x)
    T, K = x.shape
    N = _outputs("w", w)
    dtype = x.dtype
    odt = dtype if out_dtype is None else out_dtype
    if odt not in _ACT:
        raise ValueError("out_dtype must be bf16 or float32")
    _packed("w", w, (N, K), dtype, dev)
    if bias is not None:
        _packed("bias", bias, (N,), dtype, dev)
    ldr = 0 if residual is None else _rows("residual", residual, T, N, odt, dev)
    fields = (T, K, N, dt, _ACT[odt], int(act), _rows("x", x, T, K, dtype, dev), 0, ldr, 0, 0)
    prob, need = _problem(LinearProblem, fields, "moe_linear_workspace_size", 0)
    ws, n = _scratch(workspace, need, x, dev)
    y = x.new_empty((T, N), dtype=odt)
    pre = x.new_empty((T, N)) if save_pre else None
    _run(lib().moe_linear, dev, prob, x.data_ptr(), w.data_ptr(), _addr(bias),
         _addr(residual), y.data_ptr(), _addr(pre), _addr(ws), n)
    return y, pre


def linear_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, pre: Optional[torch.Tensor] = None,
                    act: int = ACT_NONE, need_bias: bool = False, workspace: Optional[torch.Tensor] = None):
    """(dx, dw, dbias) of linear, dbias None without need_bias; pre is what linear saved (needed
    with an activation).  See moe_linear_backward."""
    dt, dev = _matrix("x", x)
    T, K = x.shape
    N = _outputs("w", w)
    dtype = x.dtype
    ody, _ = _matrix("dy", dy)
    _packed("w", w, (N, K), dtype, dev)
    ldp = 0
    if act == ACT_NONE:
        pre = None
    elif pre is None:
        raise ValueError("an activation's gradient needs pre")
    else:
        ldp = _rows("pre", pre, T, N, dtype, dev)
    fields = (T, K, N, dt, ody, int(act), _rows("x", x, T, K, dtype, dev), _rows("dy", dy, T, N, dy.dtype, dev), 0, ldp, 0)
    return _backward("moe_linear_backward", LinearProblem, fields, dy, x, w, pre, N, need_bias, workspace, dev)


def _backward(fn_name, kind, fields, dy, x, w, pre, cols, need_bias, workspace, dev):
    prob, need = _problem(kind, fields, fn_name.replace("_backward", "_workspace_size"), 1 if need_bias else 2)
    ws, n = _scratch(workspace, need, x, dev)
    dx = torch.empty_like(x)
    dw = torch.empty_like(w)
    dbias = x.new_empty(cols) if need_bias else None
    _run(getattr(lib(), fn_name), dev, prob, dy.data_ptr(), x.data_ptr(), w.data_ptr(),
         _addr(pre), dx.data_ptr(), dw.data_ptr(), _addr(dbias), _addr(ws), n)
    return dx, dw, dbias


def _gated_sizes(x, w_gate_up):
    dt, dev = _matrix("x", x)
    T, H = x.shape
    I = _outputs("w_gate_up", w_gate_up) // 2
    _packed("w_gate_up", w_gate_up, (2 * I, H), x.dtype, dev)
    return dt, dev, T, H, I


def gated_linear(x: torch.Tensor, w_gate_up: torch.Tensor, bias: Optional[torch.Tensor] = None, act: int = ACT_SILU,
                 save_pre: bool = False, workspace: Optional[torch.Tensor] = None):
    """(a, pre): [gate | up] = x w_gate_up^T + bias, a = act(gate) * up [T,I], and pre = [gate |
    up] [T,2I] when save_pre (else None).  x [T,H], w_gate_up [2I,H], bias [2I]; see moe_gated_linear."""
    dt, dev, T, H, I = _gated_sizes(x, w_gate_up)
    if bias is not None:
        _packed("bias", bias, (2 * I,), x.dtype, dev)
    fields = (T, H, I, dt, int(act), _rows("x", x, T, H, x.dtype, dev), 0, 0, 0)
    prob, need = _problem(GatedProblem, fields, "moe_gated_linear_workspace_size", 0)
    ws, n = _scratch(workspace, need, x, dev)
    a = x.new_empty((T, I))
    pre = x.new_empty((T, 2 * I)) if save_pre else None
    _run(lib().moe_gated_linear, dev, prob, x.data_ptr(), w_gate_up.data_ptr(),
         _addr(bias), a.data_ptr(), _addr(pre), _addr(ws), n)
    return a, pre


def gated_linear_backward(da: torch.Tensor, x: torch.Tensor, w_gate_up: torch.Tensor, pre: torch.Tensor,
                          act: int = ACT_SILU, need_bias: bool = False, workspace: Optional[torch.Tensor] = None):
    """(dx, dw, dbias) of gated_linear from da and the pre it saved; dbias None without need_bias.
    See moe_gated_linear_backward."""
    dt, dev, T, H, I = _gated_sizes(x, w_gate_up)
    fields = (T, H, I, dt, int(act), _rows("x", x, T, H, x.dtype, dev), _rows("da", da, T, I, x.dtype, dev),
              _rows("pre", pre, T, 2 * I, x.dtype, dev), 0)
    return _backward("moe_gated_linear_backward", GatedProblem, fields, da, x, w_gate_up, pre, 2 * I, need_bias,
                     workspace, dev)
