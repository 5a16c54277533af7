"""The tiles and splits the dense operators choose (dense_plan.h, compiled for the host): the table of dense_tiles.py,
which the GPU tests run, reaches every tile kernel; what was fitted anew has to keep that."""

import os
import shutil
import subprocess

import pytest

from dense_tiles import GATED, GRADIENTS, HALVES, LINEAR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_routed_topk_amd", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "dense_plan_check")
    src = os.path.join(ROOT, "tests", "cpp", "dense_plan_check.cpp")
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-I", CSRC, src, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]

    def ask(*fields):
        out = subprocess.run([exe], input=" ".join(map(str, fields)), capture_output=True, text=True, timeout=60)
        return [int(v) for v in out.stdout.split()]

    return ask


@pytest.mark.parametrize("gated,cases", [(0, LINEAR), (1, GATED)], ids=["linear", "gated"])
def test_forward_tiles(plan, gated, cases):
    for dtype, T, K, N, rows, split in cases:
        tile, splits, halves = plan("fwd", dtype, T, N, K, gated)
        assert (tile, splits > 1, halves) == (rows, split, 0), (dtype, T, K, N, tile, splits, halves)
    assert {(c[0], c[4], c[5]) for c in cases} == {(d, r, s) for d, rs in (("bf16", (64, 128, 256)), ("f32", (32, 64, 128)))
                                                  for r in rs for s in (False, True)}


def test_half_tiles(plan):
    for T, K, N, gated in HALVES:
        assert plan("fwd", "bf16", T, N, K, int(gated)) == [256, 1, 1]


def test_gradient_tiles(plan):
    for dtype, T, K, cols, a, b, sa, sb in GRADIENTS:
        rx, rw, sx, sw = plan("grad", dtype, T, K, cols)
        assert (rx, rw, sx > 1, sw > 1) == (a, b, sa, sb), (dtype, T, K, cols, rx, rw, sx, sw)
    assert {(c[0], c[4]) for c in GRADIENTS} == {("bf16", r) for r in (64, 128, 256)} | {("f32", r) for r in (32, 64, 128)}
