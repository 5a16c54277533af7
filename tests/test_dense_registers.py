"""Registers of the norm's and the elementwise backward kernels (norm.hip, dense_backward.hip), which include no DMA and
so are not among test_dense_isa.py's: only the norm's instances for rows of more than 8192 columns keep
values in scratch memory, as norm.hip says, and none uses packed float32."""

import os
import re
import subprocess

import pytest

from mixture_experts_routed_topk_amd import build_lib

# sixteen waves a row, of 4 (H <= 32768) or 8 pieces a lane (f: float32, t: bf16)
SPILL = {"rms_norm_backward_kernelIfLi16ELi4E", "rms_norm_backward_kernelItLi16ELi4E", "rms_norm_backward_kernelIfLi16ELi8E",
         "rms_norm_backward_kernelItLi16ELi8E", "rms_norm_kernelIfLi16ELi8ELb0E", "rms_norm_kernelItLi16ELi8ELb1E"}


@pytest.mark.skipif(not os.path.exists(build_lib.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", ["norm.hip", "dense_backward.hip"])
def test_no_scratch_but_for_the_longest_rows(src, tmp_path):
    asm = tmp_path / (src + ".s")
    cmd = [build_lib.HIPCC, *build_lib.FLAGS, "--cuda-device-only", "-S", os.path.join(build_lib.CSRC, src), "-o", str(asm)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(asm).read()
    sizes = re.findall(r"\.name:\s+(\S+)\s+\.private_segment_fixed_size:\s*(\d+)", text)
    assert len(sizes) == text.count(".private_segment_fixed_size:") > 0
    spilling = [n for n, b in sizes if int(b) > 0]
    assert all(any(k in n for k in SPILL) for n in spilling), spilling
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
