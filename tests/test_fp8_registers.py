"""Registers of the e4m3 quantisers and of the permutations (fp8_quant.hip, permute.hip), which include no DMA and so are not among
test_dense_isa.py's: no kernel keeps values in scratch memory, and none uses packed float32."""

import os
import re
import subprocess

import pytest

from mixture_experts_routed_topk_amd import build_lib


@pytest.mark.skipif(not os.path.exists(build_lib.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", ["fp8_quant.hip", "permute.hip"])
def test_no_scratch_and_no_packed_float32(src, tmp_path):
    asm = tmp_path / (src + ".s")
    cmd = [build_lib.HIPCC, *build_lib.FLAGS, "--cuda-device-only", "-S", os.path.join(build_lib.CSRC, src), "-o", str(asm)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(asm).read()
    sizes = re.findall(r"\.name:\s+(\S+)\s+\.private_segment_fixed_size:\s*(\d+)", text)
    assert len(sizes) == text.count(".private_segment_fixed_size:") > 0
    assert [n for n, b in sizes if int(b) > 0] == []
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
