"""The dense operators' LDS-DMA loads (dense_tile.h) are inline asm: each carries its own wait
states (an s_nop 4 right before it), since the compiler's hazard checks do not look inside.  This compiles
the sources that use them to gfx950 assembly and checks the instruction before each load, that no
kernel spills registers to scratch inside a loop of such loads, and that none uses packed float32."""

import os
import re
import subprocess

import pytest

from mixture_experts_routed_topk_amd import build_lib


def _tile_sources():
    return [f for f in sorted(os.listdir(build_lib.CSRC))
            if f.endswith(".hip") and '#include "dense_tile.h"' in open(os.path.join(build_lib.CSRC, f)).read()]


@pytest.mark.skipif(not os.path.exists(build_lib.HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src", _tile_sources())
def test_dense_dma_loads_carry_wait_states(src, tmp_path):
    asm = tmp_path / (src + ".s")
    cmd = [build_lib.HIPCC, *build_lib.FLAGS, "--cuda-device-only", "-S", os.path.join(build_lib.CSRC, src), "-o", str(asm)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(asm).read()
    ins = [t for t in (line.strip() for line in text.splitlines())
           if t and not t.startswith((";", ".", "//")) and not t.endswith(":")]
    loads = [i for i, t in enumerate(ins) if t.startswith("global_load_lds")]
    assert loads or src == "dense_rows.hip"          # (that one takes the fragment types alone)
    for i in loads:
        m = re.match(r"s_nop\s+(\d+)", ins[i - 1])
        assert m and int(m.group(1)) >= 4, f"{src}: '{ins[i]}' is preceded by '{ins[i - 1]}'"
    assert not re.search(r"\bv_pk_(add|mul|fma)_f32\b", text)
    assert all(int(n) == 0 for n in re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text))
