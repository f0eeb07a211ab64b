"""Kernels whose lanes exchange data through LDS inside a wave, without a barrier of the block, have to
say so: a store by one lane and a load by another are ordered for the compiler by a fence alone.  Read
from the intermediate code that hipcc makes of the sources (no GPU needed)."""
import os
import re
import subprocess

import pytest

from combine_ep_get_02_amd import build as hip_build

# a source, and what the names of its kernels with such exchanges hold
EXCHANGES = [("ep_expert_gemm.hip", "expert_gemm_narrow_kernel"), ("ep_route.hip", "12route_kernel")]


@pytest.mark.parametrize("source,kernel", EXCHANGES)
def test_lanes_of_a_wave_order_what_they_exchange(source, kernel, tmp_path):
    src = next(s for s in hip_build.SOURCES if os.path.basename(s) == source)
    flags = [f for f in hip_build.FLAGS if f != "-shared"]
    out = tmp_path / "kernels.ll"
    subprocess.run(["hipcc", *flags, "--cuda-device-only", "-S", "-emit-llvm", src, "-o", str(out)], check=True,
                   capture_output=True)
    text = {m.group(1): m.group(0) for m in re.finditer(r"^define [^\n]*@(\S+?)\(.*?^}", out.read_text(), flags=re.S | re.M)}
    found = {name: body for name, body in text.items() if kernel in name}
    assert found
    for name, body in found.items():
        fences = len(re.findall(r'fence syncscope\("wavefront"\) acq_rel', body))
        # one between what a tile's lanes store and load, and one before the next tile takes its place
        assert fences >= 2, (name, fences)
