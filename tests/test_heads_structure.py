"""Structure of the attention operators' compiled kernels (CPU only: compiles to
assembly): none keeps vector registers in scratch memory but the fp32 kernel of
many rows with heads of 256 values, whose queries take three terms."""

import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "all_reduce_reduction_rank_amd", "csrc")


@pytest.mark.parametrize("source,kernels", [("rope", 26), ("cache", 12), ("attention", 21)])
def test_no_scratch_memory(tmp_path, source, kernels):
    out = tmp_path / "k.s"
    cmd = ["hipcc", "--offload-arch=gfx950", "-O3", "-std=c++17", "-S", "--cuda-device-only", "-Xclang", "-target-feature",
           "-Xclang", "-packed-fp32-ops", "-o", str(out), os.path.join(CSRC, source + ".hip")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    sizes = re.findall(r"\.name:\s+(\S+)\s.*?\.private_segment_fixed_size:\s+(\d+)", out.read_text(), re.S)
    sizes = [(n, int(x)) for n, x in sizes if "_kernel" in n]
    assert len(sizes) == kernels
    for name, size in sizes:
        assert size == 0 or "many_rows_kernelILi0ELi256E" in name, (name, size)
