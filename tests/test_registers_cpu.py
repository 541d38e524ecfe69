"""What the norms' and products' kernels keep in registers stays there: nothing
that nvcc compiles of them has a stack or spills (no GPU)."""
import os
import re
import subprocess

import pytest

from fp4_block_scaled_gb300 import _build


@pytest.mark.parametrize("src,kernels", [("norm.cu", 126), ("mxquant.cu", 9), ("linear.cu", 4), ("linear_pair.cu", 4)])
def test_no_kernel_spills(src, kernels, tmp_path):
    r = subprocess.run([_build.nvcc(), *_build.ARCH, *_build.FLAGS, "-Xptxas", "-v", "-c", os.path.join(_build.CSRC, src), "-o", str(tmp_path / "o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = re.findall(r"Function properties for (\w+)\s+(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads", r.stdout + r.stderr)
    assert len(found) == kernels
    assert [f for f in found if f[1:] != ("0", "0", "0")] == []
