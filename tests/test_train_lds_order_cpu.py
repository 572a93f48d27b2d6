"""The product's kernels pass c between lanes through LDS.  In the compiler's
intermediate code of every kernel a fence stands between such writes and the
reads that follow them, and between reads and the writes that follow: without
one nothing keeps the compiler from moving one across the other, since it only
has to honour what a single lane can tell."""
import os
import re
import subprocess

import pytest

from sharded_mixed_precision_step_amd import _build

pytestmark = pytest.mark.cpu


def test_a_fence_stands_between_writes_and_reads_of_the_turn(tmp_path):
    out = str(tmp_path / "gemm.ll")
    flags = [f for f in _build.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([_build.hipcc(), *flags, "-I", _build.INCLUDE, "--cuda-device-only", "-S",
                    "-emit-llvm", os.path.join(_build.CSRC, "zero_q8_gemm.hip"), "-o", out],
                   check=True, capture_output=True)
    kernels, last, open_pairs = 0, None, []
    for line in open(out):
        if line.startswith("define amdgpu_kernel"):
            kernels, last, name = kernels + 1, None, line.split("@")[1].split("(")[0]
        elif re.match(r"\s*fence ", line):
            last = None
        elif re.search(r"store <4 x float> .*addrspace\(3\)", line):
            if last == "read":
                open_pairs.append((name, "write after read"))
            last = "write"
        elif re.search(r"load <4 x float>, ptr addrspace\(3\)", line):
            if last == "write":
                open_pairs.append((name, "read after write"))
            last = "read"
    assert kernels == 20    # four tile variants and few rows, four pairs of formats each
    assert not open_pairs, (len(open_pairs), open_pairs[0])
