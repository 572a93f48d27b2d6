"""How a call's workgroups are cut into HIP launches, which have fewer than 2^32
lanes each: on the host, with the launches counted instead of made."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include <stdio.h>
#include "zero_train_internal.h"
int main() {
    const int64_t blocks[] = {1, 255, (1 << 22) - 1, 1 << 22, (1 << 22) + 1, (1 << 24) - 1,
                              1 << 24, (1 << 26) - 1, 1 << 26, (1 << 26) + 3, 0x7fffffff};
    for (int64_t lanes = 64; lanes <= 1024; lanes += 64)
        for (int64_t n : blocks) {
            int64_t next = 0, launches = 0;
            const hipError_t e = zero::in_launches(n, lanes, [&](int64_t first, uint32_t grid) {
                if (first != next || grid == 0 || grid * lanes >= (int64_t{1} << 32))
                    return hipErrorInvalidValue;
                next = first + grid;
                ++launches;
                return hipSuccess;
            });
            if (e != hipSuccess || next != n || launches > n * lanes / 0xffff0000 + 1) {
                printf("%lld blocks of %lld lanes\n", (long long)n, (long long)lanes);
                return 1;
            }
        }
    int made = 0;
    const hipError_t e = zero::in_launches(int64_t{1} << 30, 64, [&](int64_t, uint32_t) {
        return ++made == 2 ? hipErrorOutOfMemory : hipSuccess;
    });
    return e == hipErrorOutOfMemory && made == 2 ? 0 : 2;
}
"""


def test_every_launch_has_fewer_than_2_32_lanes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    src, exe = tmp_path / "launches.cpp", str(tmp_path / "launches")
    src.write_text(SOURCE)
    includes = [x for d in (os.path.join(ROOT, "include"), "/opt/rocm/include",
                            os.path.join(ROOT, "sharded_mixed_precision_step_amd", "csrc"))
                for x in ("-I", d)]
    subprocess.run([gxx, "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", *includes, str(src), "-o",
                    exe], check=True)
    run = subprocess.run([exe], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
