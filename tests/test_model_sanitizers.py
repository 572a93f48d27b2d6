"""The host layer of zero_model.h's operators under AddressSanitizer and
UndefinedBehaviorSanitizer, and under ThreadSanitizer for concurrent calls: 160,000
draws of every entry point's arguments over their whole ranges, with stubs of the
device side that hold each accepted call to what the kernels assume
(tests/host_harness/model_harness.cpp).  Built with g++, host code only."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.cpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HARNESS = os.path.join(ROOT, "tests", "host_harness", "model_harness.cpp")
CSRC = os.path.join(ROOT, "sharded_mixed_precision_step_amd", "csrc")


def _run(tmp_path, sanitize, env, *args):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.isdir("/opt/rocm/include"):
        pytest.skip("needs g++ and the ROCm headers")
    exe = str(tmp_path / "model_harness")
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-pthread", sanitize,
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__"]
    for inc in (os.path.join(ROOT, "include"), CSRC, "/opt/rocm/include"):
        cmd += ["-I", inc]
    build = subprocess.run([*cmd, HARNESS, os.path.join(CSRC, "zero_model_abi.cpp"), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-4000:]
    run = subprocess.run([exe, *args], capture_output=True, text=True, env=dict(os.environ, **env),
                         timeout=300)
    assert run.returncode == 0, (run.stdout + run.stderr)[-4000:]
    assert "model harness: ok" in run.stdout


def test_host_layer_under_sanitizers(tmp_path):
    _run(tmp_path, "-fsanitize=address,undefined",
         dict(ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0",
              UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1"))


def test_host_layer_from_many_threads_under_tsan(tmp_path):
    _run(tmp_path, "-fsanitize=thread", dict(TSAN_OPTIONS="halt_on_error=1"), "threads")
