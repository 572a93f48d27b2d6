"""The build script: what the files it leaves are like, without compiling."""
import os
import stat
import subprocess
import sys
import sysconfig

import pytest
import torch

from sharded_mixed_precision_step_amd import _build

pytestmark = pytest.mark.cpu


def _into(monkeypatch, folder):
    """The build's libraries in `folder`, and a compiler that writes into the file it is
    given, as g++ does: the file keeps the mode that it has."""
    libs = ("LIB", "TWIN_LIB", "GEN_LIB", "MARSHAL_LIB")
    for name in libs:
        monkeypatch.setattr(_build, name, str(folder / os.path.basename(getattr(_build, name))))

    def run_all(commands, verbose):
        for cmd in commands:
            with open(cmd[cmd.index("-o") + 1], "wb") as f:
                f.write(b"x")

    monkeypatch.setattr(_build, "_run_all", run_all)
    monkeypatch.setattr(_build, "hipcc", lambda: "hipcc")
    return [getattr(_build, name) for name in libs]


def test_every_library_may_be_loaded_by_every_user(monkeypatch, tmp_path):
    libs = _into(monkeypatch, tmp_path)
    # of earlier builds, whose calls may no longer fit
    (tmp_path / "_marshal.so").write_bytes(b"old")
    (tmp_path / "_marshal.cpython-39-x86_64-linux-gnu.torch-1.0.so").write_bytes(b"old")
    _build.build()
    for lib in libs:
        assert stat.S_IMODE(os.stat(lib).st_mode) == 0o755, lib
    assert sorted(os.listdir(tmp_path)) == sorted(os.path.basename(lib) for lib in libs)


@pytest.mark.parametrize("which", ["compile", "host", "link"])
def test_an_error_names_the_compiler_and_the_file(tmp_path, which):
    failing = tmp_path / "failing"
    failing.write_text("#!/bin/sh\necho no such thing >&2\nexit 3\n")
    failing.chmod(0o755)
    cmd, file = {
        "compile": ([str(failing), "-I", "include", "-o", "1.o", "-c", "csrc/a.hip"], "csrc/a.hip"),
        "host": ([str(failing), *_build.marshal_command("m.tmp")[1:]], _build.MARSHAL_SOURCE),
        "link": ([str(failing), "1.o", "2.o", "-o", ".lib.tmp"], ".lib.tmp"),
    }[which]
    with pytest.raises(RuntimeError) as error:
        _build._run_all([cmd], False)
    first = str(error.value).splitlines()[0]
    assert first.startswith("failing failed (3) for ") and file in first
    assert "no such thing" in str(error.value)


def _package(folder):
    """The package in `folder` without a host library of the binding."""
    package = folder / "sharded_mixed_precision_step_amd"
    package.mkdir()
    for name in os.listdir(_build.HERE):
        if name.endswith(".py") or name.startswith("lib"):
            (package / name).symlink_to(os.path.join(_build.HERE, name))
    return package


# Refused by the library at once, so that no device is asked for.
_IMPORT = """
import warnings
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    import sharded_mixed_precision_step_amd as zs
from sharded_mixed_precision_step_amd import _marshal, model, train
args = [1, 7, 4096, None, 1, 4096, 1, None, 1, -1, 4096, 1e-5, None, 0, None, 1, 4096, None, 0,
        4096, None, 32, None, None, None]
assert model._calls.zero_layernorm(*args) == -1
assert "rows = -1" in zs.lib.zero_last_error_string().decode()
print(_marshal is None, train._mat is train._mat_checked, [str(w.message) for w in seen])
"""


@pytest.mark.parametrize("found", ["none", "another torch's", "broken"])
def test_without_a_host_library_of_its_own_the_binding_goes_through_ctypes(tmp_path, found):
    package = _package(tmp_path)
    if found == "another torch's":      # the untagged name, and another version's
        (package / "_marshal.so").write_bytes(b"no library")
        (package / "_marshal.cpython-39-x86_64-linux-gnu.torch-1.0.so").write_bytes(b"no library")
    elif found == "broken":
        (package / os.path.basename(_build.MARSHAL_LIB)).write_bytes(b"no library")
    run = subprocess.run([sys.executable, "-c", _IMPORT], cwd=tmp_path, capture_output=True,
                         text=True, timeout=300, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert run.returncode == 0, run.stderr
    last = run.stdout.splitlines()[-1]
    assert last.startswith("True True ") and "calls go through ctypes" in last, last


def test_the_host_library_belongs_to_one_python_and_one_torch():
    name = os.path.basename(_build.MARSHAL_LIB)
    assert torch.__version__ in name and sysconfig.get_config_var("SOABI") in name


@pytest.mark.parametrize("how", ["no g++", "no headers", "no success"])
def test_the_other_libraries_are_built_without_the_host_library(monkeypatch, tmp_path, how):
    libs = _into(monkeypatch, tmp_path)
    run_all = _build._run_all
    if how == "no g++":
        monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    elif how == "no headers":
        monkeypatch.setattr(_build, "_marshal_includes", lambda: [str(tmp_path)])
    else:
        def failing(commands, verbose):
            if any(_build.MARSHAL_SOURCE in cmd for cmd in commands):
                raise RuntimeError("g++ failed (1)")
            run_all(commands, verbose)
        monkeypatch.setattr(_build, "_run_all", failing)
    with open(libs[3], "wb") as f:      # of an earlier build: its calls may no longer fit
        f.write(b"old")
    with pytest.warns(RuntimeWarning, match="host library is not built"):
        _build.build()
    assert sorted(os.listdir(tmp_path)) == sorted(os.path.basename(lib) for lib in libs[:3])
    with pytest.warns(RuntimeWarning, match="host library is not built"):
        _build.ensure_built()           # the others are there
