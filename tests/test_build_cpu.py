"""The build script: what the files it leaves are like, without compiling."""
import os
import stat

import pytest

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
    _build.build()
    for lib in libs:
        assert stat.S_IMODE(os.stat(lib).st_mode) == 0o755, lib
    assert sorted(os.listdir(tmp_path)) == sorted(os.path.basename(lib) for lib in libs)
