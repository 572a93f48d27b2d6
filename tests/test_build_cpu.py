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
