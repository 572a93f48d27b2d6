"""Build of libzerostep.so (the gfx950 kernels and the C-ABI host layer), of
libzerotwin.so (the benchmark's measurement aids, zero_twin.h), of
workloads/libzerogen.so (the device side of the seeded input generators) and of
the binding's host library _marshal (what it reads off tensors).

hipcc cross-compiles for gfx950 on any host, so this runs without a GPU.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libzerostep.so")
SOURCES = [os.path.join(CSRC, name) for name in (
    "zero_kernels.hip", "zero_abi.cpp",
    # the training operators (zero_train.h)
    "zero_train_abi.cpp", "zero_norm.hip", "zero_norm_backward.hip", "zero_q8.hip",
    "zero_q8_gemm.hip", "zero_distill.hip",
    # the operators of zero_model.h
    "zero_model_abi.cpp", "zero_embed.hip", "zero_layernorm.hip", "zero_layernorm_backward.hip",
    "zero_act.hip", "zero_logprob.hip")]
TWIN_LIB = os.path.join(HERE, "libzerotwin.so")
TWIN_SOURCES = [os.path.join(CSRC, "zero_twin.hip")]
# the device side of the seeded input generators (workloads/), test and
# benchmark infrastructure
GEN_DIR = os.path.join(ROOT, "workloads", "csrc")
GEN_LIB = os.path.join(ROOT, "workloads", "libzerogen.so")
GEN_SOURCES = [os.path.join(GEN_DIR, "zero_gen.hip")]
# host code against torch's and Python's headers, by g++: it holds internal symbols of
# both, so each pair has a file of its own and none loads another's
MARSHAL_LIB = os.path.join(HERE, f"_marshal.{sysconfig.get_config_var('SOABI')}."
                                 f"torch-{torch.__version__}.so")
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # every fp32 operation separately rounded, as the step is defined
    "-ffp-contract=off",
    # no packed fp32 arithmetic in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _marshal_includes() -> list:
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    return [root, os.path.join(root, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"]]


def marshal_missing() -> Optional[str]:
    """What its build lacks here, or None.  The package does without the library (train.py)."""
    if shutil.which("g++") is None:
        return "g++"
    for header in ("torch/csrc/autograd/python_variable.h", "Python.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in _marshal_includes()):
            return header
    return None


def marshal_command(out: str) -> list:
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return [shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(a for d in _marshal_includes() for a in ("-isystem", d)), "-I", INCLUDE,
            MARSHAL_SOURCE, "-o", out, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch",
            "-lc10"]


def _drop_marshals() -> None:
    """Remove host libraries of earlier builds, of every Python and torch: they may call
    the others by signatures that those no longer have."""
    folder = os.path.dirname(MARSHAL_LIB)
    for name in os.listdir(folder):
        if name.startswith("_marshal.") and name.endswith(".so"):
            os.unlink(os.path.join(folder, name))


def build_marshal(verbose: bool = False) -> Optional[str]:
    """Compile the binding's host library, written atomically.  Where that is not
    possible a warning says why, and the binding goes without it."""
    missing = marshal_missing()
    if missing is None:
        tmp = None
        try:
            tmp = _temp(MARSHAL_LIB)
            _run_all([marshal_command(tmp)], verbose)
            _put(tmp, MARSHAL_LIB)
            return MARSHAL_LIB
        except (RuntimeError, OSError) as e:
            missing = str(e)
        finally:
            if tmp is not None and os.path.exists(tmp):
                os.unlink(tmp)
    warnings.warn(f"the binding's host library is not built, calls go through ctypes: {missing}",
                  RuntimeWarning, stacklevel=2)
    return None


def code_text(src: str) -> str:
    """C/C++ source with its comments removed and each run of whitespace
    collapsed to one space: what the compiler sees, so that editing a comment
    does not change a digest.  String and character literals are kept as
    they are."""
    out, i, n = [], 0, len(src)
    while i < n:
        c = src[i]
        if c in "\"'":
            j = i + 1
            while j < n and src[j] != c:
                j += 2 if src[j] == "\\" else 1
            out.append(src[i:j + 1])
            i = j + 1
        elif src.startswith("//", i):
            j = src.find("\n", i)
            i = n if j < 0 else j
        elif src.startswith("/*", i):
            j = src.find("*/", i + 2)
            out.append(" ")
            i = n if j < 0 else j + 2
        else:
            out.append(c)
            i += 1
    return " ".join("".join(out).split())


def kernel_digest() -> str:
    """SHA-256 over the code of the sources that fix the kernels' code and
    launch shapes (the device source and the internal header), comments and
    layout aside.  Hardware counters taken on one digest do not describe
    kernels built from another."""
    import hashlib
    h = hashlib.sha256()
    for p in (os.path.join(CSRC, "zero_kernels.hip"), os.path.join(CSRC, "zero_internal.h")):
        with open(p, encoding="utf-8") as f:
            h.update(os.path.basename(p).encode())
            h.update(code_text(f.read()).encode())
    return h.hexdigest()


def _source(cmd) -> str:
    """The source that a command compiles, or the file that it links."""
    sources = [a for a in cmd if a.endswith((".hip", ".cpp"))]
    return sources[0] if sources else cmd[cmd.index("-o") + 1]


def _run_all(commands, verbose: bool) -> None:
    """Run the commands side by side; raise with the output of those that fail."""
    procs = []
    try:
        for cmd in commands:
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.PIPE, text=True)))
        errors = []
        for cmd, proc in procs:
            out, err = proc.communicate()
            if proc.returncode != 0:
                errors.append(f"{os.path.basename(cmd[0])} failed ({proc.returncode}) for "
                              f"{_source(cmd)}:\n{out}\n{err}")
            elif verbose and err.strip():
                print(err, flush=True)
        if errors:
            raise RuntimeError("\n".join(errors))
    finally:
        for _, proc in procs:
            if proc.poll() is None:
                proc.kill()


def _temp(lib: str) -> str:
    """A new file beside the library, to be put in its place."""
    fd, tmp = tempfile.mkstemp(prefix=f".{os.path.basename(lib)}.", suffix=".tmp",
                               dir=os.path.dirname(lib))
    os.close(fd)
    return tmp


def _put(tmp: str, lib: str) -> None:
    os.chmod(tmp, 0o755)  # g++ leaves the temporary file's mode, its owner's alone
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    """Compile the three libraries for gfx950, each source to an object (hipcc
    processes side by side), then each library from its objects, and the
    binding's host library; each written atomically."""
    libs = ((LIB, SOURCES), (TWIN_LIB, TWIN_SOURCES), (GEN_LIB, GEN_SOURCES))
    compile_flags = [f for f in FLAGS if f != "-shared"]
    link_flags = [f"--offload-arch={ARCH}", "-fPIC", "-shared"]
    temps = []
    with tempfile.TemporaryDirectory(prefix="zerostep_build_") as objdir, \
            ThreadPoolExecutor(1) as beside:
        _drop_marshals()
        host = beside.submit(build_marshal, verbose)
        try:
            compiles, links = [], []
            for lib, sources in libs:
                objects = []
                for src in sources:
                    obj = os.path.join(objdir, f"{len(compiles)}.o")
                    objects.append(obj)
                    compiles.append([hipcc(), *compile_flags, "-I", INCLUDE, "-I", CSRC, "-I",
                                     GEN_DIR, "-o", obj, "-c", src])
                temps.append(_temp(lib))
                links.append((lib, temps[-1], [hipcc(), *link_flags, *objects, "-o", temps[-1]]))
            _run_all(compiles, verbose)
            _run_all([cmd for _, _, cmd in links], verbose)
            for lib, tmp, _ in links:
                _put(tmp, lib)
        finally:
            for tmp in temps:
                if os.path.exists(tmp):
                    os.unlink(tmp)
        host.result()
    return LIB


def ensure_built() -> str:
    """Build only what is missing."""
    if not all(os.path.exists(p) for p in (LIB, TWIN_LIB, GEN_LIB)):
        build()
    elif not os.path.exists(MARSHAL_LIB):
        build_marshal()
    return LIB
