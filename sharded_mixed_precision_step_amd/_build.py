"""Build of libzerostep.so (the gfx950 kernels and the C-ABI host layer), of
libzerotwin.so (the benchmark's measurement aids, zero_twin.h) and of
workloads/libzerogen.so (the device side of the seeded input generators).

hipcc cross-compiles for gfx950 on any host, so this runs without a GPU.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libzerostep.so")
SOURCES = [os.path.join(CSRC, name) for name in (
    "zero_kernels.hip", "zero_abi.cpp",
    # the training operators (zero_train.h)
    "zero_train_abi.cpp", "zero_norm.hip", "zero_norm_backward.hip", "zero_q8.hip",
    "zero_q8_gemm.hip", "zero_distill.hip")]
TWIN_LIB = os.path.join(HERE, "libzerotwin.so")
TWIN_SOURCES = [os.path.join(CSRC, "zero_twin.hip")]
# the device side of the seeded input generators (workloads/), test and
# benchmark infrastructure
GEN_DIR = os.path.join(ROOT, "workloads", "csrc")
GEN_LIB = os.path.join(ROOT, "workloads", "libzerogen.so")
GEN_SOURCES = [os.path.join(GEN_DIR, "zero_gen.hip")]
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
                errors.append(f"hipcc failed ({proc.returncode}) for {cmd[-1]}:\n{out}\n{err}")
            elif verbose and err.strip():
                print(err, flush=True)
        if errors:
            raise RuntimeError("\n".join(errors))
    finally:
        for _, proc in procs:
            if proc.poll() is None:
                proc.kill()


def build(verbose: bool = False) -> str:
    """Compile the three libraries for gfx950: each source to an object (hipcc
    processes side by side), then each library from its objects, written
    atomically."""
    libs = ((LIB, SOURCES), (TWIN_LIB, TWIN_SOURCES), (GEN_LIB, GEN_SOURCES))
    compile_flags = [f for f in FLAGS if f != "-shared"]
    link_flags = [f"--offload-arch={ARCH}", "-fPIC", "-shared"]
    temps = []
    with tempfile.TemporaryDirectory(prefix="zerostep_build_") as objdir:
        try:
            compiles, links = [], []
            for lib, sources in libs:
                objects = []
                for src in sources:
                    obj = os.path.join(objdir, f"{len(compiles)}.o")
                    objects.append(obj)
                    compiles.append([hipcc(), *compile_flags, "-I", INCLUDE, "-I", CSRC, "-I",
                                     GEN_DIR, "-o", obj, "-c", src])
                name = os.path.basename(lib)
                fd, tmp = tempfile.mkstemp(prefix=f".{name}.", suffix=".tmp",
                                           dir=os.path.dirname(lib))
                os.close(fd)
                temps.append(tmp)
                links.append((lib, tmp, [hipcc(), *link_flags, *objects, "-o", tmp]))
            _run_all(compiles, verbose)
            _run_all([cmd for _, _, cmd in links], verbose)
            for lib, tmp, _ in links:
                os.replace(tmp, lib)
        finally:
            for tmp in temps:
                if os.path.exists(tmp):
                    os.unlink(tmp)
    return LIB


def ensure_built() -> str:
    """Build only if a library is missing."""
    if not all(os.path.exists(p) for p in (LIB, TWIN_LIB, GEN_LIB)):
        build()
    return LIB
