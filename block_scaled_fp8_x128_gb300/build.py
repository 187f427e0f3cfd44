"""Builds libr9q.so in-tree: every CUDA translation unit compiled for sm_103a in
parallel with nvcc, then linked into one shared library (static cudart, no
libcuda link: the tensor-map encoder is fetched through the runtime's driver
entry-point query).  Beside it _calls.so, the Python side of the calls that last
microseconds (host C++, against the installed torch)."""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libr9q.so")
CALLS = os.path.join(PKG, "_calls.so")
BUILD_DIR = os.path.join(ROOT, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
    "-I", CSRC,
]


# per-translation-unit extra nvcc flags
PER_FILE_FLAGS: dict[str, list[str]] = {}


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _torch_version() -> str:
    text = open(os.path.join(_torch_dir(), "version.py")).read()
    return re.search(r"^__version__ = ['\"](.+)['\"]", text, re.M).group(1)


def _built_for() -> str:
    """What _calls.so depends on beside its sources."""
    return f"torch {_torch_version()} {sys.implementation.cache_tag}\n"


def _other_than(path: str, text: str) -> bool:
    return not os.path.exists(path) or open(path).read() != text


def _calls_compile(src: str, obj: str) -> list[str]:
    include = os.path.join(_torch_dir(), "include")
    paths = [include, os.path.join(include, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
             os.path.join(ROOT, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", f'-DR9Q_TORCH_VERSION="{_torch_version()}"', *(f"-I{p}" for p in paths),
            "-c", src, "-o", obj]


def _calls_link(obj: str, out: str) -> list[str]:
    """It finds libr9q.so beside itself; torch's libraries are those that are loaded."""
    return ["g++", "-shared", obj, "-o", out, f"-L{PKG}", "-lr9q", f"-L{os.path.join(_torch_dir(), 'lib')}",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if stale) and return the path of libr9q.so."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                     glob.glob(os.path.join(ROOT, "include", "*.h")))
    nvcc = _nvcc()
    procs, objs = [], []
    for src in sources:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *NVCC_FLAGS, *PER_FILE_FLAGS.get(os.path.basename(src), []), "-c", src, "-o", obj]
            if verbose_ptxas:
                cmd[1:1] = ["-Xptxas", "-v"]
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    calls_src, calls_obj = os.path.join(CSRC, "r9q_calls.cpp"), os.path.join(BUILD_DIR, "r9q_calls.o")
    record = os.path.join(BUILD_DIR, "r9q_calls.for")
    other = _other_than(record, _built_for())
    if force or other or _stale(calls_obj, [calls_src, *headers]):
        procs.append((calls_src, subprocess.Popen(_calls_compile(calls_src, calls_obj), stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose_ptxas and text:
            sys.stderr.write(text)
    msg = "compilation failed:\n" + "\n".join(f"--- {s}\n{t}" for s, t in failed)
    if any(s != calls_src for s, _ in failed):
        raise RuntimeError(msg)
    if force or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp, *objs]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if failed:                                                # libr9q.so is there for what does without _calls.so
        raise RuntimeError(msg)
    if force or other or _stale(CALLS, [calls_obj]):
        tmp = CALLS + ".tmp.%d" % os.getpid()
        subprocess.run(_calls_link(calls_obj, tmp), check=True)
        os.replace(tmp, CALLS)
        with open(record, "w") as f:
            f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
