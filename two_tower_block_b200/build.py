"""Build libtt_block_attn.so in-tree with nvcc for sm_100a.

Usage: python -m two_tower_block_b200.build [--force] [-v]
Objects go to two_tower_block_b200/_build/; the shared library is written
next to this file so that it travels with the source tree, and so is _marshal,
the argument marshalling of the Python binding (the only part that knows torch).
"""
from __future__ import annotations

import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtt_block_attn.so")
MARSHAL = os.path.join(HERE, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))   # of this Python's ABI
MARSHAL_FOR = os.path.join(BUILD, "marshal.torch")   # the torch that it was built against
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _marshal_cmd(src):
    import torch
    t = os.path.dirname(torch.__file__)
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DTT_TORCH_VERSION="{torch.__version__}"', "-I" + os.path.join(t, "include"),
            "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
            "-I" + sysconfig.get_paths()["include"], src, "-o", MARSHAL + ".tmp", "-L" + os.path.join(t, "lib"),
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]


def _torch_version():
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return ""


def _marshal_is_current(binding):
    """Newer than its source, and built against the torch that is installed: it uses torch's classes by their
    layout."""
    if not os.path.exists(MARSHAL) or os.path.getmtime(MARSHAL) < os.path.getmtime(binding):
        return False
    try:
        with open(MARSHAL_FOR) as f:
            return f.read() == _torch_version()
    except OSError:
        return False


def _build_marshal(binding):
    """The library does without it (ops.py has the same in Python), so a machine without a host compiler, or
    without Python's or torch's headers, is told and goes on."""
    try:
        r = subprocess.run(_marshal_cmd(binding), capture_output=True, text=True)
        why = r.stderr if r.returncode != 0 else None
    except (OSError, ImportError, AttributeError) as e:   # (AttributeError: a torch that is not whole)
        why = str(e)
    if why is None:
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(MARSHAL_FOR, "w") as f:
            f.write(_torch_version())
    else:
        sys.stderr.write(why)
        warnings.warn("the compiled argument marshalling could not be built: the binding's Python form will run")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    binding = os.path.join(CSRC, "marshal.cpp")
    srcs.remove(binding)
    hdr_mtime = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s) + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_mtime):
            cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_info and s.endswith(".cu") else [])
            cmd += ["-x", "cu" if s.endswith(".cu") else "c++", "-c", s, "-o", o]
            jobs.append(cmd)

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        for cmd, r in ex.map(run, jobs):
            if r.returncode != 0 or verbose or ptxas_info:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("build failed: " + " ".join(cmd))
    if jobs or force or not os.path.exists(LIB):
        cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", LIB + ".tmp"] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(LIB + ".tmp", LIB)
    if force or not _marshal_is_current(binding):
        _build_marshal(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
