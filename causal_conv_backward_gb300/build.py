"""Builds libmcc1d.so in-tree with nvcc for sm_103a (GB300).

Translation units compile in parallel, then link into
``causal_conv_backward_gb300/_build/libmcc1d.so``. A build is skipped when the
library is newer than every source and header.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmcc1d.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmcc1d")
    return nvcc


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in deps)


def launch_registers(src: str) -> int:
    """The registers a thread that a source's kernels start with and share out again
    (setmaxnreg), 0 for sources that leave them as they are."""
    with open(src) as f:
        m = re.search(r"\bkRegLaunch = (\d+)", f.read())
    return int(m.group(1)) if m else 0


def check_registers(src: str, log: str) -> None:
    """Such kernels refuse to be launched with any other number: one that the
    compiler gave another fails here, not at its first call."""
    want, used = launch_registers(src), [int(n) for n in re.findall(r"Used (\d+) registers", log)]
    if want and (not used or any(n != want for n in used)):
        raise RuntimeError(f"{os.path.basename(src)}: its kernels are written for {want} registers a thread, the compiler used {used}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA/C++ source of the library for sm_103a; returns the .so path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs = []
    cmds = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        extra = ["-Xptxas", "-v"] if src.endswith(".cu") and (verbose or launch_registers(src)) else []
        cmds.append([nvcc, *ARCH, *COMMON, *extra, "-c", src, "-o", obj])
        objs.append(obj)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    # biggest translation units first, so they start early
    srcs = sources()
    order = sorted(range(len(cmds)), key=lambda k: -os.path.getsize(srcs[k]))
    cmds = [cmds[k] for k in order]
    objs = [objs[k] for k in order]
    with cf.ThreadPoolExecutor(max_workers=len(cmds)) as ex:
        logs = list(ex.map(run, cmds))
    for k, log in zip(order, logs):
        check_registers(srcs[k], log)
    if verbose:
        print("".join(logs))
    tmp = LIB + f".tmp{os.getpid()}"
    run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
