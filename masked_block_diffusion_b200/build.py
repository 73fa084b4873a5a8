"""Builds libdllm.so (and the synthetic-weight filler libsynth.so) in-tree for sm_100a."""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdllm.so")
SYNTH_SRC = os.path.join(ROOT, "synth", "csrc", "synth_fill.cu")
SYNTH_LIB = os.path.join(ROOT, "synth", "libsynth.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMMON = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC"]
# the library's translation units, compiled side by side, and the headers each one reads
UNITS = {
    "engine": ["attention.cuh", "attention_tc.cuh", "common.cuh", "gemm_tc.cuh", "kernels.cuh"],
    "kv4": ["attention.cuh", "attention_tc.cuh", "common.cuh", "attention_kv4.cuh", "attention_kv4_tc.cuh", "kv4.cuh",
            "rope.cuh"],
}
OBJ = os.path.join(PKG, "_build")


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build_dllm(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    objs, running = [], []
    for name, headers in UNITS.items():
        obj = os.path.join(OBJ, name + ".o")
        objs.append(obj)
        srcs = [os.path.join(CSRC, f) for f in [name + ".cu", *headers]] + [os.path.join(INCLUDE, "dllm.h")]
        # without its object files (a tree that got the library alone) the library's own age counts
        if not force and not _stale(obj if os.path.exists(obj) else LIB, srcs):
            continue
        cmd = [nvcc(), *ARCH, *COMMON, "-c", "-I", INCLUDE, "-I", CSRC, os.path.join(CSRC, name + ".cu"), "-o", obj + ".tmp"]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        running.append((subprocess.Popen(cmd), cmd, obj))
    failed = None
    for p, cmd, obj in running:   # all of them, so that none still writes its file when a later build begins
        if p.wait() == 0:
            os.replace(obj + ".tmp", obj)
        elif failed is None:
            failed = subprocess.CalledProcessError(p.returncode, cmd)
    if failed is not None:
        raise failed
    # an object file may be newer than the library without a unit compiled here: the last link did not finish
    if running or _stale(LIB, [o for o in objs if os.path.exists(o)]):
        missing = [o for o in objs if not os.path.exists(o)]
        if missing:
            return build_dllm(True, verbose_ptxas)
        subprocess.run([nvcc(), *ARCH, "-shared", *objs, "-o", LIB + ".tmp"], check=True)
        os.replace(LIB + ".tmp", LIB)
    return LIB


def build_synth(force: bool = False) -> str:
    if force or _stale(SYNTH_LIB, [SYNTH_SRC]):
        cmd = [nvcc(), *ARCH, *COMMON, "-shared", SYNTH_SRC, "-o", SYNTH_LIB + ".tmp"]
        subprocess.run(cmd, check=True)
        os.replace(SYNTH_LIB + ".tmp", SYNTH_LIB)
    return SYNTH_LIB


def build_all(force: bool = False) -> None:
    build_dllm(force)
    build_synth(force)


if __name__ == "__main__":
    build_all(force="--force" in sys.argv)
    print(LIB)
    print(SYNTH_LIB)
