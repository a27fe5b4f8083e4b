"""Builds libinjectstore.so in-tree for sm_100a (nvcc, no JIT cache).

    python -m kv_cache_injection_gather_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libinjectstore.so")
_HEADERS = [os.path.join(ROOT, "include", "inject_store.h")]
# every source and the headers it includes; each is compiled to an object of
# its own, side by side, and linked into the one library
UNITS = {
    os.path.join(CSRC, "inject_store.cu"): [os.path.join(CSRC, "inject_kernels.cuh"), *_HEADERS],
    os.path.join(CSRC, "query.cu"): [os.path.join(CSRC, "query_rows.cuh"), os.path.join(CSRC, "attend_common.cuh"),
                                     os.path.join(CSRC, "attend_rows.cuh"), os.path.join(CSRC, "attend_tiles.cuh"),
                                     os.path.join(ROOT, "include", "inject_query.h"), *_HEADERS],
}
SOURCES = list(UNITS)
DEPS = sorted(set(SOURCES).union(*UNITS.values()))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _object(source: str) -> str:
    return os.path.join(HERE, "build", os.path.basename(source) + ".o")


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(target) >= os.path.getmtime(d) for d in deps)


def compile_command(source: str, out: str, verbose: bool = False) -> list[str]:
    cmd = ["nvcc", "-O3", "-std=c++17", "-c", "-Xcompiler", "-fPIC,-O2", "-lineinfo", *ARCH,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-o", out, source]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def build(force: bool = False, verbose: bool = False) -> str:
    if not (force or verbose) and _newer(LIB, DEPS):
        return LIB
    os.makedirs(os.path.join(HERE, "build"), exist_ok=True)
    running = []
    for source, headers in UNITS.items():
        if force or verbose or not _newer(_object(source), [source, *headers]):
            tmp = _object(source) + f".tmp{os.getpid()}"
            running.append((subprocess.Popen(compile_command(source, tmp, verbose)), tmp, _object(source)))
    failed = None
    for proc, tmp, obj in running:
        if proc.wait() != 0:
            failed = subprocess.CalledProcessError(proc.returncode, proc.args)
        else:
            os.replace(tmp, obj)
    if failed:
        raise failed
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run(["nvcc", "-shared", *ARCH, "-o", tmp, *map(_object, SOURCES)], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
