"""Build libmuir.so in-tree for B200 (sm_100a) with nvcc (cross-compiles without a GPU)."""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmuir.so")
# the checking build: the same library with device-side index checks (-DMUIR_CHECK)
CHECK_LIB = os.path.join(PKG, "libmuir_check.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "--expt-relaxed-constexpr",
]


# The translation units of the library, compiled side by side and linked.
UNITS = ("muir.cu", "layer.cu")
OBJ = os.path.join(PKG, "_build")


def sources(unit: str) -> list[str]:
    """The unit and every in-tree file it includes."""
    todo, seen = [os.path.join(CSRC, unit)], []
    while todo:
        f = os.path.normpath(todo.pop())
        if f in seen or not os.path.exists(f):
            continue
        seen.append(f)
        with open(f, encoding="utf-8") as src:
            todo += [os.path.join(os.path.dirname(f), m) for m in re.findall(r'^\s*#include "([^"]+)"', src.read(), re.M)]
    return seen


def _object(lib: str, unit: str) -> str:
    return os.path.join(OBJ, f"{os.path.basename(lib)[:-3]}_{unit[:-3]}.o")


def _stale(out: str, inputs: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in inputs)


def needs_build(lib: str = LIB) -> bool:
    return any(_stale(lib, sources(u)) for u in UNITS)


def _start(args: list[str], out: str, verbose: bool):
    cmd = [os.environ.get("NVCC", "nvcc"), *NVCC_FLAGS, *args, "-o", out + ".tmp"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _finish(proc, out: str, verbose: bool) -> None:
    text, err = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc failed ({proc.returncode}):\n{text}\n{err}")
    if verbose and (text or err):
        print(text + err, file=sys.stderr)  # e.g. the -Xptxas -v report
    os.replace(out + ".tmp", out)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, check: bool = False) -> str:
    """Build libmuir.so (and, with check=True, libmuir_check.so at the same time)."""
    os.makedirs(OBJ, exist_ok=True)
    libs = [(LIB, [])] + ([(CHECK_LIB, ["-DMUIR_CHECK"])] if check else [])
    todo = [(lib, flags) for lib, flags in libs if force or needs_build(lib)]
    jobs = []
    for lib, flags in todo:
        for u in UNITS:
            o = _object(lib, u)
            if force or _stale(o, sources(u)):
                jobs.append((o, _start([*(extra or []), *flags, "-c", os.path.join(CSRC, u)], o, verbose)))
    failed = None
    for o, proc in jobs:  # every compiler has ended before an error is raised
        try:
            _finish(proc, o, verbose)
        except RuntimeError as e:
            failed = failed or e
    if failed:
        raise failed
    for lib, _ in todo:
        _finish(_start(["-shared", *(_object(lib, u) for u in UNITS)], lib, verbose), lib, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None, check="--check" in sys.argv)
    print(LIB)
