"""Build in-tree: libmpnum.so (nvcc for sm_103a, one object per .cu, compiled in
parallel) and _mpcall, the native argument marshalling of the block operators: an
extension of the running interpreter, named with its ABI tag so that another one
neither loads it nor takes it as up to date.  Where that interpreter's headers are
missing it is left out, and the package marshals in Python."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmpnum.so")
CALL = os.path.join(PKG, "_mpcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
UNTAGGED = os.path.join(PKG, "_mpcall.so")  # the extension's name in earlier builds
PYTHON_H = os.path.join(sysconfig.get_paths()["include"], "Python.h")
HEADER = os.path.join(ROOT, "include", "mpnum.h")

SOURCES = ["mp_common.cu", "mp_adamw.cu", "mp_fp8.cu", "mp_nvfp4.cu", "mp_mx.cu", "mp_norm.cu", "mp_swiglu.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = GENCODE + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                        "-I", os.path.join(ROOT, "include")]


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [HEADER, __file__]


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    cmd = ["nvcc", *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{p.stderr}")
    if verbose and p.stderr:
        sys.stderr.write(p.stderr)
    return obj


def _call_stale() -> bool:
    return os.path.exists(UNTAGGED) or ((os.path.exists(PYTHON_H) or os.path.exists(CALL)) and _stale(CALL))


def _compile_call() -> None:
    without = not os.path.exists(PYTHON_H)
    for old in (UNTAGGED, CALL) if without else (UNTAGGED,):  # nothing out of date stays to be loaded
        if os.path.exists(old):
            os.remove(old)
    if without:
        sys.stderr.write(f"{PYTHON_H} is missing: {os.path.basename(CALL)} is not built\n")
        return
    tmp = CALL + f".tmp{os.getpid()}"
    p = subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-Wall", "-Wextra", "-I", os.path.join(ROOT, "include"), "-I",
                        os.path.dirname(PYTHON_H), os.path.join(CSRC, "mp_call.c"), "-o", tmp],
                       capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"gcc failed for mp_call.c:\n{p.stderr}")
    os.replace(tmp, CALL)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu and link libmpnum.so and _mpcall next to this file; returns the library's path."""
    if not force and not _stale(LIB):
        if _call_stale():
            _compile_call()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call = ex.submit(_compile_call)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        call.result()
    tmp = LIB + f".tmp{os.getpid()}"
    p = subprocess.run(["nvcc", *GENCODE, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
