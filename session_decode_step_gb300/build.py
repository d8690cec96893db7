"""Build libkd.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file compiles in parallel into _build/, then one shared library is
linked next to this file.  No CMake; the static CUDA runtime is linked in, so
loading the library needs no GPU (a call that reaches CUDA then fails cleanly).
The binding's marshalling module, _kdcall, is compiled for the running Python and
linked against it; its file carries the interpreter's ABI suffix.  Without a C compiler
or Python's headers it is left out, and the binding makes those calls through ctypes.
"""
from __future__ import annotations

import importlib.machinery
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = PKG / "libkd.so"
CALL = PKG / ("_kdcall" + importlib.machinery.EXTENSION_SUFFIXES[0])

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v",
              f"-I{INCLUDE}", f"-I{CSRC}"] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkd.so")


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _older(target: Path, deps) -> bool:
    """target is missing, or older than one of deps or than the headers and this file."""
    if not target.exists():
        return True
    t = target.stat().st_mtime
    return any(d.stat().st_mtime > t for d in [*deps, *INCLUDE.glob("*.h"), Path(__file__)])


def _stale() -> bool:
    return _older(LIB, [*_sources(), *CSRC.glob("*.h"), *CSRC.glob("*.cuh")])


def _cc():
    return os.environ.get("CC") or shutil.which("cc") or shutil.which("gcc")


def _python_headers():
    inc = Path(sysconfig.get_paths()["include"])
    return inc if (inc / "Python.h").exists() else None


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile every CUDA source, link libkd.so and compile the marshalling module; returns libkd.so's path."""
    if force or _stale():
        _build_lib(verbose)
    if force or _older(CALL, [CSRC / "kd_py.c"]):
        _build_call()
    return LIB


def _build_lib(verbose: bool):
    BUILD.mkdir(exist_ok=True)
    nv = nvcc()

    def compile_one(src: Path):
        obj = BUILD / (src.stem + ".o")
        cmd = [nv] + NVCC_FLAGS + ["-c", str(src), "-o", str(obj)]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            print(log)
    (BUILD / "ptxas.log").write_text("".join(log for _, log in results))
    tmp = str(LIB) + ".tmp"
    cmd = [nv, "-shared", "-o", tmp] + [str(o) for o, _ in results] + ARCH + ["-lcudart_static", "-ldl",
                                                                            "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking libkd.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_call():
    cc, headers = _cc(), _python_headers()
    if not cc or not headers:
        CALL.unlink(missing_ok=True)  # what is there is out of date
        return
    tmp = str(CALL) + ".tmp"
    cmd = [cc, "-O2", "-fPIC", "-shared", "-Wall", f"-I{headers}", f"-I{INCLUDE}",
           str(CSRC / "kd_py.c"), "-o", tmp, f"-L{PKG}", "-l:libkd.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {CALL.name} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
