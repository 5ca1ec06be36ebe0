"""Build libcp.so (the CUDA lookup-decode and its C ABI) in-tree for sm_103a.

Each .cu file compiles in its own nvcc process (in parallel), then one link.
Output: trellis_row_decode_gb300/_build/libcp.so, and beside it _calls (cp_calls.cpp, host code for
this Python, linked to libcp.so; its file's name says for which), where the Python's headers are there.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
BUILD = PKG / "_build"
LIB = BUILD / "libcp.so"
CALLS = BUILD / ("_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
           "-I", str(ROOT / "include"), "-I", str(CSRC)]


def nvcc() -> str:
    for c in [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]:
        if c and Path(c).exists():
            return c
    raise RuntimeError("nvcc not found")


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def build_calls() -> Path | None:
    """_calls, linked to the libcp.so that is there; None where this Python's headers or g++ are not:
    the calls then go through ctypes alone."""
    include = Path(sysconfig.get_paths()["include"])
    if not (include / "Python.h").exists() or shutil.which("g++") is None:
        CALLS.unlink(missing_ok=True)            # (one that is there may be of another libcp.so)
        warnings.warn("no Python.h or g++: small calls of linear, linear_grad and dropout will take "
                      "longer on the host", RuntimeWarning, stacklevel=2)
        return None
    tmp = CALLS.with_name(f"{CALLS.name}.{os.getpid()}.tmp")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", str(include),
           "-I", str(ROOT / "include"), "-o", str(tmp), str(CSRC / "cp_calls.cpp"),
           "-L", str(BUILD), "-lcp", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for cp_calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    return CALLS


def build(verbose: bool = False, ptxas_info: bool = False) -> Path:
    BUILD.mkdir(parents=True, exist_ok=True)
    nv = nvcc()
    headers = list(CSRC.glob("*.h")) + list(CSRC.glob("*.cuh")) + list((ROOT / "include").glob("*.h"))
    newest_header = max((h.stat().st_mtime for h in headers), default=0)

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        if obj.exists() and obj.stat().st_mtime > max(src.stat().st_mtime, newest_header) \
                and not ptxas_info:
            return obj
        cmd = [nv, *ARCH, *NVFLAGS, "-c", str(src), "-o", str(obj)]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB.with_suffix(f".{os.getpid()}.tmp.so")
    cmd = [nv, *ARCH, "-shared", "-o", str(tmp), *map(str, objs), "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_calls()
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_info="-v" in sys.argv))
