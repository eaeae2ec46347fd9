"""Builds ``libfp8q.so`` (the C-ABI library, nvcc for sm_100a) and ``_calls.so``
(argument marshalling of some of its calls, host C++ against torch) in-tree."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
LIB = PKG / "libfp8q.so"
CALLS = PKG / "_calls.so"
CALLS_SOURCE = CSRC / "fp8q_torch.cpp"
SOURCES = [CSRC / "fp8q_api.cu"]
DEPS = SOURCES + sorted(CSRC.glob("*.cuh")) + [ROOT / "include" / "fp8q.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-shared",
]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or "/usr/local/cuda/bin/nvcc"
    return cand if os.path.exists(cand) else "nvcc"


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile the library unless it is newer than every source."""
    if not force and LIB.exists():
        newest = max(p.stat().st_mtime for p in DEPS)
        if LIB.stat().st_mtime >= newest:
            return LIB
    tmp = LIB.with_name("libfp8q.so.tmp%d" % os.getpid())
    cmd = [nvcc()] + NVCC_FLAGS + ["-I", str(ROOT / "include"), "-I", str(CSRC)]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += ["-o", str(tmp)] + [str(s) for s in SOURCES]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build_calls(force: bool = False) -> Path:
    """Compile the marshalling module unless it is newer than its sources (it links to the library by name)."""
    deps = [CALLS_SOURCE, ROOT / "include" / "fp8q.h"]
    if not force and CALLS.exists() and CALLS.stat().st_mtime >= max(p.stat().st_mtime for p in deps):
        return CALLS
    import torch
    base = Path(torch.__file__).resolve().parent
    cuda = Path(nvcc()).resolve().parent.parent if os.path.exists(nvcc()) else Path("/usr/local/cuda")
    tmp = CALLS.with_name("_calls.so.tmp%d" % os.getpid())
    includes = [ROOT / "include", sysconfig.get_paths()["include"], base / "include",
                base / "include" / "torch" / "csrc" / "api" / "include", cuda / "include"]
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-DTORCH_API_INCLUDE_EXTENSION_H", "-DTORCH_EXTENSION_NAME=_calls",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    cmd += ["-I%s" % i for i in includes] + ["-o", str(tmp), str(CALLS_SOURCE), "-L" + str(PKG), "-l:" + LIB.name,
                                           "-Wl,-rpath,$ORIGIN"]
    cmd += ["-L%s" % (base / "lib"), "-L%s" % (cuda / "lib64")]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS)
    return CALLS


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    build_calls(force="--force" in sys.argv)
    print(LIB, CALLS)
