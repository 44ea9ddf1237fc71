"""Build libanchorattn.so in-tree with nvcc for sm_103a (no cmake, parallel TUs), and _calls.so, the per-step calls
of the serving operators for Python, which links to it and to torch."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libanchorattn.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SOURCE = "torch_calls.cpp"
CALLS_FOR = os.path.join(BUILD, "calls_for.txt")  # what _calls.so was compiled for
SOURCES = ["plan.cpp", "rope.cu", "fwd.cu", "bwd.cu", "bwd_static.cu", "shift_diag.cu", "segments.cu",
           "rope_axes.cu", "cache.cpp", "cache_io.cu", "cache_attend.cu",
           "cache_attend_short.cu", "cache_attend_short_fp8.cu", "cache_attend_chunk.cu",
           "cache_attend_chunk_fp8.cu", "cache_attend_wide.cu", "cache_tree.cu"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libanchorattn.so")
    return cand


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    cmd = [_nvcc(), ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
           "-I" + os.path.join(ROOT, "include"), "-c", path, "-o", obj]
    if src.endswith(".cu"):
        cmd[3:3] = ["--expt-relaxed-constexpr"]
    else:
        cmd[1:2] = ["-x", "c++"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _torch():
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: it is required to build _calls.so")
    return spec.submodule_search_locations[0]


def _compile_calls(src: str) -> str:
    obj, torch = os.path.join(BUILD, os.path.splitext(src)[0] + ".o"), _torch()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    dirs = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, src), "-o", obj] +
                       [x for d in dirs for x in ("-isystem", d)], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(cmd, target):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {target} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(target + ".tmp", target)


def _calls_for() -> str:
    with open(os.path.join(_torch(), "version.py")) as f:
        return f"{sys.version}\n{f.read()}"


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS) or not os.path.exists(CALLS_FOR):
        return True
    with open(CALLS_FOR) as f:
        if f.read() != _calls_for():  # another torch or Python since
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "anchorattn.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = True) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls, CALLS_SOURCE)
        objs = list(ex.map(_compile, SOURCES))
        calls = calls.result()
    _link([_nvcc(), "-shared", "-cudart", "static", "-o", LIB + ".tmp"] + objs + ["-lpthread", "-ldl", "-lrt"], LIB)
    lib = os.path.join(_torch(), "lib")
    if os.path.exists(CALLS_FOR):
        os.remove(CALLS_FOR)
    _link(["g++", "-shared", "-o", CALLS + ".tmp", calls, "-L" + PKG, "-l:" + os.path.basename(LIB), "-L" + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(_calls_for())
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv)
