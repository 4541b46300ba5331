"""Builds libsdpa_gb300.so in-tree with nvcc for sm_103a, and _sdpa_calls.so,
the Python entry of the paged-cache operators, with the host compiler.

Each .cu file compiles to an object in parallel; the objects link into one
shared library with the CUDA runtime linked statically, so loading the
library needs no GPU and no libcuda (the driver entry point used for TMA
descriptors is resolved at run time through the runtime).
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import threading
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libsdpa_gb300.so")
CALLS = os.path.join(BUILD, "_sdpa_calls.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + [os.path.join(ROOT, "include", "sdpa.h"), __file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _calls_stamp() -> str:
    import sysconfig
    import torch
    return f"{torch.__version__} {sysconfig.get_config_var('SOABI')}"


def calls_up_to_date() -> bool:
    stamp = CALLS + ".torch"  # the module goes with the torch and the Python it was built against
    if not (os.path.exists(CALLS) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        if f.read() != _calls_stamp():
            return False
    t = os.path.getmtime(CALLS)
    return all(os.path.getmtime(p) <= t for p in (CALLS_SRC, os.path.join(ROOT, "include", "sdpa.h"), __file__))


def build_calls(force: bool = False) -> str:
    """The CPython module that checks the paged-cache operators' tensors and calls the library."""
    if not force and calls_up_to_date():
        return CALLS
    import sysconfig
    import torch
    os.makedirs(BUILD, exist_ok=True)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    includes = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = CALLS + f".tmp{os.getpid()}.{threading.get_ident()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{p}" for p in includes] + [CALLS_SRC, "-o", tmp, "-L" + os.path.join(base, "lib")]
    cmd += ["-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {CALLS_SRC} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS + ".torch", "w") as f:
        f.write(_calls_stamp())
    return CALLS


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    flags += list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
    print(build_calls(force="--force" in sys.argv))
