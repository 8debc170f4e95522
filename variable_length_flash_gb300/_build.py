"""Builds, in-tree and without cmake, libvlf.so from csrc/*.cu with nvcc for sm_103a (parallel TUs) and
_calls.so, the native side of the decoding entry points' Python calls, from csrc/calls.cpp with g++."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libvlf.so")
CALLS_SRC = os.path.join(CSRC, "calls.cpp")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_FOR = os.path.join(BUILD, "calls.for")  # what _calls.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(sources, headers, target=LIB) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in sources + headers)


def _calls_for() -> str:
    """The torch and the Python that are installed."""
    import sysconfig

    import torch
    return f"{torch.__version__} {sysconfig.get_config_var('EXT_SUFFIX')}"


def _calls_stale() -> bool:
    """Whether _calls.so is older than its sources or was built for another torch or Python."""
    try:
        with open(CALLS_FOR) as f:
            built_for = f.read()
    except OSError:
        return True
    return built_for != _calls_for() or _stale([CALLS_SRC], [os.path.join(ROOT, "include", "vlf.h")], CALLS)


def _build_calls() -> str:
    """Compile csrc/calls.cpp against the torch that is installed."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), os.path.join(ROOT, "include"), sysconfig.get_paths()["include"]]
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fno-strict-aliasing",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DVLF_TORCH="{torch.__version__}"', *[f"-isystem{i}" for i in inc], CALLS_SRC, "-o", tmp,
           "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    os.makedirs(BUILD, exist_ok=True)
    with open(CALLS_FOR, "w") as f:
        f.write(_calls_for())
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu and link libvlf.so next to this file; returns its path."""
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                     glob.glob(os.path.join(ROOT, "include", "*.h")))
    calls = force or _calls_stale()
    if not force and not _stale(sources, headers):
        if calls:
            _build_calls()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(sources) + 1)) as ex:
        pending = ex.submit(_build_calls) if calls else None
        objs = list(ex.map(compile_one, sources))
        if pending:
            pending.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
