"""Build libfcm.so in-tree with nvcc for sm_103a (GB300), one object per translation unit,
compiled in parallel, then linked into a shared library next to this file.

build(debug=True) builds libfcm_debug.so instead (objects in _build_debug): the same library
with the kernels' index checks compiled in (FCM_DEBUG_CHECKS), which record the first failed
check in the handle's error word for fcm_check to report.  Load it with load_library(path) or
the FCM_LIBRARY environment variable.

Beside the library, g++ compiles _tensor_calls.so, the Python binding's argument marshalling from
torch tensors (csrc/tensor_calls.cpp), against the torch that is installed."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfcm.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libfcm_debug.so")
TENSOR_CALLS = os.path.join(HERE, "_tensor_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def build_tensor_calls() -> str | None:
    """Compile _tensor_calls.so; None where torch is not installed (the C ABI needs none)."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = TENSOR_CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-I", os.path.join(torch, "include"),
           "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           os.path.join(CSRC, "tensor_calls.cpp"), "-o", tmp,
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on tensor_calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSOR_CALLS)
    return TENSOR_CALLS


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          debug: bool = False) -> str:
    """Compile every csrc/*.cu and link libfcm.so (libfcm_debug.so with debug=True).  Returns
    the library path."""
    lib, bdir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    def current(path: str) -> bool:
        return not force and os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()

    if current(lib):
        if not current(TENSOR_CALLS):
            build_tensor_calls()
        return lib
    os.makedirs(bdir, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (extra or []) + (["-DFCM_DEBUG_CHECKS"] if debug else [])

    def compile_one(src: str) -> str:
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        calls = None if current(TENSOR_CALLS) else ex.submit(build_tensor_calls)
        objs = list(ex.map(compile_one, srcs))
        if calls is not None:
            calls.result()
    tmp = lib + ".tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
