"""Build libsdverify.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled in parallel to an object in _build/, then
linked with the static CUDA runtime into serving_sd_verify_gb300/libsdverify.so.
Beside them g++ compiles csrc/fast_calls.cpp, the Python binding's short way
into the library, against the installed torch; the file's name carries torch's and
Python's versions, so that another of either gets one of its own.  Where that
cannot be built (no g++, no headers, a torch without CUDA) a warning says so, and
the binding does without it.
The library links no libcuda: the one driver entry point it needs (tensor-map
encoding) is fetched at run time through the runtime's driver-entry-point
query, so the .so also loads on machines without a GPU driver.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsdverify.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsdverify")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _cxx11_abi() -> int:
    import torch
    return int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))


def fast_path() -> str:
    """The short way's file for the torch and the Python at hand."""
    import torch
    return os.path.join(PKG, f"_fast_calls.torch{torch.__version__}-abi{_cxx11_abi()}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _newer(out: str, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(ROOT, "include", "sd_verify.h"), os.path.abspath(__file__)])


def fast_up_to_date() -> bool:
    return _newer(fast_path(), [os.path.join(CSRC, "fast_calls.cpp"), os.path.join(ROOT, "include", "sd_verify.h"),
                                os.path.abspath(__file__)])


def _build_fast() -> None:
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(root, "lib")
    out = fast_path()
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={_cxx11_abi()}",
           *(a for d in inc for a in ("-isystem", d)), os.path.join(CSRC, "fast_calls.cpp"), "-o", tmp, "-L" + lib,
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fast_calls.cpp:\n{r.stderr}")
    os.replace(tmp, out)


def _try_build_fast() -> None:
    try:
        _build_fast()
    except (ImportError, AttributeError, OSError, RuntimeError) as e:
        warnings.warn(f"the binding's short way was not built: {e}", RuntimeWarning)


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link; returns the path of the shared library."""
    stale = force or not up_to_date()
    try:
        stale_fast = force or not fast_up_to_date()
    except (ImportError, AttributeError):
        stale_fast = True              # (no torch: said below)
    if not stale:
        if stale_fast:
            _try_build_fast()
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        fast = ex.submit(_try_build_fast) if stale_fast else None
        objs = list(ex.map(compile_one, sources()))
        if fast:
            fast.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))
