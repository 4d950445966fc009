"""Build libos2.so in-tree (rns_emulated_fp64_gb300/_build/) with nvcc.

Every CUDA source is compiled for sm_103a only, in parallel, then linked into
one shared library with the CUDA runtime linked statically.  The library has a
plain C ABI (include/os2.h); the Python binding loads it with ctypes.  Beside it
goes os2_head.so, the native argument checks of head.py (csrc/py_head.cpp, host
code built against the installed PyTorch).
"""
from __future__ import annotations

import glob
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
LIB = os.path.join(BUILD, "libos2.so")
# debug build: every kernel checks its hand-computed global indices (OS2_DEBUG)
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(BUILD_DEBUG, "libos2.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libos2")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def head_path() -> str:
    """The native part of head.py, for the PyTorch that is installed."""
    import torch
    return os.path.join(BUILD, f"os2_head-{torch.__version__}.so")


def build_head(force: bool = False) -> str:
    """Compile (if stale) and return the path of the native part of head.py."""
    import torch
    out, src, header = head_path(), os.path.join(CSRC, "py_head.cpp"), os.path.join(ROOT, "include", "os2.h")
    if not force and not _stale(out, [src, header]):
        return out
    os.makedirs(BUILD, exist_ok=True)
    base = os.path.dirname(torch.__file__)
    libs = os.path.join(base, "lib")
    incs = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
            os.path.join(base, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"],
            os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
                       + [f"-I{d}" for d in incs] + [src, "-o", tmp, f"-L{libs}", "-ltorch_python",
                       "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stderr}")
    os.replace(tmp, out)
    return out


def _stale(outputs: str, inputs: list[str]) -> bool:
    if not os.path.exists(outputs):
        return True
    t = os.path.getmtime(outputs)
    return any(os.path.getmtime(p) > t for p in inputs)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          debug: bool = False) -> str:
    """Compile (if stale) libos2.so and the native part of head.py, side by side, and
    return the path of libos2.so (debug: ``build_lib``'s, alone).  Where the native
    part cannot be built, that is raised after the library is there."""
    if debug:
        return build_lib(force, verbose, extra, debug)
    with ThreadPoolExecutor(max_workers=1) as ex:
        head = ex.submit(build_head, force)
        lib = build_lib(force, verbose, extra)
    head.result()
    return lib


def build_lib(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
              debug: bool = False) -> str:
    """Compile (if stale) and return the path of libos2.so (debug: the build with
    the kernels' index checks, in _build_debug/).  Needs nvcc alone."""
    bdir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    os.makedirs(bdir, exist_ok=True)
    headers = [h for d, ext in ((CSRC, "*.cuh"), (CSRC, "*.h"), (os.path.join(ROOT, "include"), "*.h"))
               for h in glob.glob(os.path.join(d, ext))]
    srcs = sources()
    if not force and not _stale(lib, srcs + headers + [__file__]):
        return lib
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]
    if debug:
        flags += ["-DOS2_DEBUG"]
    flags += list(extra or [])
    objs = []

    def compile_one(src):
        obj = os.path.join(bdir, os.path.basename(src) + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(os.cpu_count() or 8, len(srcs)))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if v else None
    print(build(force=True, verbose=v, extra=extra))
