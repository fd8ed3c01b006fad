"""Build liblinattn.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit under ``csrc/`` is compiled in parallel, then the
objects are linked into ``_build/liblinattn.so`` against the shared CUDA
runtime (the same libcudart.so that PyTorch loads).  Beside them the host
compiler builds ``_build/la_block.so``, the CPython face of the state-space
block's operators (it calls the library by address and serves both builds).
It needs PyTorch and its headers; the library does not, and is linked first.
Run as a module (``python -m causal_kernelized_linear_gb300.build``), as a
script where PyTorch is not installed (``python
causal_kernelized_linear_gb300/build.py``), or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "liblinattn.so")
# the LA_DEBUG build (device-side index checks), apart from the product library
DEBUG_BUILD_DIR = os.path.join(PKG_DIR, "_build_debug")
DEBUG_LIB_PATH = os.path.join(DEBUG_BUILD_DIR, "liblinattn.so")

# the CPython face of the block operators (against the installed PyTorch)
EXT_SRC = os.path.join(CSRC, "py_block.cpp")
EXT_PATH = os.path.join(BUILD_DIR, "la_block.so")
EXT_STAMP = EXT_PATH + ".for"   # the PyTorch and Python it was built for

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
CXX_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
             "--expt-relaxed-constexpr", "-Xptxas", "-O3"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblinattn")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(path: str, deps) -> bool:
    """Whether ``path`` exists and is newer than every one of ``deps``."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in deps)


def _ext_target() -> str:
    import torch
    return (f"PyTorch {torch.__version__}, Python {sys.version.split()[0]} "
            f"({sysconfig.get_config_var('SOABI')})")


def ext_built_for() -> str:
    """What ``la_block.so`` was built for ("" if that is not known)."""
    try:
        with open(EXT_STAMP) as f:
            return f.read()
    except OSError:
        return ""


def lib_up_to_date(debug: bool = False) -> bool:
    return _newer(DEBUG_LIB_PATH if debug else LIB_PATH, _deps())


def ext_up_to_date() -> bool:
    """Whether ``la_block.so`` is built from its source for this PyTorch and Python."""
    deps = [EXT_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return _newer(EXT_PATH, deps) and ext_built_for() == _ext_target()


def up_to_date(debug: bool = False) -> bool:
    return lib_up_to_date(debug) and ext_up_to_date()


def _build_ext():
    """Compile ``la_block.so`` with the host compiler; returns its log."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("a C++ compiler is required to build la_block")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    libs = library_paths()
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = EXT_PATH + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, *[a for p in include_paths() for a in ("-I", p)],
           "-I", sysconfig.get_paths()["include"], "-I", cuda, EXT_SRC, "-o", tmp,
           *[a for p in libs for a in ("-L" + p, "-Wl,-rpath," + p)],
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for {EXT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT_PATH)
    with open(tmp, "w") as f:
        f.write(_ext_target())
    os.replace(tmp, EXT_STAMP)
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False,
          debug: bool = False) -> str:
    """Compile every ``csrc/*.cu`` for sm_103a and link liblinattn.so; with
    ``debug``, the LA_DEBUG build (kernels check their indices) in a folder
    of its own.  ``la_block.so`` is left out where PyTorch is not installed; if
    it fails to compile, that is raised once the library is linked."""
    lib_path = DEBUG_LIB_PATH if debug else LIB_PATH
    try:
        import torch  # noqa: F401
        want_ext = force or not ext_up_to_date()
    except ImportError:
        want_ext = False
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(_build_ext) if want_ext else None
        if force or not lib_up_to_date(debug):
            _build_lib(lib_path, debug, verbose, ptxas_verbose)
        log = ext.result() if ext else ""
    if (verbose or ptxas_verbose) and log.strip():
        print(f"== la_block.so\n{log}", file=sys.stderr)
    return lib_path


def _build_lib(lib_path: str, debug: bool, verbose: bool, ptxas_verbose: bool):
    build_dir = os.path.dirname(lib_path)
    nvcc = _nvcc()
    os.makedirs(build_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    if debug:
        extra.append("-DLA_DEBUG")

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *CXX_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose or ptxas_verbose:
        for obj, log in results:
            if log.strip():
                print(f"== {os.path.basename(obj)}\n{log}", file=sys.stderr)
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-cudart", "shared", "-o", tmp,
           *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas-v" in sys.argv,
                debug="--debug" in sys.argv))
