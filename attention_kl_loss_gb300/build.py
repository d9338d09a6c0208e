"""Build the in-tree shared library ``_lib/libstreamkl.so`` with nvcc.

Every translation unit is compiled for sm_103a only (GB300), in parallel, then
linked with the static CUDA runtime. Nothing is installed outside the tree.

``build(debug=True)`` builds ``_lib/libstreamkl_debug.so`` from the same
sources with STREAMKL_DEVICE_CHECKS defined: the kernels then check the
operands of every TMA copy, TMEM access and mbarrier against their layout
and report a failed check as STREAMKL_ERR_DEVICE_CHECK in the caller's
status word instead of issuing the access.

``build()`` also makes ``_lib/_marshal_<torch version>.so``, the Python module
that takes tensors to the operators' C entries (``csrc/marshal.cpp``). It is
tied to the version of PyTorch that it was built with, the library is not. It
only saves host time, so where it cannot be built (it needs a C++ compiler, the
headers of Python and of a CUDA build of PyTorch) ``build()`` says so and goes on.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
LIB_NAME = "libstreamkl.so"
DEBUG_LIB_NAME = "libstreamkl_debug.so"
SOURCES = ["api.cu", "fwd.cu", "bwd.cu", "bwd_sep.cu", "bwd_short.cu", "bwd_fused.cu", "bwd_fused128.cu",
           "api_ops.cu", "rope.cu", "paged_attn.cu", "paged_decode.cu", "paged_tree.cu", "pages.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def lib_path(debug: bool = False) -> str:
    return os.path.join(OUT_DIR, DEBUG_LIB_NAME if debug else LIB_NAME)


def marshal_path() -> str:
    import torch
    return os.path.join(OUT_DIR, f"_marshal_{re.sub('[^0-9A-Za-z]', '_', torch.__version__)}.so")


def _marshal_cmd() -> list:
    import torch
    inc, lib = (os.path.join(os.path.dirname(torch.__file__), d) for d in ("include", "lib"))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [os.path.join(ROOT, "include"), inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            *(f"-I{d}" for d in dirs), os.path.join(CSRC, "marshal.cpp"), "-o", marshal_path(), f"-L{lib}",
            "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_marshal(header: str, force: bool, verbose: bool) -> None:
    """The native module, if stale. A failure is no failure of the build: calls
    then go through ctypes, and a module of older sources is not left behind."""
    target = marshal_path()
    if not (force or _stale(target, [os.path.join(CSRC, "marshal.cpp"), header])):
        return
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        output, failed = "no Python.h\n", True
    else:
        try:
            p = subprocess.run(_marshal_cmd(), capture_output=True, text=True)
            output, failed = p.stdout + p.stderr, p.returncode != 0
        except OSError as error:  # no such compiler
            output, failed = f"{error}\n", True
    if verbose or failed:
        sys.stderr.write(output)
    if failed:
        if os.path.exists(target):
            os.remove(target)
        sys.stderr.write(f"{os.path.basename(target)} was not built: calls around the KL will go through ctypes "
                         "and take longer on the host\n")


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False,
          debug: bool = False) -> str:
    """Compile (if stale) and return the library path (the debug build with
    device-side range checks when ``debug``)."""
    os.makedirs(OUT_DIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "streamkl.h"))
    objs = []
    jobs = []
    tag = "_debug" if debug else ""
    extra = ["-DSTREAMKL_DEVICE_CHECKS"] if debug else []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, src.replace(".cu", f"{tag}.o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)

    def run(cmd):
        p = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, p

    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        marshal = None if debug else ex.submit(_build_marshal, headers[-1], force, verbose)
        for cmd, p in ex.map(run, jobs):
            if verbose or ptxas_info or p.returncode != 0:
                sys.stderr.write(p.stdout + p.stderr)
            if p.returncode != 0:
                raise RuntimeError(f"compiling failed: {' '.join(cmd)}")
    if marshal is not None:
        marshal.result()
    lib = lib_path(debug)
    if force or _stale(lib, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", lib, *objs]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            sys.stderr.write(p.stdout + p.stderr)
            raise RuntimeError(f"link failed: {' '.join(cmd)}")
    return lib


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="-v" in sys.argv, force="-f" in sys.argv,
                debug="--debug" in sys.argv))
