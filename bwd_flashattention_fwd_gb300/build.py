"""Build libgbattn.so in-tree with nvcc for sm_103a.

The kernel instantiations compile as one translation unit per head dimension
(inst.cu, cache_inst.cu and paged_inst.cu with -DGBATTN_HEAD_DIM=<D>), in parallel, plus the
C-ABI unit (api.cu), the linear cross-entropy unit (lce.cu), the cache unit (cache.cu) and the
unit of the calls around attention (step.cu); the objects link into
bwd_flashattention_fwd_gb300/libgbattn.so (no library besides the CUDA
runtime).  checks.cu becomes libgbattn_checks.so, a test aid, and binding.cpp
the extension module _binding, the Python binding's fast path.  It is compiled
against the headers of this Python and torch and reads torch's structures, so it is
built again when either changes.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgbattn.so")
CHECKS_LIB = os.path.join(PKG, "libgbattn_checks.so")  # device checks of the kernels' math helpers (tests only)
DEBUG_LIB = os.path.join(PKG, "libgbattn_debug.so")  # index checks compiled in (GBATTN_DEBUG_CHECKS)
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))  # fast path of the Python binding: tensors checked in C++
BINDING_STAMP = os.path.join(BUILD, "binding.txt")  # what it was built for
HEAD_DIMS = (64, 96, 128, 256)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def built_for() -> str:
    """What the Python extension depends on besides its source (it carries the same words)."""
    import torch

    return f"Python {sys.version_info[0]}.{sys.version_info[1]}, torch {torch.__version__}"


def _binding_cmd(out: str):
    """Compile and link the Python extension against the installed torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "g++"
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DGBATTN_BUILT_FOR="{built_for()}"',
            *(f"-I{d}" for d in inc),
            os.path.join(CSRC, "binding.cpp"), "-o", out, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def _sources_mtime() -> float:
    t = 0.0
    for d in (CSRC, os.path.join(ROOT, "include")):
        for f in os.listdir(d):
            t = max(t, os.path.getmtime(os.path.join(d, f)))
    return t


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + " ".join(cmd) + "\n" + r.stdout)
    return r.stdout


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _stale(debug: bool = False) -> tuple:
    """Whether the libraries, and the Python extension, have to be built."""
    newest = _sources_mtime()

    def old(path):
        return not os.path.exists(path) or os.path.getmtime(path) < newest

    libs = (DEBUG_LIB,) if debug else (LIB, CHECKS_LIB)
    return any(old(p) for p in libs), old(BINDING) or _read(BINDING_STAMP) != built_for()


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Compile what is stale and return the path of libgbattn.so (with debug:
    libgbattn_debug.so, the kernels' index checks compiled in).  Where the
    extension module cannot be compiled the libraries are there all the same
    when this raises."""
    lib = DEBUG_LIB if debug else LIB
    libs, binding = (True, True) if force else _stale(debug)
    if not libs and not binding:
        return lib
    bdir = os.path.join(BUILD, "debug") if debug else BUILD
    os.makedirs(bdir, exist_ok=True)
    jobs, objs = [], []
    checks_obj, tmp_binding = os.path.join(bdir, "checks.o"), BINDING + ".tmp"
    if libs:
        nvcc = _nvcc()
        flags = [*FLAGS, *extra_flags] + (["-DGBATTN_DEBUG_CHECKS"] if debug else [])
        for d in HEAD_DIMS:
            for unit in ("inst", "cache_inst", "paged_inst"):
                objs.append(os.path.join(bdir, f"{unit}_d{d}.o"))
                jobs.append([nvcc, *ARCH, *flags, f"-DGBATTN_HEAD_DIM={d}", "-c", os.path.join(CSRC, unit + ".cu"), "-o", objs[-1]])
        for unit in ("api", "lce", "cache", "step"):
            objs.append(os.path.join(bdir, unit + ".o"))
            jobs.append([nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, unit + ".cu"), "-o", objs[-1]])
        if not debug:
            jobs.append([nvcc, *ARCH, *flags, "-c", os.path.join(CSRC, "checks.cu"), "-o", checks_obj])
    with ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        module = ex.submit(lambda: _run(_binding_cmd(tmp_binding))) if binding else None
        outs = list(ex.map(_run, jobs))
        if libs:
            for out, parts in ((lib, objs), *(() if debug else ((CHECKS_LIB, [checks_obj]),))):
                _run([nvcc, *ARCH, "-shared", "-o", out + ".tmp", *parts])
                os.replace(out + ".tmp", out)
    if module:
        outs.append(module.result())
    if verbose:
        for o in outs:
            sys.stdout.write(o)
    if binding:
        os.replace(tmp_binding, BINDING)
        with open(BINDING_STAMP, "w") as f:
            f.write(built_for())
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else (), debug="--debug" in sys.argv))
