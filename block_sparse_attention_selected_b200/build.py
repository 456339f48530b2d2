"""Builds the sm_100a CUDA library ``libnsa_sel.so`` in the package directory.

nvcc cross-compiles without a GPU.  The C ABI is declared in ``include/nsa_sel.h``.
Run ``python -m block_sparse_attention_selected_b200.build`` or call ``build()``.
"""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnsa_sel.so")
# the bounds-checking build (-DNSA_SEL_CHECKS): same ABI, every gathered row and K/V
# block coordinate checked before its copy (nsa_common.cuh)
LIB_CHECKS = os.path.join(HERE, "libnsa_sel_checks.so")
# the compiled marshalling of the paged-cache calls (a Python extension module)
LIB_BIND = os.path.join(HERE, "_paged_bind.so")
# ... and what it was built for: the Python and torch whose layouts are compiled into it
BIND_STAMP = os.path.join(HERE, "_build", "paged_bind.txt")
SOURCES = ["api.cu", "invert.cu", "fwd.cu", "merge.cu", "bwd.cu", "select.cu", "bsfa.cu",
           "paged.cu", "paged_attn.cu", "paged_few.cu",
           "paged_api.cu"]
HEADERS = ["nsa_common.cuh", "nsa_kernels.h", "paged.h", "paged_attn.cuh"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "nsa_sel.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def bind_target() -> str:
    """The Python and torch that run now, as _paged_bind.built_for names those it was built for."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__}"


def build_bind(force: bool = False) -> str:
    """Builds _paged_bind.so, the compiled marshalling of the paged-cache calls (g++ against the
    headers of the installed Python and torch); again where either has changed."""
    import sysconfig

    import torch
    src, header = os.path.join(CSRC, "paged_bind.cpp"), os.path.join(ROOT, "include", "nsa_sel.h")
    stamp = ""
    if os.path.exists(BIND_STAMP):
        with open(BIND_STAMP) as f:
            stamp = f.read()
    if not force and stamp == bind_target() and os.path.exists(LIB_BIND) and \
            os.path.getmtime(LIB_BIND) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return LIB_BIND
    base = os.path.dirname(torch.__file__)
    tmp = LIB_BIND + f".tmp{os.getpid()}"
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         f'-DNSA_BUILT_FOR="{bind_target()}"',
         "-isystem", os.path.join(base, "include"),
         "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
         "-I" + sysconfig.get_paths()["include"], src, "-o", tmp,
         "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, LIB_BIND)
    os.makedirs(os.path.dirname(BIND_STAMP), exist_ok=True)
    with open(BIND_STAMP, "w") as f:
        f.write(bind_target())
    return LIB_BIND


def build(force: bool = False, verbose: bool = False, checks: bool = False) -> str:
    """Builds libnsa_sel.so (checks=True: the bounds-checking libnsa_sel_checks.so), and the
    binding's compiled module, without which calls go a slower way."""
    lib = LIB_CHECKS if checks else LIB
    if force or _stale(lib):
        _build_library(lib, verbose, checks)
    try:
        build_bind(force)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"_paged_bind.so was not built, the paged calls are marshalled in Python: {e}")
    return lib


def _build_library(lib: str, verbose: bool, checks: bool) -> None:
    objdir = os.path.join(HERE, "_build_checks" if checks else "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [_nvcc(), *NVCC_FLAGS, *(["-DNSA_SEL_CHECKS"] if checks else []), "-I",
               os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        procs.append((subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), src))
        objs.append(obj)
    failed = []
    for p, src in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.check_call([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared",
                           "-o", tmp, *objs])
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                checks="--checks" in sys.argv))
