"""Build the sm_103a shared library ``libmoe_w4a16.so`` in-tree with nvcc, and
the attention operators' Python binding ``_attn_binding``.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into one
shared library next to this file. ``csrc/binding.c`` is host code for one version
of Python, which its file name says; without the Python headers it is left out, and
only the attention operators' Python calls miss it. Rebuilds what is older than its
sources.

    python -m w4a16_routed_expert_router_gb300._build [--force] [--verbose]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_w4a16.so")
BINDING_SRC = os.path.join(CSRC, "binding.c")
BINDING = os.path.join(PKG, "_attn_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_w4a16")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(path, deps) -> bool:
    return not os.path.exists(path) or any(
        os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _stale() -> bool:
    """The library is missing or older than a source."""
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return _older(LIB, deps + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def python_headers():
    """The folder of Python.h, or None."""
    path = sysconfig.get_paths()["include"]
    return path if os.path.exists(os.path.join(path, "Python.h")) else None


def build_binding(force: bool = False) -> bool:
    """The Python binding for this interpreter; False where it has no headers."""
    headers = python_headers()
    if headers is None:
        return False
    deps = [BINDING_SRC, os.path.join(INCLUDE, "moe_attn.h"), os.path.abspath(__file__)]
    if not force and not _older(BINDING, deps):
        return True
    tmp = BINDING + ".tmp"
    cmd = [nvcc(), "-O2", "-cudart", "none", "-shared", "-Xcompiler", "-fPIC", "-I" + headers,
           BINDING_SRC, "-o", tmp]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"building {BINDING_SRC} failed:\n{res.stderr}")
    os.replace(tmp, BINDING)
    return True


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not build_binding(force):
        sys.stderr.write("no Python headers: built without the attention operators' binding\n")
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    xflags = list(extra)
    if verbose:
        xflags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *xflags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        return obj, res.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, sources()))
    for _, log in results:
        if verbose and log:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
