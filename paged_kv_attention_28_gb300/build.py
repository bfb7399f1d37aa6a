"""Build the sm_103a shared library ``libpkvattn.so`` in-tree with nvcc.

Each ``csrc/*.cu`` file compiles to an object in parallel, then one link step
makes the library. The CUDA runtime is linked statically, and nothing links
against the driver library, so the library also loads on a machine without a
GPU (for the export checks). ``csrc/pycall.cpp`` becomes ``_pycall.so``, the CPython
module of the binding's small calls, linked against the library. Run ``python -m paged_kv_attention_28_gb300.build``.
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
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpkvattn.so")
PYCALL = os.path.join(PKG, "_pycall.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkvattn.so")


def torch_lib() -> str:
    import torch  # for the place of its headers and libraries

    return os.path.join(os.path.dirname(torch.__file__), "lib")


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _needs_rebuild(srcs) -> bool:
    if not os.path.exists(LIB) or not os.path.exists(PYCALL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(PYCALL))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if not force and not _needs_rebuild(srcs):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = _flags(verbose_ptxas)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    def compile_pycall():
        inc = os.path.join(os.path.dirname(torch_lib()), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")
        src, obj = os.path.join(CSRC, "pycall.cpp"), os.path.join(BUILD, "pycall.cpp.o")
        cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-I", INCLUDE, "-isystem", inc,
               "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
               "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj]
        return src, obj, subprocess.run(cmd, capture_output=True, text=True)

    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        module = ex.submit(compile_pycall)
        results = list(ex.map(compile_one, srcs))
        module = module.result()
    failed = False
    for src, _, r in results + [module]:
        if r.returncode != 0 or (verbose_ptxas and not quiet):
            sys.stderr.write(r.stdout + r.stderr)
        failed |= r.returncode != 0
    if failed:
        raise RuntimeError("a compiler failed; see the messages above")
    objs = [o for _, o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    tmp = PYCALL + ".tmp"
    # PyTorch's libraries are those that the importing process has loaded: no run path for them
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, module[1], "-L", PKG, "-l:libpkvattn.so",
           "-Wl,-rpath,$ORIGIN", "-L", torch_lib(), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("the Python module's build failed")
    os.replace(tmp, PYCALL)
    if not quiet:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
