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
import importlib.metadata
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
PYCALL_FOR = os.path.join(BUILD, "pycall_torch_version")  # the PyTorch that it was built for
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


def _older_than(path: str, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _headers():
    return [p for d in (CSRC, INCLUDE) for ext in ("*.cuh", "*.h") for p in glob.glob(os.path.join(d, ext))]


def _library_is_stale(srcs) -> bool:
    return _older_than(LIB, srcs + _headers())


def _torch_version() -> str:
    """PyTorch's version without importing it, "" where there is none."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return ""


def _module_is_older_than_its_sources() -> bool:
    return _older_than(PYCALL, glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _module_is_stale() -> bool:
    """Also where it was built for another PyTorch: a tensor's layout is the version's."""
    if _module_is_older_than_its_sources():
        return True
    try:
        with open(PYCALL_FOR) as f:
            return f.read() != _torch_version()
    except OSError:
        return True


def _run(cmd) -> str | None:
    """None, or what the command said when it failed."""
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return f"{cmd[0]}: {e}"
    return r.stdout + r.stderr + f"{cmd[0]} returned {r.returncode}" if r.returncode else None


def _compile_module(obj: str) -> str | None:
    try:
        inc = os.path.join(os.path.dirname(torch_lib()), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    except (ImportError, RuntimeError) as e:
        return str(e)
    return _run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-I", INCLUDE, "-isystem", inc,
                 "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
                 "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "pycall.cpp"), "-o", obj])


def _link_module(obj: str) -> str | None:
    tmp = PYCALL + ".tmp"
    # PyTorch's libraries are those that the importing process has loaded: no run path for them
    said = _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libpkvattn.so",
                 "-Wl,-rpath,$ORIGIN", "-L", torch_lib(), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"])
    if said is None:
        os.replace(tmp, PYCALL)
        with open(PYCALL_FOR, "w") as f:
            f.write(_torch_version())
    return said


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = False) -> str:
    """Builds what is out of date. A library that cannot be built raises; a module that cannot says so on
    stderr and leaves the calls that need it to raise: the others need the library alone."""
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    library, module = force or _library_is_stale(srcs), force or _module_is_stale()
    if not library and not module:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    flags = _flags(verbose_ptxas)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    module_obj = os.path.join(BUILD, "pycall.cpp.o")
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        said = ex.submit(_compile_module, module_obj) if module else None
        results = list(ex.map(compile_one, srcs)) if library else []
        said = said.result() if module else None
    failed = False
    for src, _, r in results:
        if r.returncode != 0 or (verbose_ptxas and not quiet):
            sys.stderr.write(r.stdout + r.stderr)
        failed |= r.returncode != 0
    if failed:
        raise RuntimeError("nvcc failed; see the messages above")
    if library:
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for _, o, _ in results] + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    if module:
        said = said if said is not None else _link_module(module_obj)
        if said is not None:
            # one that only may be for another PyTorch stays: the binding looks at what it was built for
            if os.path.exists(PYCALL) and _module_is_older_than_its_sources():
                os.remove(PYCALL)
            sys.stderr.write(f"{said}\n_pycall.so was not built: without it the calls that go through it raise\n")
    if not quiet:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
