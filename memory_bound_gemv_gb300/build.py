"""Builds the CUDA library ``_build/libmbgemv.so`` in-tree with nvcc.

Every translation unit under ``csrc/`` is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``) in parallel, then linked into
one shared library with the CUDA runtime linked statically.  ``ptxas -v``
output (registers, spills, shared memory per kernel) is kept in
``_build/ptxas.log``.  Rebuilds only when a source or header is newer than
the library.  Beside it the host compiler makes ``_build/_mbgbinding.so`` from
``csrc/binding.cpp``, for the installed torch: the quick form of the
decode-step calls' argument checks.  The library needs neither torch nor the
host compiler for it: where the quick form cannot be built, a warning says so and
the checks run in Python.
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmbgemv.so")
BINDING = os.path.join(BUILD, "_mbgbinding.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "-Xptxas", "-v", "--expt-relaxed-constexpr",
                     "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _newer(made, deps) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(p) <= os.path.getmtime(made) for p in deps)


def up_to_date() -> bool:
    """Whether the library needs no build (``binding_up_to_date`` for the quick form of the checks)."""
    return _newer(LIB, _deps())


def _torch_version():
    """Version of the installed torch, which is not imported for it; None where there is none."""
    import importlib.util

    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    try:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        return None
    return found.group(1) if found else None


def binding_up_to_date() -> bool:
    """Whether the quick form is there, made for the installed torch, or none can be."""
    version = _torch_version()
    if version is None:
        return True
    try:
        with open(BINDING + ".torch") as f:
            made_for = f.read()
    except OSError:
        return False
    deps = [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "gemv.h"), os.path.abspath(__file__)]
    return made_for == version and _newer(BINDING, deps)


def _build_binding():
    """csrc/binding.cpp against the installed torch's headers, with the host compiler."""
    import sysconfig

    import torch

    top = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    includes = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           f'-DMBG_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in includes], os.path.join(CSRC, "binding.cpp"), "-L" + os.path.join(top, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("compiling binding.cpp failed")
        os.replace(tmp, BINDING)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
    with open(BINDING + ".torch", "w") as f:
        f.write(torch.__version__)


def _try_binding():
    """Builds the quick form; what stands in its way is told, and stands in the library's way no more."""
    try:
        _build_binding()
    except Exception as e:  # noqa: BLE001 - a broken torch, no compiler, no headers ...
        sys.stderr.write(f"memory_bound_gemv_gb300: without the compiled argument checks ({e}); they run in Python\n")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is needed; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_try_binding) if force or not binding_up_to_date() else None
        if force or not up_to_date():
            _build_library(verbose)
        if binding:
            binding.result()
    return LIB


def _build_library(verbose):
    nvcc = _nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    workers = min(len(srcs), os.cpu_count() or 4)
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as ex:
        results = list(ex.map(compile_one, srcs))
    log = []
    for src, obj, r in results:
        log.append(f"== {os.path.basename(src)}\n{r.stdout}{r.stderr}")
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for _, o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("linking libmbgemv.so failed")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
