"""Build the CUDA library ``libna.so`` in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked into
one shared library with a C ABI (``include/na.h``).  ``csrc/paged_calls.cpp``,
compiled meanwhile with the host compiler against torch's headers, becomes the
extension module ``_paged_calls``.  Both outputs sit beside this file so the
Python binding finds them without installation.  ``libna.so`` needs neither
torch nor Python and is linked whatever becomes of the extension module, which
is left out, with a warning, where torch or a header that it needs is missing.
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libna.so")
# named for the Python whose ABI it has: another one does not take it for its own
CALLS = os.path.join(PKG, "_paged_calls" + sysconfig.get_config_var("EXT_SUFFIX"))
# the torch that it was compiled against, whose classes it reads through inline code
BUILT_FOR = os.path.join(BUILD, "paged_calls.torch")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_identity(torch) -> str:
    """Version and commit of the torch in directory `torch`, without importing it."""
    v = runpy.run_path(os.path.join(torch, "version.py"))
    return f"{v['__version__']} {v['git_version']}"


def _built_for() -> str:
    if not os.path.exists(BUILT_FOR):
        return ""
    with open(BUILT_FOR) as f:
        return f.read()


def _calls_missing(torch, include) -> str:
    """What the extension module needs and this machine has not, or ''."""
    if torch is None:
        return "torch"
    for path in (os.path.join(include, "Python.h"),
                 os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h"),
                 os.path.join(torch, "lib", "libc10_cuda.so")):
        if not os.path.exists(path):
            return path
    return ""


def build_calls(cuda: str) -> str | None:
    """Compile (if stale) and return the path of the extension module _paged_calls; None, with a
    warning, where something that it needs is missing."""
    src = os.path.join(CSRC, "paged_calls.cpp")
    spec = importlib.util.find_spec("torch")
    torch = list(spec.submodule_search_locations)[0] if spec else None
    include = sysconfig.get_paths()["include"]
    missing = _calls_missing(torch, include)
    if missing:
        warnings.warn(f"the paged calls (csrc/paged_calls.cpp) are not built: {missing} is missing")
        return None
    identity = _torch_identity(torch)
    # (file times do not tell one torch from another: an older one may be installed later)
    if _stale(CALLS, [src, __file__, os.path.join(INCLUDE, "na.h")]) or _built_for() != identity:
        tmp = CALLS + f".tmp{os.getpid()}"
        cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", src, "-o",
               tmp, f'-DNA_TORCH="{identity}"', "-I", INCLUDE, "-I", os.path.join(torch, "include"), "-I",
               os.path.join(cuda, "include"), "-I", include, "-L", os.path.join(torch, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"compiling {src} failed:\n{res.stderr}")
        os.replace(tmp, CALLS)
        with open(BUILT_FOR, "w") as f:
            f.write(identity)
    return CALLS


def build(verbose: bool = False, extra_flags=None) -> str:
    """Compile (if stale) and return the path of libna.so."""
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "na.h")]
    flags = NVCC_FLAGS + list(extra_flags or [])
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        if _stale(obj, [src, __file__] + headers):
            cmd = [cc] + ARCH + flags + ["-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd))
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
            if verbose and res.stderr:
                print(res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(sources) + 1) as ex:
        calls = ex.submit(build_calls, os.path.dirname(os.path.dirname(os.path.realpath(cc))))
        objs = list(ex.map(compile_one, sources))
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stderr}")
        os.replace(tmp, LIB)
    calls.result()  # an error of its compiler is raised with the library in place
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
