"""In-tree build of libdspark.so (the CUDA kernels behind the C ABI) for sm_103a, and of the
Python module of calls.cpp beside it.

Each .cu file is compiled to an object in parallel, then linked into one shared library
with the CUDA runtime linked statically (the driver is reached through the runtime's
entry-point query, so the library has no link-time dependency on libcuda).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libdspark.so")
# (named after the interpreter whose C API it is compiled against: another's is another file)
CALLS = os.path.join(BUILD, "_dspark_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdspark")
    return exe


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "dspark.h")]


def _stale(target, deps) -> bool:
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in deps)


def build_calls(force: bool = False) -> bool:
    """Compile the Python module of calls.cpp.  Where that cannot be done (no headers of this interpreter)
    it is left out with a warning, and the calls are checked in Python: target.py has every check."""
    source = os.path.join(CSRC, "calls.cpp")
    if not force and not _stale(CALLS, [source, os.path.join(ROOT, "include", "dspark.h")]):
        return True
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I",
           sysconfig.get_paths()["include"], source, "-o", tmp]
    try:
        os.makedirs(BUILD, exist_ok=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode == 0:
            os.replace(tmp, CALLS)
            return True
        why = f"{res.stdout}\n{res.stderr}"
    except OSError as e:
        why = str(e)
    if os.path.exists(CALLS):
        os.remove(CALLS)                     # (an older one may call the library otherwise)
    warnings.warn(f"the module of calls.cpp was not built, calls are checked in Python: {why}", RuntimeWarning)
    return False


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile every kernel source for sm_103a and link libdspark.so (returns its path), and the
    Python module."""
    if not force and not _stale(LIB, _deps()):
        build_calls()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc()] + ARCH + flags + ["-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        calls = ex.submit(build_calls, force)
        objs = list(ex.map(compile_one, _sources()))
        calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link of libdspark.so failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
