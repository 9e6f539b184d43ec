"""Build libfd.so in-tree with nvcc for sm_103a (GB300).

Each ``csrc/*.cu`` file compiles to an object in parallel, then one link
step makes ``libfd.so`` next to this file; ``csrc/fd_torch.cpp``, the marshalling
extension of ``fd.py``, becomes ``_fd_torch.so`` with g++ at the same time.  The CUDA runtime is linked
statically, so loading the library needs no libcudart on the search path.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfd.so")
NATIVE_SRC = os.path.join(CSRC, "fd_torch.cpp")
NATIVE = os.path.join(HERE, "_fd_torch.so")
NATIVE_FOR = os.path.join(BUILD_DIR, "_fd_torch.for")   # the versions it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "fd.h"), __file__]


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def build_native(force: bool = False) -> str:
    """The marshalling extension, against the headers and libraries of the
    installed PyTorch; built again where another one, or another Python, is
    installed than the one it was built for."""
    import torch
    built_for = "torch %s, %s\n" % (torch.__version__, sysconfig.get_config_var("SOABI"))
    if not force and _newer(NATIVE, [NATIVE_SRC, os.path.join(INCLUDE, "fd.h"), __file__]) \
            and os.path.exists(NATIVE_FOR) and open(NATIVE_FOR).read() == built_for:
        return NATIVE
    home = os.path.dirname(torch.__file__)
    include = os.path.join(home, "include")
    tmp = NATIVE + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           NATIVE_SRC, "-o", tmp, "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s%s" % (cmd[0], NATIVE_SRC, r.stdout, r.stderr))
    if os.path.exists(NATIVE_FOR):
        os.remove(NATIVE_FOR)   # (a build that ends here is seen as none)
    os.replace(tmp, NATIVE)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(NATIVE_FOR, "w") as f:
        f.write(built_for)
    return NATIVE


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        build_native()
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        native = ex.submit(build_native, force)
        objs = list(ex.map(compile_one, srcs))
        native.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
