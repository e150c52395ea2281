"""Build the sm_100a selective-scan library in-tree: selective_state_space_34_b200/libssm_scan.so, and beside it the
native marshalling module _marshal.so (csrc/ssm_marshal.cpp, against the installed torch's headers).

nvcc compiles every csrc/*.cu for sm_100a (-gencode arch=compute_100a,code=sm_100a) and links a
shared library with the CUDA runtime linked statically, so the .so has no dependency beyond the
driver. Run as ``python -m selective_state_space_34_b200.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libssm_scan.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
BUILD = os.path.join(ROOT, "_build")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for c in [os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"]:
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "ssm_scan.h")]


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _marshal_deps():
    return [os.path.join(CSRC, "ssm_marshal.cpp"), os.path.join(ROOT, "include", "ssm_scan.h")]


def built_for() -> str:
    """The torch and the Python that _marshal.so is compiled against; the module carries it as BUILT_FOR."""
    import torch

    return "torch %s, %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def _marshal_matches() -> bool:
    with open(MARSHAL, "rb") as f:
        return built_for().encode() + b"\0" in f.read()


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile _marshal.so: plain C++ (no device code), linked to the library beside it and to torch."""
    if not force and _newer(MARSHAL, _marshal_deps()) and _marshal_matches():
        return MARSHAL
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    inc = os.path.join(torch_dir, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), '-DSSM_BUILT_FOR="%s"' % built_for(),
           "-I" + sysconfig.get_paths()["include"], "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), os.path.join(CSRC, "ssm_marshal.cpp"), "-o", tmp,
           "-L" + PKG, "-l:libssm_scan.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch_dir, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("marshalling module failed to build:\n" + r.stderr[-4000:])
    os.replace(tmp, MARSHAL)
    if verbose:
        print("built", MARSHAL)
    return MARSHAL


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        build_marshal(verbose=verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        with open(obj + ".log", "w") as f:
            f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s" % (src, r.stderr[-4000:]))
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr[-4000:])
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
