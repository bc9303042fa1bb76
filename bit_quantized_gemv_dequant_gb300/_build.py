"""Build libqgemv.so in-tree: every .cu under csrc/ compiled for sm_103a in
parallel with nvcc, then linked into one shared library (CUDA runtime linked
statically, so the library needs only the driver at run time). Beside it the
Python module _serving.so (csrc/serving.cpp) against this interpreter's and
torch's headers, which calls that library."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "qgemv")
LIB = os.path.join(PKG, "libqgemv.so")
MODULE = os.path.join(PKG, "_serving.so")
MODULE_SRC = os.path.join(CSRC, "serving.cpp")
HEADER = os.path.join(INCLUDE, "qgemv.h")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
         "-fvisibility=hidden", "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "qgemv.h")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, extra):
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    if _stale(obj, [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "qgemv.h")]):
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr
    return obj, ""


def _compile_module():
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(OBJDIR, "serving.cpp.o")
    if _stale(obj, [MODULE_SRC, HEADER, os.path.join(base, "version.py")]):
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-I{INCLUDE}",
               f"-I{sysconfig.get_paths()['include']}", f"-I{base}/include", "-I/usr/local/cuda/include", "-c",
               MODULE_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {MODULE_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj, os.path.join(base, "lib")


def _link_module(obj, torch_lib):
    tmp = MODULE + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libqgemv.so", f"-L{torch_lib}", "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MODULE)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    if not force and not _stale(LIB, _deps()) and not _stale(MODULE, [MODULE_SRC, HEADER, LIB]):
        return LIB
    if force:
        for o in glob.glob(os.path.join(OBJDIR, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        module = ex.submit(_compile_module)
        results = list(ex.map(lambda s: _compile(s, list(extra)), _sources()))
        module = module.result()
    if verbose:
        for _, log in results:
            if log:
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_module(*module)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
