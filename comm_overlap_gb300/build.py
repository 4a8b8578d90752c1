"""Builds libdomino.so (the C-ABI library in include/domino.h) in-tree with nvcc.

Every translation unit is compiled for sm_103a only, in parallel, then linked with the
static CUDA runtime so the library loads without a separate libcudart on the path.  Beside it g++ builds
torch_calls (csrc/torch_calls.cpp) against the installed PyTorch.
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

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdomino.so")
CALLS = os.path.join(HERE, "torch_calls" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS_FOR = os.path.join(OBJ, "torch_calls.for")  # the PyTorch that it was built for
HEADER = os.path.join(ROOT, "include", "domino.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [HEADER,
                                                                                                        __file__]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # one that runs from its sources
        import torch
        return torch.__version__


def _calls_need_build() -> bool:
    """Also for another PyTorch, whose tensors may be laid out in another way."""
    t = os.path.getmtime(CALLS) if os.path.exists(CALLS) else 0
    if any(os.path.getmtime(p) > t for p in (CALLS_SRC, HEADER, __file__)) or not os.path.exists(CALLS_FOR):
        return True
    with open(CALLS_FOR, encoding="utf-8") as f:
        return f.read() != _torch_version()


def _build_calls() -> None:
    """torch_calls only shortens calls: where this PyTorch or its headers do not go with it, the rest is built without."""
    import torch
    base = os.path.dirname(torch.__file__)
    dirs = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
            os.path.join(ROOT, "include")]
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in dirs), CALLS_SRC, "-o", tmp,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(f"torch_calls is not built, calls of the cache's operators will take longer:\n{r.stderr[-2000:]}\n")
        return
    os.replace(tmp, CALLS)
    os.makedirs(OBJ, exist_ok=True)
    with open(CALLS_FOR, "w", encoding="utf-8") as f:
        f.write(_torch_version())


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(_build_calls) if force or _calls_need_build() else None
        if force or needs_build():
            _build_lib(verbose)
        if calls:
            calls.result()
    return LIB


def _build_lib(verbose: bool) -> None:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
