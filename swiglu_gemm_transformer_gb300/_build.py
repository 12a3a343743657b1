"""Build the sm_103a CUDA library in-tree with nvcc, and the PyTorch module with g++ (no cmake).

Each translation unit under ``csrc/`` compiles in parallel to an object file
under ``_build/``; the objects link into ``libswiglu_gb300.so`` beside this
file (CUDA runtime linked statically, the driver reached through
cudaGetDriverEntryPoint, so the library needs no libcuda at link time).  The
PyTorch module ``_swiglu_torch.so`` links to it and to the running torch; where
there is no PyTorch with CUDA, only the C library is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libswiglu_gb300.so")
TORCH_SRC = os.path.join(CSRC, "torch_binding.cpp")
TORCH_LIB = os.path.join(PKG, "_swiglu_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "swiglu.h"))
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_command(target: str):
    """g++ command of the PyTorch module (the torch that runs this process)."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           INCLUDE]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
            *(f"-I{p}" for p in inc), TORCH_SRC, "-o", target, "-L", os.path.join(home, "lib"), "-L", PKG,
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-l:" + os.path.basename(LIB),
            "-Wl,-rpath,$ORIGIN"]


def _torch_stamp() -> str:
    import torch
    return torch.__version__


def build_torch(force: bool = False):
    """Build the PyTorch module; it links to the CUDA library, so that comes first.

    Returns its path, or None where there is no PyTorch with CUDA."""
    try:
        import torch
    except ModuleNotFoundError:
        torch = None
    if torch is None or torch.version.cuda is None:
        print(f"no PyTorch with CUDA: {os.path.basename(TORCH_LIB)} is not built", file=sys.stderr)
        return None
    stamp = os.path.join(BUILD, "torch_version")
    same = os.path.exists(stamp) and open(stamp).read() == _torch_stamp()
    if not force and same and not _stale(TORCH_LIB, [TORCH_SRC, os.path.join(INCLUDE, "swiglu.h")]):
        return TORCH_LIB
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    r = subprocess.run(_torch_command(tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(TORCH_SRC)}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(stamp, "w") as f:
        f.write(_torch_stamp())
    return TORCH_LIB


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    hdrs = _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        if not force and not _stale(obj, [src] + hdrs):
            return obj, ""
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", CSRC, "-I", INCLUDE, "-c", src, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, obj)
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose:
        for obj, log in logs:
            if log:
                print(f"--- {os.path.basename(obj)}\n{log}")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    build_torch(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
