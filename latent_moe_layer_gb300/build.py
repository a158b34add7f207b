"""Compile libk3moe.so (every .cu under csrc/) for sm_103a with nvcc, and the Python binding of the expert
training operators (csrc/experts_py.cpp, against the installed PyTorch) with the host compiler; in-tree.

The C ABI needs the library alone: `build(binding=False)` (`build.py --library`), and where PyTorch is not
installed the binding is left out."""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libk3moe.so")
BINDING = os.path.join(PKG, "_experts.so")
BINDING_SRC = os.path.join(CSRC, "experts_py.cpp")
BINDING_KEY = os.path.join(BUILD, "experts_binding.txt")        # what BINDING was built against
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
         "-I", CSRC, "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "k3moe.h")])


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps())


def _torch_release(base: str) -> str:
    with open(os.path.join(base, "version.py")) as f:
        return "".join(line for line in f if "version" in line and "=" in line)


def binding_key() -> str:
    """What a built binding depends on besides its sources: Python's and PyTorch's versions (their C++ ABIs); empty
    where PyTorch is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return ""
    base = os.path.dirname(spec.origin)
    return f"{sysconfig.get_config_var('SOABI') or sys.version}\n{base}\n{_torch_release(base)}"


def binding_matches() -> bool:
    """Whether the built binding was built against the Python and PyTorch that run now."""
    try:
        with open(BINDING_KEY) as f:
            return f.read() == binding_key()
    except OSError:
        return False


def _build_binding() -> None:
    import torch
    base = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), os.path.join(ROOT, "include")]
    lib = os.path.join(base, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           *[a for i in inc for a in ("-isystem", i)], f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-o", tmp,
           BINDING_SRC, f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed on {BINDING_SRC} (the C ABI needs only build(binding=False)):\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_KEY, "w") as f:
        f.write(binding_key())


def _binding_stale() -> bool:
    return not os.path.exists(BINDING) or not binding_matches() or any(
        os.path.getmtime(f) > os.path.getmtime(BINDING) for f in (BINDING_SRC, os.path.join(ROOT, "include", "k3moe.h")))


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    if binding and not binding_key():
        sys.stderr.write("PyTorch is not installed: the binding of the expert training operators is left out\n")
        binding = False
    with ThreadPoolExecutor(1) as ex:                       # beside the CUDA sources
        job = ex.submit(_build_binding) if binding and (force or _binding_stale()) else None
        lib = _build_library(force, verbose)
        if job:
            job.result()
    return lib


def _build_library(force: bool, verbose: bool) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, binding="--library" not in sys.argv))
