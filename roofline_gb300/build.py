"""Builds libgb300gemm.so in-tree with nvcc for sm_103a, and the torch binding
of its feed-forward operators.

Each .cu file in csrc/ is compiled to an object in parallel, then linked
into one shared library (static CUDA runtime, no torch dependency).
torch_binding.cpp becomes the Python module _ff_native.so beside it, built
with g++ against the installed torch's headers; without torch only the library
is built.  Run
``python -m roofline_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libgb300gemm.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING = os.path.join(BUILD, "_ff_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgb300gemm.so")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(out: str, deps) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(f) > os.path.getmtime(out)
                                          for f in deps)


def _torch_dir():
    """The installed torch's folder; None without torch, which only the binding needs."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _compile(src: str, log_dir: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, os.path.basename(src) + ".ptxas.txt"), "w") as f:
        f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
    return obj


def _compile_binding(log_dir: str) -> str:
    """torch_binding.cpp to an object (its link needs the library)."""
    torch_dir = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD, "torch_binding.o")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-Wall", "-I", INCLUDE, "-isystem", os.path.join(torch_dir, "include"), "-isystem",
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(os.path.join(log_dir, "torch_binding.cpp.txt"), "w") as f:
        f.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    torch_dir = _torch_dir()
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, "-L",
           os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-L", BUILD, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, BINDING)


def _link(objs) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC"] + objs + ["-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is older than its sources: libgb300gemm.so, then,
    where torch is installed, its binding.  The library is there whatever
    becomes of the binding, whose failure is raised last."""
    srcs = _sources()
    lib = force or _stale(LIB, srcs + _headers())
    torch = _torch_dir() is not None and \
        (lib or _stale(BINDING, [BINDING_SRC, LIB] + _headers()))
    if not lib and not torch:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(12, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding, BUILD) if torch else None
        if lib:
            _link(list(ex.map(lambda s: _compile(s, BUILD), srcs)))
        if binding:
            _link_binding(binding.result())
    if verbose and lib:
        for s in srcs:
            with open(os.path.join(BUILD, os.path.basename(s) + ".ptxas.txt")) as f:
                sys.stdout.write(f.read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
