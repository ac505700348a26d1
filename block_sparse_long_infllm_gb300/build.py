"""Build libinfllmv2.so in-tree with nvcc for sm_103a (GB300), and the Python module _binding.

Each translation unit compiles in parallel to `_build/`, then nvcc links the
shared library next to this file.  The CUDA runtime is linked as a shared
library so the process shares one runtime (and one set of stream handles)
with PyTorch.  That needs nvcc alone.  Where PyTorch is installed, `_binding.so`
(csrc/binding.cpp, the host compiler) is then linked to that library and to PyTorch's.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build", "infllmv2")
LIB_PATH = os.path.join(HERE, "libinfllmv2.so")
BINDING_PATH = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "kernel_pool.cu", "select.cu", "decode.cu", "prefill.cu", "decode_noalloc.cu", "tmap.cu", "prefill_tc.cu", "score_tc.cu", "decode_cluster.cu", "bwd.cu", "bwd_tc.cu", "tree_attn.cu", "rope.cu", "verify.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "infllmv2.h"))
    files.append(os.path.abspath(__file__))
    return files


def _with_binding() -> bool:
    return importlib.util.find_spec("torch") is not None


def _stale() -> bool:
    outputs = [LIB_PATH] + ([BINDING_PATH] if _with_binding() else [])
    if not all(os.path.exists(f) for f in outputs):
        return True
    t = min(os.path.getmtime(f) for f in outputs)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _compile_binding() -> str:
    """csrc/binding.cpp to an object file, against PyTorch's and Python's headers."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{p}" for p in include] + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the host compiler failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB_PATH, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", f"-Wl,-rpath,$ORIGIN:{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking _binding.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if any source is newer than the library) and return the library path."""
    if not force and not ptxas_info and not _stale():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if _with_binding() else None
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", "-soname=" + os.path.basename(LIB_PATH), "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if binding is not None:  # a fault of the binding's leaves the library in place
        _link_binding(binding.result())
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
