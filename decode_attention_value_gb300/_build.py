"""Build libkvz.so in-tree with nvcc for sm_103a (no torch extension machinery), and the
Python module _binding beside it (csrc/python, against torch's headers and libkvz.so).

Each translation unit is compiled in parallel, then linked into one shared library
next to this file.  Rebuilds only when a source is newer than the libraries, or when the
binding was compiled against another torch or Python than the ones in use.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import importlib.util
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvz.so")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
STAMP = os.path.join(PKG, "_binding.against")  # the torch and Python that it was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libkvz needs the CUDA 13 toolkit to build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _against() -> str:
    """What the binding depends on beside its sources: the torch and the Python in use."""
    spec = importlib.util.find_spec("torch")
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return f"{sys.version}\n{spec.origin}\n{f.read()}"


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    try:
        with open(STAMP) as f:
            if f.read() != _against():
                return False
    except OSError:
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _binding_object() -> str:
    """Compile the Python module (without its link, which wants libkvz.so)."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(BUILD, "binding.cpp.o")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", BINDING_SRC, "-o", obj,
           f"-I{os.path.join(ROOT, 'include')}", f"-I{sysconfig.get_paths()['include']}",
           "-isystem", os.path.join(torch_dir, "include"), "-isystem", os.path.join(cuda, "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str):
    torch_lib = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libkvz.so", "-Wl,-rpath,$ORIGIN",
           f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(STAMP, "w") as f:
        f.write(_against())


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc, *FLAGS, *extra, "-x", "c++", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        binding = ex.submit(_binding_object)
        objs = list(ex.map(compile_one, sources()))
        binding = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True, extra=["-Xptxas", "-v"] if "-v" in sys.argv else None))
