"""Builds the in-tree CUDA library ``paged_kv_gb300/libpkv.so`` for sm_103a, and
``paged_kv_gb300/_binding.so``, the Python binding of the serving operators.

Each ``.cu`` file under ``csrc/`` is compiled to an object in parallel with
``nvcc -gencode arch=compute_103a,code=sm_103a``, then the objects are linked
into one shared library against the shared CUDA runtime.  The binding
(``csrc/binding.cpp``, plain C++ against the installed torch's headers) is
compiled beside them and linked against that library.  Objects go to
``paged_kv_gb300/_build/`` (git-ignored); both are rebuilt only when a source or
header is newer than them, or when the binding was made for another torch or Python.
"""

from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding_for.txt")  # the torch that it was made for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _nvcc() -> str:
    return os.path.join(_cuda_home(), "bin", "nvcc")


def _torch_dir() -> str:
    """The installed torch's folder, found without importing it."""
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def _binding_for() -> str:
    """What the binding's C++ interface depends on."""
    return "\n".join((_torch_dir(), importlib.metadata.version("torch"), sys.version))


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    files = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    files += glob.glob(os.path.join(CSRC, "*.cpp"))
    files += glob.glob(os.path.join(ROOT, "include", "*.h"))
    files.append(os.path.abspath(__file__))
    return files


def stale() -> bool:
    if not all(os.path.exists(f) for f in (LIB, BINDING, BINDING_FOR)):
        return True
    with open(BINDING_FOR) as f:
        if f.read() != _binding_for():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link libpkv.so and the binding if they are missing or stale; returns
    the library's path."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr, flush=True)
        return obj

    def compile_binding():
        torch_dir = _torch_dir()
        obj = os.path.join(BUILD, "binding.o")
        dirs = [os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(_cuda_home(), "include")]
        _run(["g++", "-O2", "-std=c++17", "-fPIC", *("-I" + d for d in dirs), "-c",
              os.path.join(CSRC, "binding.cpp"), "-o", obj], "binding.cpp", verbose)
        return obj, os.path.join(torch_dir, "lib")

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(2, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, srcs))
        binding_obj, torch_lib = binding.result()
    libdir = os.path.join(_cuda_home(), "lib64")
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", f"-rpath={libdir}", "-Xlinker", "-soname=libpkv.so"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    tmp = BINDING + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, binding_obj, LIB, "-L" + torch_lib, "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_python", "-L" + libdir, "-lcudart", "-Wl,-rpath,$ORIGIN",
          "-Wl,-rpath," + torch_lib, "-Wl,-rpath," + libdir], "the binding's link", verbose)
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_for())
    return LIB


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a.startswith("-")]
    print(build(force=True, verbose=True, extra_flags=extra))
