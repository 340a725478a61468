"""Build libmoe_gb300.so in-tree with nvcc for sm_103a (one -gencode).

Each .cu file compiles to an object in parallel, then one link step makes
the shared library next to this file.  No cmake, no torch extension machinery:
the library has a plain C ABI and is loaded with ctypes.  Beside it stands
_native.so, a Python module that makes the attention sub-layer's calls on torch
tensors (host code against torch's headers and libraries); where there is no
torch, the library alone is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe_gb300.so")
BINDING = os.path.join(HERE, "_native.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["api.cu", "pack.cu", "routing.cu", "grouped_gemm.cu", "decode.cu", "small_batch.cu", "block.cu",
           "attention.cu", "linear_few.cu", "linear_many.cu", "paged.cu", "prefix.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return path


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read().strip()


def _torch_root():
    """torch's folder, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_flags(torch: str):
    """Flags of the compile and of the link of the Python module (nvcc's, which
    brings a host compiler with it)."""
    # (torch's and CUDA's headers as system headers: their warnings are theirs)
    compile_ = ["-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-I" + os.path.join(ROOT, "include"),
                "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
                "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include")]
    link = ["-cudart", "none", "-L" + HERE, "-Xlinker", "-l:" + os.path.basename(LIB), "-Xlinker", "-rpath=$ORIGIN",
            "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_, link


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    # objects built on another machine type are never reused
    stamp = os.path.join(BUILD_DIR, "host.txt")
    host = platform.machine()
    if _read(stamp) != host:
        force = True
        with open(stamp, "w") as f:
            f.write(host + "\n")
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers.append(os.path.join(ROOT, "include", "moe.h"))
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *headers, __file__]):
            jobs.append([nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o])

    torch = _torch_root()
    binding = None
    if torch:
        # object and module are of one torch and one Python version; the object has them
        # in its name, the module in the note beside the objects
        src = os.path.join(CSRC, "binding.cpp")
        versions = importlib.metadata.version("torch") + (sysconfig.get_config_var("EXT_SUFFIX") or "")
        binding_obj = os.path.join(BUILD_DIR, "binding-" + versions + ".o")
        made_for = os.path.join(BUILD_DIR, "binding.txt")
        compile_, link = _binding_flags(torch)
        if force or _stale(binding_obj, [src, headers[-1], __file__]):
            binding = [nvcc(), *compile_, "-c", src, "-o", binding_obj]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        # (the library does not wait for the module, nor depend on it)
        module = ex.submit(run, binding) if binding else None
        for err in ex.map(run, jobs):
            if verbose and err:
                print(err, file=sys.stderr)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    if module:
        module.result()
    if torch and (force or _stale(BINDING, [binding_obj, LIB]) or _read(made_for) != versions):
        tmp = BINDING + f".tmp{os.getpid()}"
        run([nvcc(), *ARCH, "-shared", "-o", tmp, binding_obj, *link])
        os.replace(tmp, BINDING)
        with open(made_for, "w") as f:
            f.write(versions + "\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
