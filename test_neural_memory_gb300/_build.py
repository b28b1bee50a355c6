"""Builds libttm.so in-tree with nvcc for sm_103a (no torch involvement), and beside it
ttm_torch.so, the compiled part of the Python binding.

Each translation unit under ``csrc/`` is compiled in parallel, then linked
into ``_lib/libttm.so`` with the CUDA runtime linked statically, so the
library loads on machines without a GPU driver.  ``csrc/bind_train.cpp`` is
compiled by the host compiler against torch's headers and linked with libttm.so; a
binding that does not build is reported once libttm.so is in place.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "libttm.so")
BIND = os.path.join(LIBDIR, "ttm_torch.so")
BIND_SRC = os.path.join(CSRC, "bind_train.cpp")
BIND_FOR = BIND + ".for"                  # the torch and Python that BIND was compiled against
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libttm.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _bind_for() -> str:
    """The torch (its version and place) and the Python ABI that the binding is compiled against."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "no torch"
    return f"torch {importlib.metadata.version('torch')} {spec.origin} {sysconfig.get_config_var('SOABI')}"


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND) or not os.path.exists(BIND_FOR):
        return True
    with open(BIND_FOR) as f:
        if f.read() != _bind_for():
            return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    deps = sources() + [BIND_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps.append(os.path.join(ROOT, "include", "ttm.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def _bind_flags(nvcc: str) -> tuple[list[str], list[str]]:
    """Compiler and linker flags of the torch binding (torch is found, not imported)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: libttm.so is built, its torch binding is not")
    torch = spec.submodule_search_locations[0]
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    lib = os.path.join(torch, "lib")
    cflags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *(f"-I{p}" for p in inc)]
    ldflags = [f"-L{lib}", f"-L{LIBDIR}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
               "-lc10_cuda", "-lttm", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    return cflags, ldflags


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every csrc/*.cu for sm_103a and link libttm.so, then the torch binding; returns the
    path of libttm.so."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(LIBDIR, "obj")
    os.makedirs(objdir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose or os.environ.get("TTM_PTXAS_VERBOSE") else []

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if extra:
            print(r.stdout + r.stderr)
        return obj

    bind_obj = os.path.join(objdir, "bind_train.cpp.o")

    def compile_bind() -> list[str]:
        cflags, ldflags = _bind_flags(nvcc)
        r = subprocess.run(["g++", *cflags, "-c", BIND_SRC, "-o", bind_obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
        return ldflags

    with cf.ThreadPoolExecutor(max_workers=max(2, min(16, os.cpu_count() or 1))) as ex:
        bind = ex.submit(compile_bind)
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", *objs, "-lcublas",
           "-Xlinker", "-rpath=" + os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64"),
           "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    ldflags = bind.result()                 # raises if the binding did not compile
    tmp = BIND + f".{os.getpid()}.tmp"
    r = subprocess.run(["g++", "-shared", bind_obj, *ldflags, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the torch binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(BIND_FOR, "w") as f:
        f.write(_bind_for())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
