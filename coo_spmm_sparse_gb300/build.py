"""Build libsnack.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel, then linked into
coo_spmm_sparse_gb300/_build/libsnack.so against the shared CUDA runtime.
csrc/binding.cpp, the Python binding of the dense operators, is compiled by
the host compiler into _build/_dense.so, against libsnack.so and the
installed torch.  Rebuilds only when a source or header is newer than the
libraries, or they were built for another machine, Python or torch.
"""

from __future__ import annotations

import glob
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libsnack.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{os.path.join(ROOT, 'include')}"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the SNACK library needs the CUDA toolkit to build")
    return cand


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


STAMP = os.path.join(BUILD, "machine.txt")
BINDING = os.path.join(CSRC, "binding.cpp")
DENSE = os.path.join(BUILD, "_dense.so")


def _torch_dir() -> str:
    """Where torch is installed (without importing it)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found: the binding of the dense operators needs it")
    return os.path.dirname(spec.origin)


def _built_for() -> str:
    """What the built files depend on besides their sources."""
    try:
        with open(os.path.join(_torch_dir(), "version.py")) as f:
            torch_version = next((l.strip() for l in f if l.startswith("__version__")), "")
    except OSError:
        torch_version = ""
    return f"{platform.machine()} python {sys.version_info[0]}.{sys.version_info[1]} torch {torch_version}"


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(DENSE):
        return True
    try:
        with open(STAMP) as f:
            if f.read().strip() != _built_for():
                return True
    except OSError:
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(DENSE))
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [BINDING, __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _compile_binding(nvcc: str) -> str:
    """binding.cpp -> object file (the host compiler; no CUDA code in it)."""
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(BUILD, "binding.o")
    cmd = [shutil.which("g++") or "c++", "-std=c++17", "-O2", "-fPIC", "-Wall",
           f"-I{os.path.join(ROOT, 'include')}", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           os.path.join(os.path.dirname(_cuda_lib_dir(nvcc)), "include"), "-isystem",
           sysconfig.get_paths()["include"], "-c", BINDING, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {BINDING} failed:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = DENSE + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", obj, "-o", tmp, f"-L{BUILD}", "-lsnack",
           "-Wl,-rpath,$ORIGIN", f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {DENSE} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, DENSE)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libsnack.so; return its path."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *CFLAGS, *ARCH, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, nvcc)
        objs = list(ex.map(compile_one, srcs))
        binding = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", *ARCH, "-cudart", "shared", "-Xlinker",
           f"-rpath,{_cuda_lib_dir(nvcc)}", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    with open(STAMP, "w") as f:
        f.write(_built_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
