"""Build libsnack.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel, then linked into
coo_spmm_sparse_gb300/_build/libsnack.so against the shared CUDA runtime.
csrc/binding.cpp, the Python binding of the dense operators, is compiled by
the host compiler into _build/_dense.so, against libsnack.so and the
installed torch; without torch the library alone is built.  Each is rebuilt
only when a source or header is newer than it, the library also on another
machine, the binding for another machine, Python or torch.
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
DENSE_STAMP = os.path.join(BUILD, "dense.txt")


def _torch_dir() -> str | None:
    """Where torch is installed (without importing it)."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _dense_built_for(torch_dir: str) -> str:
    """What the binding depends on besides its sources."""
    try:
        with open(os.path.join(torch_dir, "version.py")) as f:
            torch_version = next((l.strip() for l in f if l.startswith("__version__")), "")
    except OSError:
        torch_version = ""
    return f"{platform.machine()} python {sys.version_info[0]}.{sys.version_info[1]} torch {torch_version}"


def _stale(path: str, stamp: str, built_for: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    try:
        with open(stamp) as f:
            if f.read().strip() != built_for:
                return True
    except OSError:
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__]


def _compile_binding(nvcc: str, torch_dir: str) -> str:
    """binding.cpp -> object file (the host compiler; no CUDA code in it)."""
    inc = os.path.join(torch_dir, "include")
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


def _link_binding(obj: str, torch_dir: str) -> None:
    libs = os.path.join(torch_dir, "lib")
    tmp = DENSE + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", obj, "-o", tmp, f"-L{BUILD}", "-lsnack",
           "-Wl,-rpath,$ORIGIN", f"-L{libs}", f"-Wl,-rpath,{libs}", "-lc10", "-lc10_cuda", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {DENSE} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, DENSE)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is stale of libsnack.so (its path is returned) and,
    where torch is installed, the binding."""
    torch_dir = _torch_dir()
    lib = force or _stale(LIB, STAMP, platform.machine(), sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
                          + _headers())
    dense = torch_dir is not None and (
        force or _stale(DENSE, DENSE_STAMP, _dense_built_for(torch_dir), [BINDING] + _headers()))
    if torch_dir is None:
        sys.stderr.write("torch not found: the Python binding of the dense operators is not built\n")
    if not lib and not dense:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *CFLAGS, *ARCH, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = sources() if lib else []
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_compile_binding, nvcc, torch_dir) if dense else None
        objs = list(ex.map(compile_one, srcs))
        binding = binding.result() if dense else None
    if lib:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, "-shared", *ARCH, "-cudart", "shared", "-Xlinker",
               f"-rpath,{_cuda_lib_dir(nvcc)}", *objs, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
        with open(STAMP, "w") as f:
            f.write(platform.machine())
    if dense:
        _link_binding(binding, torch_dir)
        with open(DENSE_STAMP, "w") as f:
            f.write(_dense_built_for(torch_dir))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
