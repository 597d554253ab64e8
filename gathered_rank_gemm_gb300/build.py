"""Builds the CUDA library ``libgathered_rank_gemm.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled to an object with nvcc in parallel, then
the objects are linked into one shared library that exports only the C ABI of
``include/gathered_rank_gemm.h``.  ``native/marshal.cpp`` becomes the Python module
``_native.so`` (argument marshalling of the per-token calls, against the installed
PyTorch); the library does not need it, and is there even where that module does not
compile.  No CPU fallback is built.
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
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libgathered_rank_gemm.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
NATIVE_SRC = os.path.join(HERE, "native", "marshal.cpp")
NATIVE_PATH = os.path.join(HERE, "_native.so")
NATIVE_FOR = os.path.join(BUILD_DIR, "native_for")  # the PyTorch that _native.so was compiled against
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + _headers())


def _older(path, deps) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _pytorch() -> str:
    """The installed PyTorch's version and place (without importing it)."""
    spec = importlib.util.find_spec("torch")
    return f"{importlib.metadata.version('torch')} {spec.origin}" if spec else "none"


def native_is_stale() -> bool:
    if _older(NATIVE_PATH, [NATIVE_SRC, *_headers()]) or not os.path.exists(NATIVE_FOR):
        return True
    with open(NATIVE_FOR) as f:
        return f.read() != _pytorch()


def library_is_stale() -> bool:
    return _older(LIB_PATH, _deps())


def is_stale() -> bool:
    return library_is_stale() or native_is_stale()


def _compile_native() -> str:
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    inc = [*cpp_extension.include_paths(), cuda, sysconfig.get_paths()["include"],
           os.path.join(ROOT, "include")]
    obj = os.path.join(BUILD_DIR, "marshal.cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in inc), "-c", NATIVE_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {NATIVE_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_native(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", f"-l:{LIB_NAME}", f"-L{lib}", "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE_PATH)
    with open(NATIVE_FOR, "w") as f:
        f.write(_pytorch())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library, then the module, where a source changed; returns the library's
    path.  The library is in place before a failure to compile the module is raised."""
    library, module = force or library_is_stale(), force or native_is_stale()
    if not library and not module:
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, *extra_flags, "-I", os.path.join(ROOT, "include"),
               "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        native = ex.submit(_compile_native) if module else None
        objs = list(ex.map(compile_one, _sources() if library else ()))
    if library:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    if native:
        _link_native(native.result())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
