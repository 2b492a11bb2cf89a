"""Build the paged-attention CUDA library in-tree for sm_103a.

``python -m paged_kv_cache_201_gb300.build`` compiles every ``csrc/*.cu`` in
parallel with nvcc and links ``_build/libpaged_attn_gb300.so`` against the
shared CUDA runtime.  That is all the C ABI needs.  Where torch, its headers
and Python's are there too, it also compiles ``csrc/binding.cpp``, the short way
from Python into some of the calls; without it they go through ctypes.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libpaged_attn_gb300.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_NAME = "_paged_attn_binding"
BINDING_PATH = os.path.join(BUILD_DIR, BINDING_NAME + ".so")
BINDING_FOR = os.path.join(BUILD_DIR, BINDING_NAME + ".for")  # the torch and the Python that it was compiled against

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-cudart", "shared"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH_FLAGS, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    return obj


def _torch_dir():
    """torch's folder, found without importing it; None without torch."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def binding_lacks() -> str:
    """What the binding's compilation would need and is not there; empty if it can be compiled."""
    torch = _torch_dir()
    if torch is None:
        return "torch"
    if not os.path.exists(os.path.join(torch, "include", "ATen", "core", "Tensor.h")):
        return "torch's headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    if not shutil.which(os.environ.get("CXX", "g++").split()[0]):
        return "a C++ compiler"
    return ""


def binding_for() -> str:
    """The torch and the Python that a binding has to be compiled against."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = ""
    return f"{version} {_torch_dir()} {sysconfig.get_config_var('SOABI')}"


def binding_fits() -> bool:
    """Whether the binding is there and was compiled against this torch and this Python."""
    try:
        with open(BINDING_FOR) as f:
            return os.path.exists(BINDING_PATH) and f.read() == binding_for()
    except OSError:
        return False


def _binding_flags():
    """Include and link flags of torch, CUDA and Python."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    libs = [os.path.join(torch, "lib"), os.path.join(cuda, "lib64")]
    return [f"-I{d}" for d in inc], [f for d in libs for f in (f"-L{d}", f"-Wl,-rpath,{d}")] + [
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-lcudart"]


def _compile_binding() -> str:
    """The binding's object; it is linked once the library is there."""
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = [*os.environ.get("CXX", "g++").split(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *_binding_flags()[0], "-c",
           BINDING_SRC, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compiling {BINDING_SRC} failed:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [*os.environ.get("CXX", "g++").split(), "-shared", "-o", tmp, obj, f"-L{BUILD_DIR}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN",
           *_binding_flags()[1]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_FOR, "w") as f:
        f.write(binding_for())


def _newer(path: str, files) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in files)


def up_to_date() -> bool:
    return _newer(LIB_PATH, sources() + _headers() + [__file__]) and (
        bool(binding_lacks()) or (binding_fits() and _newer(BINDING_PATH, _headers() + [BINDING_SRC, __file__])))


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if stale) and return the path of the shared library."""
    if not force and not verbose_ptxas and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    if os.path.exists(BINDING_FOR):  # an old binding does not meet the new library
        os.remove(BINDING_FOR)
    lacks = binding_lacks()
    if lacks:
        sys.stderr.write(f"without the short way from Python into some calls: {lacks} not found\n")
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    if binding:
        _link_binding(binding.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
