"""Build of the kvq CUDA library (sm_103a), in-tree.

``ensure_built()`` compiles every ``csrc/*.cu`` translation unit in parallel
with nvcc for ``sm_103a`` and links ``_build/libkvq.so`` when any source or
header is newer than the library.  No other architecture is built.
``ensure_binding()`` compiles ``csrc/kvq_torch.cpp`` (host code) to an extension
module beside it, whose name holds the torch and the Python it was compiled for.
Processes that build at once wait for one another.
"""

from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libkvq.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the kvq CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if verbose_ptxas:
        print(r.stderr)
    return obj


@contextlib.contextmanager
def _building():
    """One process at a time: the objects and the outputs have fixed names."""
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)  # (let go of when the file is closed)
        yield


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link the library; returns its path."""
    if not force and not is_stale():
        return LIB
    with _building():
        if not force and not is_stale():  # built while this process waited
            return LIB
        with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
            objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), _sources()))
        tmp = LIB + ".tmp"
        r = subprocess.run([nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libkvq.so", "-o", tmp, *objs],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


def ensure_built() -> str:
    return build(force=False)


def _binding_sources():
    return [os.path.join(CSRC, "kvq_torch.cpp"), os.path.join(INCLUDE, "kvq.h"), os.path.abspath(__file__)]


def binding_path() -> str:
    """The extension module for this torch and this Python: neither's interface is stable across versions."""
    import sysconfig

    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(BUILD, f"_kvq_torch-torch{torch.__version__}-cxx11abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_is_stale(path: str) -> bool:
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in _binding_sources())


def ensure_binding() -> str:
    """Compile the extension module if a source of it is newer; returns its path.  It finds libkvq.so beside itself."""
    lib, path = ensure_built(), binding_path()
    if not _binding_is_stale(path):
        return path
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = path + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in inc),
           _binding_sources()[0], "-o", tmp, lib, f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{os.path.join(root, 'lib')}"]
    with _building():
        if not _binding_is_stale(path):  # built while this process waited
            return path
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for kvq_torch.cpp:\n{r.stderr}")
        os.replace(tmp, path)
    return path


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
