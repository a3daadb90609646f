"""Build libsnk.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each .cu file compiles in its own nvcc process, in parallel; the objects are
linked into ``sparse_linear_layer_gb300/libsnk.so`` with the CUDA runtime
linked statically, so the library only needs the driver at run time.  Beside it
g++ builds ``_q8ops.so``, the Python module that calls it on torch tensors, for the
torch that is installed; without one there is only the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsnk.so")
OPS_SRC = os.path.join(CSRC, "q8_ops.cpp")
OPS = os.path.join(PKG, "_q8ops.so")   # the torch side of the 8-bit activation calls
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}",
         "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "snk.h")]


def _torch_key() -> str | None:
    """What _q8ops.so is built for: the Python and the torch (None: there is none)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        return f"{sys.implementation.cache_tag} {spec.origin}\n{f.read()}"


def has_torch() -> bool:
    return _torch_key() is not None


def _key_file() -> str:
    return os.path.join(OBJ, "_q8ops.key")


def _lib_up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _ops_up_to_date() -> bool:
    key = _torch_key()
    if key is None:
        return True
    if not os.path.exists(OPS) or not os.path.exists(_key_file()):
        return False
    with open(_key_file()) as f:
        if f.read() != key:
            return False
    return max(os.path.getmtime(p) for p in (OPS_SRC, os.path.join(INCLUDE, "snk.h"))) <= os.path.getmtime(OPS)


def up_to_date() -> bool:
    return _lib_up_to_date() and _ops_up_to_date()


def _compile(src: str, verbose: bool, obj_dir: str, extra) -> str:
    obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _build_ops() -> None:
    """_q8ops.so: g++ against torch's headers (no torch build tools)."""
    import sysconfig

    import torch
    key = _torch_key()
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"), INCLUDE]
    tmp = OPS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{p}" for p in inc), OPS_SRC,
           "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {OPS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS)
    with open(_key_file(), "w") as f:
        f.write(key)


def build(force: bool = False, verbose: bool = False, extra_flags=None, out: str | None = None) -> str:
    """Compile libsnk.so.  extra_flags (e.g. ["-DSNK_PIPE_FWD=3"]) and out
    (another library path) build a variant beside the default library.
    Processes that build at the same time (one per GPU) take turns on a lock
    file; the later ones then find the library up to date."""
    import fcntl
    extra = list(extra_flags or [])
    lib = out or LIB
    if not force and not extra and out is None and up_to_date():
        return LIB
    obj_dir = OBJ if out is None else out + ".objs"
    os.makedirs(obj_dir, exist_ok=True)
    with open(os.path.join(obj_dir, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if not force and not extra and out is None and up_to_date():
            return LIB
        all_of_it = force or bool(extra) or out is not None
        with cf.ThreadPoolExecutor(max_workers=1) as ex:
            # (the library does not depend on the torch module: it is linked whether or not that compiles)
            ops = ex.submit(_build_ops) if lib == LIB and _torch_key() and (all_of_it or not _ops_up_to_date()) else None
            if all_of_it or not _lib_up_to_date():
                _build_lib(verbose, extra, lib, obj_dir)
            if ops is not None:
                ops.result()
        return lib


def _build_lib(verbose: bool, extra, lib: str, obj_dir: str) -> None:
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, obj_dir, extra), srcs))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
