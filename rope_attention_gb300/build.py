"""Builds librope_attention.so in-tree from csrc/*.cu for sm_103a.

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into one shared library with the CUDA runtime linked statically, so the
library loads on a machine without a GPU driver (calls then fail with
RA_ERR_CUDA) and needs no libcudart at run time.  It needs nvcc alone.

Beside it, _torch_calls.<interpreter>-<torch>.so: the attention calls with torch tensors.  It is
compiled against this interpreter's and its torch's headers and named after both, so a
module for another torch is never loaded.  Where the headers or g++ are missing it is left
out, which build() says, and the calls that need it say so too.

    python -m rope_attention_gb300.build            # build if out of date
    python -m rope_attention_gb300.build --force    # rebuild
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "librope_attention.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["api.cu", "qkv_project.cu", "qk_norm_rope.cu", "kv_cache.cu", "noalloc.cu", "row_quant.cu",
           "packed_attention.cu", "paged_attention.cu", "paged_tile.cu", "cache_read.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin directory on PATH)")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "rope_attention.h"))
    files.append(os.path.abspath(__file__))
    return files


def _torch_root() -> str | None:
    """Where this interpreter's torch is, without the seconds that importing it takes."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None or not spec.origin else os.path.dirname(spec.origin)


def _torch_version() -> str:
    root = _torch_root()
    if root is None:
        return "none"
    try:
        with open(os.path.join(root, "version.py")) as f:
            found = re.search(r"^__version__\b[^=\n]*= *['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        found = None
    return found.group(1) if found else "unknown"


# the calls with torch tensors, linked to the library
CALLS_PATH = os.path.join(PKG, f"_torch_calls.{sys.implementation.cache_tag}-torch{_torch_version()}.so")


def calls_missing() -> str | None:
    """What building the calls with torch tensors lacks here; None if nothing."""
    root = _torch_root()
    if root is None:
        return "torch is not installed"
    if shutil.which("g++") is None:
        return "g++ is not on PATH"
    for header in (os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(header):
            return f"{header} does not exist"
    return None


def _fresh(path: str) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in _inputs())


def up_to_date() -> bool:
    return _fresh(LIB_PATH) and (_fresh(CALLS_PATH) or calls_missing() is not None)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), "-c", os.path.join(CSRC, src), "-o", obj, "-O3", "-std=c++17", "-lineinfo",
           *ARCH, "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def _compile_calls() -> str:
    """csrc/torch_calls.cpp, against this interpreter's torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-c", os.path.join(CSRC, "torch_calls.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem", cuda]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_PATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS_PATH)


def _link(objs: list[str]) -> None:
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static", "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    missing = calls_missing()
    if missing is not None:
        print(f"the attention calls with torch tensors are not built: {missing}", file=sys.stderr)
    want_lib = force or not _fresh(LIB_PATH)
    want_calls = missing is None and (force or not _fresh(CALLS_PATH))
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls) if want_calls else None
        if want_lib:
            _link(list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES)))
    if calls is not None:
        _link_calls(calls.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
