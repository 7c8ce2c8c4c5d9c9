"""Builds librswa.so in-tree from csrc/*.cu for sm_100a with nvcc, and the binding's tensor
checks (_tensors.<key>.so, from csrc/tensors.cpp) with g++.

Run as ``python -m long_context_decode_swa_b200.build`` or call ``build()``.
Objects go to ``long_context_decode_swa_b200/_build/`` and the library to
``long_context_decode_swa_b200/librswa.so``; a rebuild happens only when a
source or header is newer than the library.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librswa.so")
EXT_SRC = os.path.join(CSRC, "tensors.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librswa.so")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def ext_path() -> str:
    """Where the extension for this PyTorch, this Python and this source is: its name says all three, so that one
    built against others, whose object layouts may differ, is never loaded."""
    import hashlib
    import sysconfig

    import torch
    with open(EXT_SRC, "rb") as f:
        key = hashlib.sha256(f.read())
    key.update(f"{torch.__version__} {torch.compiled_with_cxx11_abi()} {sysconfig.get_config_var('EXT_SUFFIX')}".encode())
    return os.path.join(PKG, f"_tensors.{key.hexdigest()[:16]}.so")


def build_ext(force: bool = False) -> str:
    """The CPython extension that checks tensors (no CUDA in it)."""
    ext = ext_path()
    if not force and os.path.exists(ext):
        return ext
    import sysconfig

    import torch
    # torch's own header and library folders, without importing its extension builder (which looks for a GPU)
    home = os.path.dirname(torch.__file__)
    includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"]]
    tmp = ext + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-I{d}" for d in includes], EXT_SRC, "-o", tmp, f"-L{os.path.join(home, 'lib')}", "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    if shutil.which(cmd[0]) is None:
        raise RuntimeError(f"g++ not found: it builds {EXT_SRC}")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {EXT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ext)
    return ext


def build_lib(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """librswa.so, which needs neither PyTorch nor Python's headers."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """The library, then the tensor checks (left out, with a note, where there is no PyTorch or no g++)."""
    lib = build_lib(force, verbose, extra_flags)
    if importlib.util.find_spec("torch") is None or shutil.which("g++") is None:
        print(f"{EXT_SRC} not built: it needs PyTorch and g++", file=sys.stderr)
    else:
        build_ext(force)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
