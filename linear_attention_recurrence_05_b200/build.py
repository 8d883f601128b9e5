"""Build libgdn.so in-tree: every .cu under csrc/ compiled for sm_100a with nvcc.

    python -m linear_attention_recurrence_05_b200.build [--force] [-j N]

The library links the CUDA runtime statically, so it loads next to any PyTorch
build; it exports only the C ABI of include/libgdn.h.  The Python package's native host path
(csrc/fast_calls.cpp -> _fast.so) is compiled after it, against the installed PyTorch; where there is
none the library alone is built, and the package's calls do without.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
FAST_SRC = os.path.join(CSRC, "fast_calls.cpp")
FAST = os.path.join(PKG, "_fast.so")
FAST_KEY = os.path.join(BUILD, "_fast.key")          # what the present _fast.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}"]


def _deps() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def fast_key() -> str:
    """The PyTorch and Python whose headers and object layouts are compiled into _fast.so."""
    import torch
    return (f"PyTorch {torch.__version__}, C++ ABI {int(torch.compiled_with_cxx11_abi())}, "
            f"{sys.implementation.cache_tag} {sys.version.split()[0]}")


def _build_fast(force: bool) -> None:
    try:
        import torch
    except ImportError:
        sys.stderr.write("no PyTorch: libgdn.so is built, the Python package's _fast.so is not\n")
        return
    import sysconfig
    key, built_for = fast_key(), None
    if os.path.exists(FAST_KEY):
        with open(FAST_KEY, encoding="utf-8") as f:
            built_for = f.read()
    newest = max(os.path.getmtime(p) for p in [FAST_SRC, os.path.join(INCLUDE, "libgdn.h"), os.path.abspath(__file__)])
    if not force and os.path.exists(FAST) and os.path.getmtime(FAST) >= newest and built_for == key:
        return
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = f"{FAST}.{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DGDN_BUILT_FOR="{key}"', f"-I{INCLUDE}",
           f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{sysconfig.get_path('include')}", FAST_SRC, "-o", tmp, f"-L{root}/lib", "-lc10", "-lc10_cuda", "-ltorch",
           "-ltorch_cpu", "-Wl,--no-as-needed", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"libgdn.so is built, but g++ failed on {FAST_SRC}:\n{r.stderr}")
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(FAST_KEY):                          # (no moment at which the key describes another file)
        os.remove(FAST_KEY)
    os.replace(tmp, FAST)
    with open(FAST_KEY, "w", encoding="utf-8") as f:
        f.write(key)


def _compile(src: str) -> tuple:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    return obj, r.stderr


def _build_lib(force: bool, jobs: int, verbose: bool) -> None:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest = max(os.path.getmtime(p) for p in _deps() + [os.path.abspath(__file__)])
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest:
        return
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs))) as ex:
        results = list(ex.map(_compile, srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = f"{LIB}.{os.getpid()}.tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, jobs: int = 0, verbose: bool = False) -> str:
    """Builds libgdn.so, which needs nvcc alone, then _fast.so where there is a PyTorch to build it for."""
    _build_lib(force, jobs, verbose)
    _build_fast(force)
    return LIB


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=0)
    ap.add_argument("-v", action="store_true", help="print ptxas resource usage")
    a = ap.parse_args()
    print(build(force=a.force, jobs=a.j, verbose=a.v))


if __name__ == "__main__":
    main()
