"""Build libkda.so in-tree with nvcc for sm_103a, and the binding's C++ half with g++.

Each .cu under csrc/ is compiled to an object in parallel, then linked into
``gated_delta_rule_intra_gb300/libkda.so`` (git-ignored).  No CMake, no torch
extension machinery: the library is a plain C-ABI shared object.  csrc/binding.cpp becomes
``_native.so``, compiled against the installed torch's headers next to it.
(Only the short way into the recurrence, the single-token form and layer norm is in it.)
``build_debug_library()`` builds the same sources with ``-DKDA_DEBUG_CHECKS`` into
``libkda_debug.so``: every global index the kernels compute is checked against its
buffer's extent and reported through ``kda_debug_set_flags`` (tests only).
"""

from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libkda.so")
NATIVE = os.path.join(PKG, "_native.so")
DEBUG_LIB = os.path.join(PKG, "libkda_debug.so")
BUILD_DIR = os.path.join(PKG, "_build")
DEBUG_BUILD_DIR = os.path.join(PKG, "_build_debug")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Hidden visibility: only the C ABI (kda_api.cu) is exported.  Two builds loaded in one
# process (libkda.so and libkda_debug.so) then share no C++ internals; in particular no
# function-local static of a template becomes a process-wide unique symbol.
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _compile(src: str, extra, build_dir: str) -> str:
    obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def build_native() -> str:
    """Compile csrc/binding.cpp into _native.so; returns its path."""
    import torch

    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    headers = [os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = NATIVE + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), *[x for h in headers for x in ("-isystem", h)],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-Wl,-rpath," + os.path.join(home, "lib")]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, NATIVE)
    return NATIVE


def build_library(out: str = LIB, extra_flags=(), verbose: bool = False,
                  build_dir: str = BUILD_DIR) -> str:
    """Compile every csrc/*.cu for sm_103a and link libkda.so; returns its path.  Together with
    libkda.so itself _native.so is built."""
    os.makedirs(build_dir, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        native = ex.submit(build_native) if out == LIB else None
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags), build_dir), srcs))
        if native:
            native.result()
    tmp = out + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, out)
    if verbose:
        print(f"built {out}")
    return out


def build_debug_library(verbose: bool = False) -> str:
    """The bounds-checked debug build, libkda_debug.so; returns its path."""
    return build_library(DEBUG_LIB, ["-DKDA_DEBUG_CHECKS"], verbose, DEBUG_BUILD_DIR)


if __name__ == "__main__":
    build_library(verbose=True)
    build_debug_library(verbose=True)
