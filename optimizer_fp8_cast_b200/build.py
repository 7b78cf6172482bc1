"""Build libfp8train.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and _binding.so (the
Python binding of the calls whose host time matters, csrc/binding.cpp) with the host compiler.

    python -m optimizer_fp8_cast_b200.build [--verbose-ptxas]

One translation unit (csrc/fp8train.cu) holds every kernel, so the device error word is a
single symbol. No fast-math: the quantise, scale and AdamW arithmetic relies on IEEE rounding.
"""
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
MAIN = os.path.join(SRC_DIR, "fp8train.cu")
HEADER = os.path.join(ROOT, "include", "fp8train.h")
LIB = os.path.join(HERE, "libfp8train.so")
BINDING_SRC = os.path.join(SRC_DIR, "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _sources():
    out = [HEADER]
    for f in os.listdir(SRC_DIR):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(SRC_DIR, f))
    return out


def binding_key() -> str:
    """What the extension is compiled against: torch's C++ objects and Python's have other layouts in other versions."""
    import torch
    return "fp8t-binding torch %s cxx11abi %d %s" % (torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI),
                                                     sysconfig.get_config_var("SOABI"))


def binding_current() -> bool:
    """Whether the extension is there, newer than its sources, and built for this torch and Python."""
    if not os.path.exists(BINDING) or \
            os.path.getmtime(BINDING) < max(os.path.getmtime(BINDING_SRC), os.path.getmtime(HEADER)):
        return False
    with open(BINDING, "rb") as f:
        return binding_key().encode() in f.read()


def build_binding(force: bool = False) -> str:
    """Compile the extension against the installed torch's headers (it is loaded after torch, whose
    libraries give its symbols)."""
    if not force and binding_current():
        return BINDING
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
                    '-DFP8T_BUILT_FOR="%s"' % binding_key(),
                    "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
                    "-isystem", os.path.join(base, "include"),
                    "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                    "-isystem", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
                    BINDING_SRC, "-o", tmp, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch",
                    "-ltorch_cpu", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)
    return BINDING


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile the C library (it needs nvcc only)."""
    if not force and not needs_build():
        return LIB
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
           "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           "-o", tmp, MAIN]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Build what is out of date and return the library's path. Where the extension cannot be built (no C++ compiler,
    no CUDA build of torch) the library stands all the same, with a warning: only the calls that the extension binds
    are missing then, and they raise."""
    build_library(force, verbose_ptxas)
    try:
        build_binding(force)
    except (OSError, subprocess.CalledProcessError, ImportError) as e:
        if os.path.exists(BINDING):            # an older one may pass structures of an older header
            os.remove(BINDING)
        warnings.warn(f"{BINDING} could not be built, so the norm and 4-bit calls are missing: {e}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv))
