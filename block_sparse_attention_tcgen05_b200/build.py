"""Builds libbsa.so (the C-ABI library, nvcc for sm_100a) and _native.so (the native
marshalling of the calls that run down to single tokens, g++ against torch) in-tree."""

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libbsa.so")
SRC = os.path.join(HERE, "csrc", "libbsa.cu")
NATIVE = os.path.join(HERE, "_native.so")
NATIVE_SRC = os.path.join(HERE, "csrc", "binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O3",
    "-shared",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    d = os.path.join(HERE, "csrc")
    return [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh"))] + [
        os.path.join(ROOT, "include", "bsa.h")]


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def native_id():
    """What _native.so is compiled against, as it holds it: torch's C++ ABI changes with its version,
    the interpreter's with its own."""
    import torch
    return f"bsa native module for torch {torch.__version__}, {sys.implementation.cache_tag};"


def native_up_to_date():
    """Whether _native.so is newer than its sources and was built against this torch and
    interpreter."""
    if not os.path.exists(NATIVE):
        return False
    t = os.path.getmtime(NATIVE)
    if any(os.path.getmtime(s) > t for s in (NATIVE_SRC, os.path.join(ROOT, "include", "bsa.h"))):
        return False
    with open(NATIVE, "rb") as f:
        return native_id().encode() in f.read()


def _native_command(out):
    import torch
    t = os.path.dirname(torch.__file__)
    inc = [os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DBSA_NATIVE_ID="{native_id()}"',
            *[x for i in inc for x in ("-isystem", i)], NATIVE_SRC, "-o", out,
            "-L", HERE, "-l:libbsa.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(t, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def _compile(cmd, out, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed building {os.path.basename(out)}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(out + ".tmp", out)


def build_native(force=False, verbose=False):
    """Compile _native.so unless it is up to date. Returns its path."""
    if force or not native_up_to_date():
        _compile(_native_command(NATIVE + ".tmp"), NATIVE, verbose)
    return NATIVE


def build(force=False, verbose=False, extra=()):
    """Compile libbsa.so and _native.so unless they are up to date. Returns the path of
    libbsa.so."""
    if force or not up_to_date():
        _compile([NVCC, *FLAGS, *extra, SRC, "-o", LIB + ".tmp"], LIB, verbose)
    build_native(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=("-Xptxas", "-v") if "--ptxas-v" in sys.argv else ())
