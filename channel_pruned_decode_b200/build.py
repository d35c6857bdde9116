"""Build the SparK CUDA library (libspark.so) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspark.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_TAG = os.path.join(PKG, "_build", "calls_tag")

SOURCES = ["api.cu", "prune.cu", "decode.cu", "snapkv.cu", "think.cu", "pages.cu", "kv8.cu", "attn_kv8.cu"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the SparK CUDA library cannot be built")


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def calls_tag() -> str:
    """What _calls.so is compiled for: it has torch's tensor accessors and
    Python's object layout compiled in, so it fits this torch and Python only."""
    import sysconfig

    import torch
    return f"torch {torch.__version__}, Python {sysconfig.get_config_var('SOABI')}"


def calls_stale() -> bool:
    """Whether _calls.so has to be compiled (again)."""
    if _stale(CALLS, [os.path.join(CSRC, "calls.cpp"), os.path.join(INCLUDE, "spark.h"), LIB]):
        return True
    try:
        with open(CALLS_TAG) as f:
            return f.read() != calls_tag()
    except OSError:
        return True


def build_calls(force: bool = False) -> str:
    """Compile csrc/calls.cpp, the native half of the binding of the paged
    8-bit cache's calls, into _calls.so beside libspark.so."""
    if not force and not calls_stale():
        return CALLS
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    src = os.path.join(CSRC, "calls.cpp")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [INCLUDE, sysconfig.get_path("include"), cuda, *include_paths()]
    cmd = ["g++", "-shared", "-fPIC", "-O2", "-std=c++17", "-fvisibility=hidden", "-Wall", "-Wextra",
           f'-DSPARK_BUILT_FOR="{calls_tag()}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for i in includes for x in ("-isystem", i)] + [src, "-o", CALLS + ".tmp"]
    for d in library_paths():
        cmd += ["-L", d]
    cmd += ["-L", PKG, "-lspark", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(CALLS + ".tmp", CALLS)
    os.makedirs(os.path.dirname(CALLS_TAG), exist_ok=True)
    with open(CALLS_TAG, "w") as f:
        f.write(calls_tag())
    return CALLS


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into libspark.so (exported: the C ABI of
    include/spark.h only).  Returns the library path."""
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, "spark_internal.cuh"), os.path.join(CSRC, "kv8.cuh"), os.path.join(INCLUDE, "spark.h")]
    if not force and not _stale(LIB, deps):
        build_calls()
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for s in srcs:
        o = os.path.join(objdir, os.path.basename(s).replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-c", s, "-o", o]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        objs.append(o)
    tmp = LIB + ".tmp"
    # static CUDA runtime: the library needs no libcudart on the loader path
    subprocess.run([nvcc, "-shared", "-cudart", "static", "-gencode", "arch=compute_100a,code=sm_100a",
                    "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    build_calls(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
