"""Build the CUDA library in-tree for sm_100a.

    python -m bigvgan_waveform_decoder_b200.build     # writes bigvgan_waveform_decoder_b200/libmh3a.so

nvcc compiles every csrc/*.cu for sm_100a and links one shared library exporting the C ABI of
include/mh3a.h.  Where torch is installed it then builds _ops.so, the operators' front end for torch
tensors, on that library and that torch.  No GPU is needed to build.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from importlib import metadata

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmh3a.so")
OPS_SRC = os.path.join(CSRC, "torch_ops.cpp")
OPS = os.path.join(HERE, "_ops.so")
OPS_STAMP = os.path.join(HERE, "_build", "_ops.stamp")  # what OPS was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(ROOT, "include", "mh3a.h"), os.path.abspath(__file__)]


def _newer(out, deps) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """Both; without torch the library alone, which is all that the decoder needs."""
    build_library(force, verbose, extra)
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: the operators' front end (_ops.so) is not built", file=sys.stderr)
    else:
        build_ops(force, verbose)
    return LIB


def ops_stamp() -> str:
    """What else than its sources _ops.so depends on: torch, Python and the compiler."""
    return "\n".join((metadata.version("torch"), sysconfig.get_config_var("SOABI"), NVCC))


def _ops_stamp_is(stamp) -> bool:
    try:
        with open(OPS_STAMP) as f:
            return f.read() == stamp
    except OSError:
        return False


def build_ops(force: bool = False, verbose: bool = False) -> str:
    """_ops.so: csrc/torch_ops.cpp against libmh3a.so and torch."""
    header = os.path.join(ROOT, "include", "mh3a.h")
    stamp = ops_stamp()
    if not force and _ops_stamp_is(stamp) and _newer(OPS, [OPS_SRC, header, os.path.abspath(__file__)]):
        return OPS
    import torch
    from torch.utils.cpp_extension import include_paths

    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [*include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = OPS + f".tmp{os.getpid()}"
    # nvcc hands the file to its host compiler and links the C++ library dynamically, as for libmh3a.so:
    # a copy of its own inside _ops.so would not get along with torch's
    cmd = [NVCC, *FLAGS[:2], "-shared", "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_ops",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *[f for i in inc for f in ("-isystem", i)],
           OPS_SRC, "-o", tmp, "-L", HERE, "-l:libmh3a.so", "-Xlinker", "-rpath=$ORIGIN", "-L", lib, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "--cudart", "none"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OPS)
    os.makedirs(os.path.dirname(OPS_STAMP), exist_ok=True)
    with open(OPS_STAMP, "w") as f:
        f.write(stamp)
    return OPS


def build_library(force: bool = False, verbose: bool = False, extra=None) -> str:
    if not force and up_to_date():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((subprocess.Popen(cmd), cmd))
        objs.append(obj)
    for p, cmd in procs:
        if p.wait() != 0:
            raise RuntimeError("nvcc failed: " + " ".join(cmd))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC",
           *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
