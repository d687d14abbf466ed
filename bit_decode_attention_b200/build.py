"""Build libnvfp4kv.so in-tree for sm_100a (B200).

    python -m bit_decode_attention_b200.build [--force]

nvcc compiles every .cu under csrc/ into one shared library next to this
file, and g++ the argument marshalling under csrc/binding/ into the extension
module _binding.so beside it.  No --use_fast_math: the quantizer relies on IEEE fp32 division and
rounding (-prec-div=true, -prec-sqrt=true, -ftz=false, -fmad=false).
"""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libnvfp4kv.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding", "nvfp4kv_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
    "-prec-div=true", "-prec-sqrt=true", "-ftz=false", "-fmad=false",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libnvfp4kv.so")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The Python extension module: g++ against torch's headers, linked with the library beside it."""
    inputs = [BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in inputs):
        return BINDING
    import torch
    from torch.utils import cpp_extension
    tmp = BINDING + ".tmp%d" % os.getpid()
    dirs = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           *(f for d in dirs for f in ("-isystem" if d != INCLUDE else "-I", d)), BINDING_SRC, "-o", tmp,
           "-L", HERE, "-lnvfp4kv", "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        build_binding(False, verbose)
        return LIB
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-o", tmp, *sources(), "-lcudart"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    flags = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(flags), verbose=True, extra_flags=flags))
