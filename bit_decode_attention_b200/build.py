"""Build libnvfp4kv.so in-tree for sm_100a (B200).

    python -m bit_decode_attention_b200.build [--force]

nvcc compiles every .cu under csrc/ into one shared library next to this
file, and g++ the argument marshalling under csrc/binding/ into the extension
module _binding.so beside it (where torch's and Python's headers are).  No --use_fast_math: the quantizer relies on IEEE fp32 division and
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


def binding_needs() -> str:
    """What this host lacks for the extension module, or an empty string.  (The library
    itself needs nvcc and its host compiler only.)"""
    try:
        import torch  # noqa: F401
    except ImportError as e:
        return "torch cannot be imported (%s)" % e
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers are not installed"
    return "" if shutil.which("g++") else "g++ is not installed"


def binding_stamp() -> str:
    """What the extension module is compiled against; it holds this text."""
    import torch
    return "nvfp4kv binding for torch %s, Python %s" % (torch.__version__, sys.version.split()[0])


def binding_up_to_date() -> bool:
    """Newer than its sources, and built against the torch and Python at hand."""
    if not os.path.exists(BINDING):
        return False
    t = os.path.getmtime(BINDING)
    if any(os.path.getmtime(f) > t for f in (BINDING_SRC, *glob.glob(os.path.join(INCLUDE, "*.h")))):
        return False
    with open(BINDING, "rb") as f:
        return binding_stamp().encode() + b"\0" in f.read()


def build_binding(force: bool = False, verbose: bool = False) -> bool:
    """The Python extension module: g++ against torch's headers, linked with the library
    beside it.  Where those are missing it is left out, and said so."""
    lacks = binding_needs()
    if lacks:
        print("_binding.so is not built, the tree-step calls of the Python package will not run: %s" % lacks, file=sys.stderr)
        return False
    if not force and binding_up_to_date():
        return True
    import torch
    from torch.utils import cpp_extension
    tmp = BINDING + ".tmp%d" % os.getpid()
    dirs = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [shutil.which("g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DNVFP4_BINDING_STAMP="%s"' % binding_stamp(),
           *(f for d in dirs for f in ("-isystem" if d != INCLUDE else "-I", d)), BINDING_SRC, "-o", tmp,
           "-L", HERE, "-lnvfp4kv", "-Wl,-rpath,$ORIGIN", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    return True


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
