"""Build libfp4.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a.

    python -m block_scaled_fp4_05_b200.build [--force] [--verbose]

The library is compiled without fast-math (the quantizer relies on IEEE
division, reciprocal and products) and links the CUDA runtime dynamically.
The driver API (tensor-map encoding) is reached at run time through the
runtime's entry-point query, so libcuda is not a link dependency and the
library loads on machines without a GPU.

The Python calls of the INT8 entry points (csrc/int8_calls.cpp) are a small
extension module beside it, _int8_calls.so, compiled by g++ against torch's
headers: host code alone, which takes its entry points from libfp4.so.  It
holds what it was built for (torch's version, Python's ABI) and is built anew
when that changes.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp4.so")
SOURCES = ["api.cu", "quantize.cu", "gemm.cu", "quantize_int8.cu", "gemm_int8.cu", "gemv_int8.cu"]
HEADERS = ["fp4_internal.h", "quant_device.cuh", "tc_device.cuh", "int8_device.cuh"]
CALLS = os.path.join(HERE, "_int8_calls.so")
CALLS_SOURCE = os.path.join(CSRC, "int8_calls.cpp")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "shared",
    "-Xptxas", "-warn-spills",
]


def _nvcc():
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "fp4.h"))
    return files


def _newer(out, inputs):
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in inputs)


def calls_target():
    """What _int8_calls.so has to be built for: the layouts of torch's tensors
    and of Python's objects are compiled into it."""
    import torch

    return "torch %s, %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def lib_up_to_date():
    return _newer(LIB, _inputs())


def calls_up_to_date():
    if not _newer(CALLS, [CALLS_SOURCE, os.path.join(INCLUDE, "fp4.h")]):
        return False
    with open(CALLS, "rb") as f:
        return calls_target().encode() + b"\0" in f.read()


def up_to_date():
    return lib_up_to_date() and calls_up_to_date()


def build_calls(verbose=False):
    """_int8_calls.so: torch (already loaded wherever it is imported) provides
    every symbol that it does not define."""
    import torch

    home = os.path.dirname(torch.__file__)
    tmp = CALLS + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wno-attributes",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           '-DFP4_BUILT_FOR="%s"' % calls_target(),
           "-I", os.path.join(home, "include"),
           "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", sysconfig.get_paths()["include"], "-o", tmp, CALLS_SOURCE,
           "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, CALLS)
    return CALLS


def build_lib(verbose=False):
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-o", tmp] + [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        cmd.insert(1, "-Xptxas")
        cmd.insert(2, "-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


def build(force=False, verbose=False):
    if force or not lib_up_to_date():
        build_lib(verbose)
    if force or not calls_up_to_date():
        build_calls(verbose)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
