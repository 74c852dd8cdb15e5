"""Rules that the kernels' sources keep and no run can show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp4_05_b200", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def read_only_loads():
    """Names of the headers' device functions that load through the read-only path."""
    names = []
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".h", ".cuh")):
            names += re.findall(r"__device__[^;{}]*?\b(\w+)\s*\([^)]*\)\s*\{(?:(?!\n\}).)*?ld\.global\.nc", code(name), re.S)
    return names


# Kernels launched with programmatic serialization start before the kernel
# before them has ended.  What that one writes may not be read through the
# read-only path, whose data have to stay as they are while the kernel lives.
@pytest.mark.parametrize("name", ["quantize_int8.cu", "gemm_int8.cu", "gemv_int8.cu"])
def test_early_started_kernels_do_not_read_through_the_read_only_path(name):
    text = code(name)
    assert "cudaLaunchAttributeProgrammaticStreamSerialization" in text
    assert "ld_stream" in read_only_loads()
    for word in ["ld.global.nc", "__ldg"] + [r"\b%s\(" % n for n in read_only_loads()]:
        if name == "gemv_int8.cu" and word == r"\bld_stream\(":
            continue   # (its own, the load without .nc)
        assert not re.search(word, text), word
