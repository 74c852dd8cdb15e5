"""What is built anew when: the library by its sources, the extension module of
the INT8 calls also by the torch and the Python that it was compiled for.  And
which sources the recorded DRAM traffic of the FP4 kernels hangs on."""
import os
import shutil
import sys

import pytest
import torch

from block_scaled_fp4_05_b200 import build, fp4


@pytest.fixture
def built(monkeypatch):
    """Names of what build() builds, with everything newer than its sources."""
    names, newer = [], {build.LIB: True, build.CALLS: True}
    monkeypatch.setattr(build, "_newer", lambda out, inputs: newer[out])
    monkeypatch.setattr(build, "build_lib", lambda verbose=False: names.append("lib"))
    monkeypatch.setattr(build, "build_calls", lambda verbose=False: names.append("calls"))
    return names, newer


def test_nothing_is_built_while_all_is_current(built):
    build.build()
    assert built[0] == []
    build.build(force=True)
    assert built[0] == ["lib", "calls"]


@pytest.mark.parametrize("part", ["lib", "calls"])
def test_each_part_is_built_by_itself(built, part):
    built[1][build.LIB if part == "lib" else build.CALLS] = False
    assert not build.up_to_date()
    build.build()
    assert built[0] == [part]


def test_another_torch_or_python_needs_another_module(built, monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        assert not build.up_to_date()
        build.build()
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
        assert not build.up_to_date()
        build.build()
    assert built[0] == ["calls", "calls"] and build.up_to_date()


def test_a_module_built_for_another_torch_is_not_used(monkeypatch):
    monkeypatch.setattr(fp4, "_calls", None)
    assert fp4._int8_calls().built_for == build.calls_target()
    monkeypatch.setattr(fp4, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for torch .*, this is torch 0.0.1"):
        fp4._int8_calls()


def test_why_a_module_does_not_load_is_said(monkeypatch):
    name = "block_scaled_fp4_05_b200._int8_calls"
    monkeypatch.setattr(fp4, "_calls", None)
    monkeypatch.delattr(sys.modules["block_scaled_fp4_05_b200"], "_int8_calls", raising=False)
    monkeypatch.setitem(sys.modules, name, None)
    with pytest.raises(RuntimeError, match="cannot be loaded .*%s" % os.path.basename(name)):
        fp4._int8_calls()


def test_recorded_traffic_hangs_on_the_headers_too(tmp_path):
    import bench
    sources = bench.kernel_sources(build.CSRC)
    assert {"gemm.cu", "quantize.cu", "tc_device.cuh", "quant_device.cuh", "fp4_internal.h"} <= set(sources)
    for name in sources:
        copy = str(tmp_path / name)
        shutil.copytree(build.CSRC, copy)
        assert bench.kernel_source_hash(copy) == bench.kernel_source_hash()
        with open(os.path.join(copy, name), "a") as f:
            f.write("// another byte\n")
        assert bench.kernel_source_hash(copy) != bench.kernel_source_hash()
    with open(os.path.join(copy, "gemm_int8.cu"), "a") as f:   # no part of these kernels
        f.write("\n")
    with open(os.path.join(copy, name), "rb+") as f:
        f.seek(-len("// another byte\n"), 2)
        f.truncate()
    assert bench.kernel_source_hash(copy) == bench.kernel_source_hash()
