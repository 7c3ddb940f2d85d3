"""The expert products' parameter blocks in C and in the binding, and the
second scratch buffer of down (no GPU)."""

import ctypes
import subprocess

import pytest

import decode_expert_routing_gb300 as mr
from decode_expert_routing_gb300 import build as mrbuild
from tests.test_experts_cpu import DOWN, call

BLOCKS = [("mr_mx_gemm_params", "MxGemmParams"), ("mr_moe_gate_up_params", "GateUpParams"),
          ("mr_moe_down_params", "DownParams")]


@pytest.fixture(scope="module")
def lib():
    mrbuild.build()
    return mr.load_library()


@pytest.mark.parametrize("name,cls", BLOCKS)
def test_parameter_blocks_match_the_header(tmp_path, name, cls):
    cls = getattr(mr, cls)
    fields = [f for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "moe_route.h"\nint main(void) {\n'
                   + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields)
                   + f'  printf("%zu\\n", sizeof({name}));\n  return 0;\n}}\n')
    subprocess.run(["gcc", "-std=c11", "-I", mrbuild.INCLUDE, "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(cls, f).offset for f in fields] + [ctypes.sizeof(cls)]


def test_scratch_of_unrounded_slots(lib):
    """The buffer of the lower halves is checked as the other one."""
    need = lib.mr_expert_scratch_bytes(DOWN["M"], DOWN["topk"], DOWN["R"])
    low = DOWN["scratch"]
    assert call(lib, "down", dict(scratch_low=low, scratch_low_bytes=need - 1)) == mr.MR_ERR_SCRATCH_TOO_SMALL
    assert call(lib, "down", dict(scratch_low=low + 16, scratch_low_bytes=need)) == mr.MR_ERR_INVALID_ARG
