"""The expert products' parameter blocks in C and in the binding, and the
scratch of down's unrounded slots (no GPU)."""

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
    """Twice the bytes: those of twice the columns."""
    f = lib.mr_expert_scratch_bytes
    need = f(DOWN["M"], DOWN["topk"], 2 * DOWN["R"])
    assert need >= DOWN["M"] * DOWN["topk"] * DOWN["R"] * 4
    short = dict(slots_fp32=1, scratch_bytes=need - 1)
    assert call(lib, "down", short) == mr.MR_ERR_SCRATCH_TOO_SMALL
    assert call(lib, "down", dict(slots_fp32=1, scratch_bytes=f(DOWN["M"], DOWN["topk"], DOWN["R"]))) \
        == mr.MR_ERR_SCRATCH_TOO_SMALL
