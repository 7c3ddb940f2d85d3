"""Loads of kernels that may start before the kernel launched before them has ended, read off the sources."""

import os
import re

import decode_expert_routing_gb300 as mr

CSRC = os.path.join(os.path.dirname(os.path.abspath(mr.__file__)), "csrc")


def _sources():
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as src:
            yield f, re.sub(r"//[^\n]*", "", src.read())


def test_what_the_kernel_before_may_write_is_not_read_as_constant():
    """A load by the read-only path states that the memory does not change while the kernel is resident, so the compiler
    may put it before griddepcontrol.wait.  Only weights that the header lets be read there are loaded so."""
    constant, weights = [], []
    for f, text in _sources():
        assert "__restrict__" not in text, f
        for m in re.finditer(r"ld\.global\.nc\b|ld\.global\.[\w.:]*\.nc\b|__ldg\(([^;]*)", text):
            constant.append((f, (m.group(1) or "nc").split(")")[0]))
        weights += [(f, m.group(1)) for m in re.finditer(r"ld_weight_v4\((\w+)(?: \+[^;]*)?\)", text)]
    assert constant == [("common.cuh", "nc"), ("route_kernel.cuh", "src + b0 + b")]
    assert weights == [("gemv.cuh", "wrow"), ("route_kernel.cuh", "wp")]
    route = dict(_sources())["route_kernel.cuh"]
    # (the shared expert's scale bytes, with its codes)
    at = route.index("__ldg(src + b0 + b)")
    assert "const uint8_t* src = sg8" in route[at - 400:at] and route.index("pdl_wait();", at) - at < 400


def test_the_bias_is_read_after_the_wait():
    route = dict(_sources())["route_kernel.cuh"]
    kernel = route[route.index("route_cluster_kernel(RouteArgs a)"):]
    assert kernel.index("pdl_wait();") < kernel.index("a.bias[")
