"""Stream order of launches that may overlap the kernel before them, read off
the sources (the library launches every kernel so under MR_LAUNCH_PDL)."""

import os
import re

import decode_expert_routing_gb300 as mr

CSRC = os.path.join(os.path.dirname(os.path.abspath(mr.__file__)), "csrc")


def _body(text, start):
    """The braces that follow position start of text."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i:j + 1]
    raise AssertionError("unbalanced braces")


def _functions():
    """({kernel: body}, {device function: [bodies]}) of every source."""
    kernels, device = {}, {}
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as src:
            text = re.sub(r"//[^\n]*", "", src.read())
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\((?:[^()]|\([^()]*\))*\)\s*)?(\w+)\s*\(", text):
            kernels[m.group(1)] = _body(text, m.end())
        for m in re.finditer(r"__device__ __forceinline__ [\w:]+ (\w+)\s*\(", text):
            device.setdefault(m.group(1), []).append(_body(text, m.end()))
    return kernels, device


def test_every_kernel_waits_for_the_kernel_before_it():
    kernels, device = _functions()
    assert len(kernels) >= 11 and "mx_pack_kernel" in kernels and "expert_kernel" in kernels

    def waits(body, seen=frozenset()):
        if "pdl_wait()" in body:
            return True
        calls = set(re.findall(r"\b(\w+)\s*(?:<[^;{}()]*>)?\(", body)) & set(device) - seen
        return any(waits(b, seen | calls) for c in calls for b in device[c])

    late = [k for k, body in kernels.items() if not waits(body)]
    assert not late, f"kernels that never wait for the one before them: {late}"
