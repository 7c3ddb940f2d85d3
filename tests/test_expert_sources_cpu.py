"""What the expert kernel's hand-overs promise each other, read off the sources."""

import os
import re

import decode_expert_routing_gb300 as mr

CSRC = os.path.join(os.path.dirname(os.path.abspath(mr.__file__)), "csrc")


def _read(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_operands_are_handed_to_another_cta_by_a_release():
    """A pair's first CTA issues products that read the second one's shared memory.  Relaxed arrivals publish nothing:
    the kernel has them only where an accumulator is given back, whose reads are over when the arrival is issued."""
    kernel, helpers = _read("expert_gemm.cuh"), _read("cluster.cuh")
    calls = dict(re.findall(r"\b(mbar_arrive_remote\w*)\(([^;]*)\);", kernel))
    assert calls["mbar_arrive_remote"] == "tfree"
    assert len(re.findall(r"\bmbar_arrive_remote\(", kernel)) == 1
    for name in set(calls) - {"mbar_arrive_remote"}:
        body = re.search(r"void %s\(uint32_t bar\) \{(.*?)\n\}" % name, helpers, re.S).group(1)
        fence, arrive = body.find("fence.release.sync_restrict::shared::cta.cluster"), body.find("mbarrier.arrive.")
        assert 0 <= fence < arrive, f"{name} releases nothing"
