"""Stream order of the expert products' calls and of the memory they make."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_experts import mr, quant, routed  # noqa: E402, F401

BF16 = torch.bfloat16


def _rows(seed, m, k):
    return torch.randn(m, k, generator=torch.Generator("cpu").manual_seed(seed)).to(BF16).cuda()


def _with_flags(mr, flags, run, times):
    mr.set_launch_flags(flags)
    try:
        out = [run() for _ in range(times)]
        torch.cuda.synchronize()
        return out
    finally:
        mr.set_launch_flags(0)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_scales_are_laid_out_in_stream_order(mr, fmt):
    """Under MR_LAUNCH_PDL: a weight quantised just before its scales are laid
    out, products just before and after they are laid out again, and a product
    of the call before the layout."""
    M, R, K = 300, 4096, 2048
    w, w2 = _rows(1, R, K), _rows(2, R, K) * 8
    x = quant(mr, _rows(3, M, K), fmt)
    E, topk, I, block = 4, 2, 512, 64
    ids, wts = routed(M, E, topk, 1)
    st, ex, _ = mr.moe_sort(ids, E, block)
    w13 = mr.MxWeight(*ref.random_mx((E, 2 * I, K), fmt, 6, 112, 116), fmt, gate_up=True)
    down = mr.MxWeight(*ref.random_mx((E, K, I), fmt, 7, 112, 116), fmt)
    torch.cuda.synchronize()

    def run():
        codes, scale = quant(mr, w, fmt)
        W = mr.MxWeight(codes, scale, fmt)  # (scale is being written by the kernel before)
        first = mr.mx_gemm(*x, W)
        W.scale = quant(mr, w2, fmt)[1]
        again = mr.mx_gemm(*x, W)
        W.refresh()  # (the product before still reads the scales as they were)
        last = mr.mx_gemm(*x, W)
        act = mr.moe_gate_up(*x, w13, st, ex, topk, block, quant=fmt)
        W.refresh()
        out = mr.moe_down(*act, down, ids, wts, st, ex, block)
        return first, again, last, out

    want = _with_flags(mr, 0, run, 1)[0]
    assert torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2])
    for got in _with_flags(mr, mr.LAUNCH_PDL, run, 20):
        for g, o in zip(got, want):
            assert torch.equal(g, o)
