"""Products whose every sum is exact in fp32, so that a misplaced, missing or
stale element, scale or slice shows as a wrong number."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_experts import mr  # noqa: E402, F401

FMTS = ["mxfp8", "mxfp4"]


def exact_mx(shape, fmt, seed):
    """Codes of up to 3 bits and scales of 1 and 2: products are multiples of 1/4 below 2^8."""
    codes, scale = ref.random_mx(shape, fmt, seed, 127, 129)
    if fmt == "mxfp8":  # 0, 1, 1.5, 2, 3, 4, 6, 8 and their negatives
        lut = torch.tensor([0x00, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C, 0x50], dtype=torch.uint8, device="cuda")
        codes = lut[(codes & 7).long()] | (codes & 128)
    return codes, scale


def exact_product(x, w):
    """x @ w^T in 64 bits; any order of summation in fp32 gives the same: multiples of 1/4, 24 bits at most."""
    assert (x.abs() @ w.abs().T).max() * 4 < 1 << 24
    return x @ w.T


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,R,K", [(64, 2000, 2048), (150, 4000, 1056), (300, 1000, 8192), (700, 6144, 768)])
def test_pairs_are_exact_time_after_time(mr, fmt, M, R, K):
    """Two CTAs to a tile; new operands in the same buffers for each call."""
    x, w = exact_mx((M, K), fmt, 1), exact_mx((R, K), fmt, 2)
    W = mr.MxWeight(*w, fmt)
    gemm = mr.PreparedMxGemm(*x, W, out_dtype=torch.float32)
    wv = ref.value64(*w, fmt)
    for seed in range(5):
        y = exact_mx((M, K), fmt, 10 + seed)
        x[0].copy_(y[0])
        x[1].copy_(y[1])
        want = exact_product(ref.value64(*x, fmt), wv)
        for _ in range(5):
            gemm.out.zero_()
            assert torch.equal(gemm().double(), want)
