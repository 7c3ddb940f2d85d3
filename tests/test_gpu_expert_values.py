"""moe_gate_up, moe_down and mx_gemm on values at the ends of their ranges."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_experts import mr  # noqa: E402, F401

FMTS = ["mxfp8", "mxfp4"]
BF16 = torch.bfloat16
ONE = {"mxfp8": 0x38, "mxfp4": 2}


def put(codes, fmt, row, k, code):
    """Element k of a row of codes."""
    if fmt == "mxfp8":
        codes[row, k] = code
    else:
        b = int(codes[row, k // 2])
        codes[row, k // 2] = (b & 0xF0) | code if k % 2 == 0 else (b & 0x0F) | (code << 4)


@pytest.mark.parametrize("fmt", FMTS)
def test_silu_of_very_negative_gates(mr, fmt):
    """silu(g) down to where e^g has a handful of bits, times up values that bring it back: products of single
    elements, so that g and u are exact.  Gates (-88, -80, ...) + 0, 0.5, ... 1.5 around -87.3 (e^-g past 2^126) and
    -88.7 (past fp32)."""
    I, K = 32, 64
    codes = torch.zeros(2 * I, K if fmt == "mxfp8" else K // 2, dtype=torch.uint8)
    scale = torch.full((2 * I, 2), 127, dtype=torch.uint8)
    scale[:I, 0] = 127 + 4  # gates: 16 times the sum of two elements, and one element as it is
    # in 16ths: 5.5, 5, 5.75, 6, 6.5, 3, 1, 0.5 as a sum of two codes' values
    sums = [(4.0, 1.5), (4.0, 1.0), (6.0, 0.0), (6.0, 0.5), (3.0, 0.0), (1.0, 0.0), (0.5, 0.0), (0.0, 0.0)]
    bits8 = {0.0: 0x00, 0.5: 0x30, 1.0: 0x38, 1.5: 0x3C, 3.0: 0x44, 4.0: 0x48, 6.0: 0x4C}
    bits4 = {0.0: 0, 0.5: 1, 1.0: 2, 1.5: 3, 3.0: 5, 4.0: 6, 6.0: 7}
    bits, minus = (bits8, 0x80) if fmt == "mxfp8" else (bits4, 8)
    for i in range(I):
        a, b = sums[i // 4]
        put(codes, fmt, i, 0, bits[a] | minus)
        put(codes, fmt, i, 1, bits[b] | minus)
        put(codes, fmt, i, 32, bits[[0.0, 0.5, 1.0, 1.5][i % 4]])
        put(codes, fmt, I + i, 0, ONE[fmt])
        scale[I + i, 0] = 127 + (110, 100, 90, 0)[i % 4]
    x = torch.zeros(1, codes.shape[1], dtype=torch.uint8)
    for k in (0, 1, 32):
        put(x, fmt, 0, k, ONE[fmt])
    xs = torch.full((1, 2), 127, dtype=torch.uint8)
    x, xs, codes, scale = (t.cuda() for t in (x, xs, codes, scale))
    ids = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    st, ex, _ = mr.moe_sort(ids, 1, 16)
    out = mr.moe_gate_up(x, xs, mr.MxWeight(codes[None], scale[None], fmt, gate_up=True), st, ex, 1, 16)[0]
    h = ref.value64(x, xs, fmt) @ ref.value64(codes, scale, fmt).T
    g, u = h[0, :I], h[0, I:]
    assert g.min() == -104 and ((g < -87.3) & (g > -88.7)).any()
    want = g * torch.sigmoid(g) * u
    # e^-|g| is good to 2 ulps (of 2^-149 where it is subnormal), g e^g and the quotient to as many steps
    tol = 8 * 2.0 ** -23 * want.abs() + (2 * g.abs() + 3) * u.abs() * 2.0 ** -149
    half = ref.half_step(BF16)
    ref.assert_close(out, want, tol + half * (want.abs() + tol) + 2.0 ** -133)
    assert (out[(g < 0) & (g > -102) & (want.abs() > 2.0 ** -120)] != 0).all()
