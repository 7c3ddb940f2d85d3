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


# ------------------------------------------------------------------ NaN and infinity stay where they belong

def moe(mr, fmt, M, E, topk, K, I, block):
    from tests.test_gpu_experts import routed
    ids, wts = routed(M, E, topk, M + E)
    st, ex, _ = mr.moe_sort(ids, E, block)
    return (ids, wts, st, ex, ref.random_mx((M, K), fmt, 1), ref.random_mx((E, 2 * I, K), fmt, 2, 112, 116),
            ref.random_mx((st.numel(), I), fmt, 3), ref.random_mx((E, K, I), fmt, 4, 112, 116))


SIZES = [(6, 4, 2, 256, 64, 16), (1, 8, 2, 6144, 32, 16), (300, 3, 2, 416, 96, 64), (40, 2, 1, 5152, 32, 8)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,K,I,block", SIZES)
def test_gate_up_nan_stays_in_its_row_and_feature(mr, fmt, M, E, topk, K, I, block):
    """NaN by the scale byte and by the code of a token's element, and by a weight's scale: those results and no
    others; quantised results are the quantiser's of the bf16 rows; sorted rows beside NaN padding."""
    ids, _, st, ex, x, w13, _, _ = moe(mr, fmt, M, E, topk, K, I, block)
    mk = M * topk
    real = st < mk
    clean = mr.moe_gate_up(*x, mr.MxWeight(*w13, fmt, gate_up=True), st, ex, topk, block)
    assert not clean[real].isnan().any()
    bad = [M // 2]
    x[1][M // 2, K // 32 - 1] = 255
    if fmt == "mxfp8":
        x[0][M - 1, 5] = 0xFF
        bad.append(M - 1)
    e, feature = int(ids[0, 0]), 17
    w13[1][e, I + feature, 0] = 255
    W = mr.MxWeight(*w13, fmt, gate_up=True)
    token = (st.long() // topk).clamp(max=M - 1)
    nan = torch.zeros_like(clean, dtype=torch.bool)
    for m in bad:
        nan[real & (token == m)] = True
    nan[real & (ex.repeat_interleave(block)[:st.numel()] == e), feature] = True
    out = mr.moe_gate_up(*x, W, st, ex, topk, block)
    assert out[nan].isnan().all()
    rest = real[:, None] & ~nan
    assert torch.equal(out[rest], clean[rest])
    for qf in FMTS:
        c, s = mr.moe_gate_up(*x, W, st, ex, topk, block, quant=qf)
        rc, rs = (mr.mxfp8_quant if qf == "mxfp8" else mr.mxfp4_quant)(torch.where(real[:, None], out, 0))
        assert torch.equal(c[real], rc[real]) and torch.equal(s[real], rs[real]), qf
    # rows at the sorted positions: the padding's are NaN
    qs, ss = x[0][token].masked_fill(~real[:, None], 255), x[1][token].masked_fill(~real[:, None], 255)
    out2 = mr.moe_gate_up(qs, ss, W, st, ex, topk, block, num_tokens=M, sorted_rows=True)
    assert torch.equal(out2[real].view(torch.int16), out[real].view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,K,I,block", SIZES)
def test_down_nan_stays_in_its_token_and_column(mr, fmt, M, E, topk, K, I, block):
    ids, wts, st, ex, _, _, a, w2 = moe(mr, fmt, M, E, topk, K, I, block)
    real = st < M * topk
    # rows that hold no assignment may be anything
    q, s = a[0].masked_fill(~real[:, None], 255), a[1].masked_fill(~real[:, None], 255)
    W = mr.MxWeight(*w2, fmt)
    for fp32 in (False, True):
        clean = mr.moe_down(*a, W, ids, wts, st, ex, block, slots_fp32=fp32)
        assert not clean.isnan().any()
        assert torch.equal(mr.moe_down(q, s, W, ids, wts, st, ex, block, slots_fp32=fp32), clean)
    pos, f = ref.used_positions(st, M * topk)
    p, token = int(pos[-1]), int(f[-1]) // topk
    s[p, I // 32 - 1] = 255
    e, column = int(ids[0, topk - 1]), K - 3
    w2[1][e, column, 0] = 255
    W = mr.MxWeight(*w2, fmt)
    nan = torch.zeros_like(clean, dtype=torch.bool)
    nan[token] = True
    nan[(ids == e).any(1), column] = True
    for fp32 in (False, True):
        clean = mr.moe_down(*a, mr.MxWeight(w2[0], w2[1].masked_fill(w2[1] == 255, 112), fmt), ids, wts, st, ex, block,
                            slots_fp32=fp32)
        out = mr.moe_down(q, s, W, ids, wts, st, ex, block, slots_fp32=fp32)
        assert out[nan].isnan().all()
        assert torch.equal(out[~nan], clean[~nan])


@pytest.mark.parametrize("fmt", FMTS)
def test_sums_past_the_largest_number_are_infinite(mr, fmt):
    """Products of one element: past fp32 and past bf16's rounding (its largest is 2^128 - 2^120)."""
    M, R, K = 3, 130, 64
    x = torch.zeros(M, K if fmt == "mxfp8" else K // 2, dtype=torch.uint8)
    w = torch.zeros(R, x.shape[1], dtype=torch.uint8)
    xs, ws = torch.full((M, 2), 127, dtype=torch.uint8), torch.full((R, 2), 127, dtype=torch.uint8)
    minus = 0x80 if fmt == "mxfp8" else 8
    for m in range(M):
        put(x, fmt, m, 0, ONE[fmt] | (minus if m == 1 else 0))
    xs[:2, 0] = 127 + 120
    for r in (4, 129):
        put(w, fmt, r, 0, ONE[fmt])
        ws[r, 0] = 127 + 9
    x, xs, w, ws = (t.cuda() for t in (x, xs, w, ws))
    W = mr.MxWeight(w, ws, fmt)
    for dtype in (torch.float32, BF16):
        out = mr.mx_gemm(x, xs, W, out_dtype=dtype)
        want = torch.zeros(M, R, device="cuda")
        want[0, 4] = want[0, 129] = float("inf")
        want[1, 4] = want[1, 129] = -float("inf")
        want[2, 4] = want[2, 129] = 512.0
        assert torch.equal(out.float(), want), dtype
    # an infinite gate, up value and slot
    I = 32
    w13 = torch.zeros(1, 2 * I, x.shape[1], dtype=torch.uint8, device="cuda")
    s13 = torch.full((1, 2 * I, 2), 127, dtype=torch.uint8, device="cuda")
    for i in range(I):
        put(w13[0], fmt, i, 0, ONE[fmt])
        put(w13[0], fmt, I + i, 0, ONE[fmt])
    s13[0, 3, 0] = s13[0, I + 5, 0] = 127 + 9
    ids = torch.zeros(M, 1, dtype=torch.int32, device="cuda")
    st, ex, _ = mr.moe_sort(ids, 1, 16)
    xs[:2, 0] = 127 + 120
    xs[0, 0] = 127  # token 0: 1, token 1: -2^120, token 2: 1
    out = mr.moe_gate_up(x, xs, mr.MxWeight(w13, s13, fmt, gate_up=True), st, ex, 1, 16)[:M].float()
    one = torch.sigmoid(torch.ones(1, dtype=torch.float64)).item()
    want = torch.full((M, I), one, dtype=torch.float64, device="cuda")
    want[:, 3], want[:, 5] = 512.0, one * 512
    keep = torch.tensor([0, 2], device="cuda")
    ref.assert_close(out[keep], want[keep], 2.0 ** -8 * want[keep] * 1.01)
    assert (out[1, [c for c in range(I) if c not in (3, 5)]] == 0).all()  # silu(-2^120) is 0, times -2^120
    assert out[1, 3].isnan() and out[1, 5].isnan()  # -inf / inf and 0 times infinity, as the formula has it
