"""moe_down's rounding of the slots' rows: with it within its bound, without
it (slots_fp32) against the definition with the one rounding of the result."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_experts import mr, routed  # noqa: E402, F401

FMTS = ["mxfp8", "mxfp4"]
BF16 = torch.bfloat16
HALF = ref.half_step(BF16)


def definition(a, w2, st, ex, ids, wts, block, add):
    """(out, bound before its rounding, sum |w y|) of the formula without y's rounding, in 64 bits."""
    M, topk = ids.shape
    E, R, _ = w2.shape
    y = torch.zeros(M * topk, R, dtype=torch.float64, device=a.device)
    d = torch.zeros_like(y)
    pos, f = ref.used_positions(st, M * topk)
    e = ex[pos // block].long()
    for k in e.unique().tolist():
        m = e == k
        rows = a[pos[m]]
        y[f[m]] = rows @ w2[k].T
        d[f[m]] = ref.sum_bound(rows.shape[1]) * (rows.abs() @ w2[k].abs().T)
    used = ((ids >= 0) & (ids < E))[..., None]
    w = torch.where(used, wts.double()[..., None], 0.0)
    y, d = y.unflatten(0, (M, topk)), d.unflatten(0, (M, topk))
    out, mag = (w * y).sum(1), (w * y).abs().sum(1)
    if add is not None:
        out = out + add.double()
    # every fp32 addition and product is off by half a step of a partial sum
    tol = (w.abs() * d).sum(1) + (topk + 1) * 2.0 ** -24 * (mag + (0 if add is None else add.double().abs()))
    return out, tol, mag


SHAPES = [  # M, E, topk, R, I, block, share of slots without an expert, skew
    (1, 8, 2, 128, 32, 16, 0.0, 0), (1, 1, 1, 1, 32, 1, 0.0, 0), (7, 16, 4, 256, 64, 16, 0.3, 0),
    (33, 5, 3, 33, 160, 8, 0.3, 1), (64, 8, 8, 1032, 64, 32, 0.0, 0), (300, 2, 2, 130, 128, 64, 0.0, 0),
    (513, 9, 3, 288, 64, 64, 0.05, 2), (40, 1024, 16, 96, 32, 16, 0.0, 0), (20, 6, 4, 1000, 6176, 16, 0.1, 0),
    (70, 40, 32, 64, 64, 16, 0.1, 0),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,R,I,block,invalid,skew", SHAPES)
def test_unrounded_slots(mr, fmt, M, E, topk, R, I, block, invalid, skew):
    ids, wts = routed(M, E, topk, M + E, invalid, skew)
    st, ex, _ = mr.moe_sort(ids, E, block)
    w = ref.random_mx((E, R, I), fmt, I, 117, 122)
    a = ref.random_mx((st.numel(), I), fmt, R)
    add = torch.randn(M, R, generator=torch.Generator("cpu").manual_seed(R)).to(BF16).cuda()
    W = mr.MxWeight(*w, fmt)
    av, wv = ref.value64(*a, fmt), ref.value64(*w, fmt)
    scratch = mr.ExpertScratch(M, topk, R, slots_fp32=True)
    for extra in (None, add):
        want, tol, mag = definition(av, wv, st, ex, ids, wts, block, extra)
        out = mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra, scratch=scratch, slots_fp32=True)
        ref.assert_close(out, want, tol + HALF * (want.abs() + tol), "unrounded")
        assert torch.equal(out, mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra, slots_fp32=True))
        # what a call of this size does by itself
        assert torch.equal(out, mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra))
        # the rounded form: 2^-8 of every slot more
        tol = tol + HALF * (mag + tol)
        out2 = mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra, scratch=scratch, slots_fp32=False)
        ref.assert_close(out2, want, tol + HALF * (want.abs() + tol), "rounded")
    inplace = add.clone()
    mr.moe_down(*a, W, ids, wts, st, ex, block, add=inplace, out=inplace, scratch=scratch, slots_fp32=True)
    assert torch.equal(inplace, out)


@pytest.mark.parametrize("fmt", FMTS)
def test_slots_that_cancel(mr, fmt):
    """Two experts that differ in a thousandth, weighted 1 and -1 (and a sum that add takes away): the result is the
    difference, with a relative error like any other's when slots are not rounded."""
    M, E, topk, R, I, block = 40, 2, 2, 200, 64, 16
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(M, 1)
    wts = torch.tensor([[1.0, -1.0]], device="cuda").repeat(M, 1)
    st, ex, _ = mr.moe_sort(ids, E, block)
    # elements of one size, so that no product is lost in its sum: 1 or 1.5 in block 0, the same 2^-10 times in block 1
    g = torch.Generator("cpu").manual_seed(1)
    one, more = (0x38, 0x3C) if fmt == "mxfp8" else (2, 3)

    def codes(*shape):
        c = torch.where(torch.rand(*shape, generator=g) < 0.5, one, more).to(torch.uint8)
        return c if fmt == "mxfp8" else c[..., 0::2] | (c[..., 1::2] << 4)

    rows = codes(M, I).cuda()
    pos, f = ref.used_positions(st, M * topk)
    a = torch.zeros(st.numel(), rows.shape[1], dtype=torch.uint8, device="cuda")
    a[pos] = rows[f // topk]
    a_scale = torch.full((st.numel(), 2), 127, dtype=torch.uint8, device="cuda")
    w = codes(1, R, I).repeat(2, 1, 1)
    w[1, :, w.shape[2] // 2:] = codes(R, I)[:, w.shape[2] // 2:]
    w_scale = torch.full((2, R, 2), 127, dtype=torch.uint8)
    w_scale[:, :, 1] = 117
    w, w_scale = w.cuda(), w_scale.cuda()
    W = mr.MxWeight(w, w_scale, fmt)
    want, tol, mag = definition(ref.value64(a, a_scale, fmt), ref.value64(w, w_scale, fmt), st, ex, ids, wts, block, None)
    assert want.abs().max() < mag.min() * 2.0 ** -9 and (want != 0).any()
    out = mr.moe_down(a, a_scale, W, ids, wts, st, ex, block, slots_fp32=True)
    # every sum here is of at most 64 terms in units of 2^-12 below 2^8: exact in fp32
    assert torch.equal(out, want.to(BF16))
    rounded = mr.moe_down(a, a_scale, W, ids, wts, st, ex, block, slots_fp32=False)
    ref.assert_close(rounded, want, HALF * mag + HALF * (want.abs() + HALF * mag))
    assert not torch.equal(rounded, out)
    # add takes the first slot away
    wts = torch.tensor([[1.0, 0.0]], device="cuda").repeat(M, 1)
    whole, _, _ = definition(ref.value64(a, a_scale, fmt), ref.value64(w, w_scale, fmt), st, ex, ids, wts, block, None)
    add = (-whole).to(BF16)
    out = mr.moe_down(a, a_scale, W, ids, wts, st, ex, block, add=add, slots_fp32=True)
    assert torch.equal(out, (whole + add.double()).to(BF16))


def test_unrounded_slots_touch_their_own_scratch_only(mr):
    M, E, topk, I, block = 19, 8, 3, 256, 16
    ids, wts = routed(M, E, topk, 3, invalid=0.2)
    st, ex, _ = mr.moe_sort(ids, E, block)
    for R in (32, 64, 1032, 130):
        a, W = ref.random_mx((st.numel(), I), "mxfp4", 1), mr.MxWeight(*ref.random_mx((E, R, I), "mxfp4", 2), "mxfp4")
        want = mr.moe_down(*a, W, ids, wts, st, ex, block, slots_fp32=True)
        scratch = mr.ExpertScratch(2 * M, topk, R, slots_fp32=True)
        rest = [t[M * topk * R * 2:] for t in (scratch.tensor, scratch.low)]
        call = mr.PreparedDown(*a, W, ids, wts, st, ex, block, scratch=scratch, slots_fp32=True)
        for i in range(10):
            for t in rest:
                t.fill_(i)
            assert torch.equal(call(), want)
            assert all((t == i).all() for t in rest)


def test_scratch_of_either_kind(mr, monkeypatch):
    """A scratch without the lower halves' room, or with room for a few, is refused where it is needed; calls past the
    limit round unless they are told not to."""
    M, E, topk, R, I, block = 19, 8, 3, 128, 64, 16
    ids, wts = routed(M, E, topk, 3)
    st, ex, _ = mr.moe_sort(ids, E, block)
    a, W = ref.random_mx((st.numel(), I), "mxfp8", 1), mr.MxWeight(*ref.random_mx((E, R, I), "mxfp8", 2))

    def run(**kw):
        return mr.moe_down(*a, W, ids, wts, st, ex, block, **kw)

    whole, rounded = run(slots_fp32=True), run(slots_fp32=False)
    assert not torch.equal(whole, rounded)
    plain = mr.ExpertScratch(M, topk, R, slots_fp32=False)
    assert plain.low is None and torch.equal(run(scratch=plain, slots_fp32=False), rounded)
    assert torch.equal(run(scratch=plain), rounded)
    with pytest.raises(ValueError):
        run(scratch=plain, slots_fp32=True)
    assert torch.equal(run(scratch=mr.ExpertScratch(M, topk, R)), whole)
    monkeypatch.setattr(mr, "SLOTS_FP32_MAX", M * topk * R - 1)
    assert torch.equal(run(), rounded) and torch.equal(run(scratch=mr.ExpertScratch(M, topk, R)), rounded)
    assert torch.equal(run(slots_fp32=True), whole)
    with pytest.raises(mr.MoeRouteError) as e:
        run(scratch=mr.ExpertScratch(M, topk, R), slots_fp32=True)
    assert e.value.status == mr.MR_ERR_SCRATCH_TOO_SMALL
    # a scratch for more tokens than the limit serves the few that are kept whole
    monkeypatch.setattr(mr, "SLOTS_FP32_MAX", M * topk * R)
    big = mr.ExpertScratch(4 * M, topk, R)
    assert big.low_nbytes == 2 * M * topk * R and torch.equal(run(scratch=big), whole)
