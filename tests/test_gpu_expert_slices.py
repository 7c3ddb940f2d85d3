"""Products of few tiles, whose K range several CTAs share, on operands whose
every sum is exact in fp32: a slice's border that is off by one block, or a
slice added twice, shows as a wrong number."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_expert_pairs import exact_mx, exact_product  # noqa: E402
from tests.test_gpu_experts import mr, routed  # noqa: E402, F401

FMTS = ["mxfp8", "mxfp4"]
BF16 = torch.bfloat16


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,R,K", [
    (1, 1, 16416), (1, 128, 6144), (64, 500, 4128), (64, 500, 6144), (129, 130, 12320), (33, 6144, 6144), (250, 300, 2976),
    (256, 100, 20480), (600, 200, 8192), (895, 1420, 4736), (17, 64, 2592)])
def test_products(mr, fmt, M, R, K):
    x, w = exact_mx((M, K), fmt, M), exact_mx((R, K), fmt, R)
    want = exact_product(ref.value64(*x, fmt), ref.value64(*w, fmt))
    assert torch.equal(mr.mx_gemm(*x, mr.MxWeight(*w, fmt), out_dtype=torch.float32).double(), want)


EXPERTS = [(1, 8, 2, 6144, 64, 16), (5, 4, 2, 4128, 96, 16), (40, 2, 2, 5152, 32, 8), (130, 3, 1, 12320, 160, 64),
           (3, 1, 1, 8192, 32, 1), (300, 1, 1, 6176, 64, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,K,I,block", EXPERTS)
def test_gate_up(mr, fmt, M, E, topk, K, I, block):
    """h is exact: what remains is SwiGLU's own error.  The scales take h to some units, where silu is no constant."""
    ids, _ = routed(M, E, topk, M + K)
    st, ex, _ = mr.moe_sort(ids, E, block)
    x, w = exact_mx((M, K), fmt, 1), exact_mx((E, 2 * I, K), fmt, 2)
    xv, wv = ref.value64(*x, fmt), ref.value64(*w, fmt)
    w = w[0], w[1] - 9
    real = st < M * topk
    pos, f = ref.used_positions(st, M * topk)
    h = torch.stack([exact_product(xv[t][None], wv[e])[0] for t, e in
                     zip((f // topk).tolist(), ex[pos // block].tolist())]) * 2.0 ** -9
    g, u = h[:, :I], h[:, I:]
    want = g * torch.sigmoid(g) * u
    out = mr.moe_gate_up(*x, mr.MxWeight(*w, fmt, gate_up=True), st, ex, topk, block)
    tol = 8 * 2.0 ** -23 * want.abs()
    ref.assert_close(out[pos], want, tol + ref.half_step(BF16) * (want.abs() + tol) + 2.0 ** -133)
    q, s = x[0][st[real].long() // topk], x[1][st[real].long() // topk]
    qs, ss = torch.zeros(st.numel(), q.shape[1], dtype=torch.uint8, device="cuda"), torch.full(
        (st.numel(), s.shape[1]), 255, dtype=torch.uint8, device="cuda")
    qs[real], ss[real] = q, s
    out2 = mr.moe_gate_up(qs, ss, mr.MxWeight(*w, fmt, gate_up=True), st, ex, topk, block, num_tokens=M,
                          sorted_rows=True)
    assert torch.equal(out[real], out2[real])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,I,R,block", EXPERTS)
def test_down(mr, fmt, M, E, topk, I, R, block):
    """Routing weights of 1, 2 and 4 and unrounded slots: the sum over slots is exact too."""
    ids, _ = routed(M, E, topk, M + I)
    wts = 2.0 ** torch.randint(0, 3, (M, topk), generator=torch.Generator("cpu").manual_seed(I)).float().cuda()
    st, ex, _ = mr.moe_sort(ids, E, block)
    a, w = exact_mx((st.numel(), I), fmt, 1), exact_mx((E, R, I), fmt, 2)
    av, wv = ref.value64(*a, fmt), ref.value64(*w, fmt)
    pos, f = ref.used_positions(st, M * topk)
    y = torch.zeros(M * topk, R, dtype=torch.float64, device="cuda")
    for p, i, e in zip(pos.tolist(), f.tolist(), ex[pos // block].tolist()):
        y[i] = exact_product(av[p][None], wv[e])[0]
    y = y.unflatten(0, (M, topk)) * wts.double()[..., None]
    assert y.abs().sum(1).max() * 4 < 1 << 24
    out = mr.moe_down(*a, mr.MxWeight(*w, fmt), ids, wts, st, ex, block, slots_fp32=True)
    assert torch.equal(out, y.sum(1).to(BF16))
