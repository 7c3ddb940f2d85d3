"""The residual norm over the whole range of its operands: rows whose squares, or their sum, leave fp32."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests.test_gpu_add_norm import same  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    return mr


def sized(e, K, gen):
    """K values of random sign and mantissa in [2^e, 2^(e + 1))."""
    v = torch.ldexp(1 + torch.rand(K, generator=gen, dtype=torch.float64) * 0.99, torch.tensor(e))
    return torch.where(torch.rand(K, generator=gen) < 0.5, -v, v).to(BF16)


def ends(K, seed=1):
    """Rows of every size up to that whose squares leave fp32: evenly sized ones, one value among zeros, and sizes mixed
    over the whole range below."""
    gen = torch.Generator("cpu").manual_seed(seed)
    rows = []
    for e in [*range(-133, -58, 3), -40, -30, -29, -1, 0, 30, 50, *range(54, 64)]:
        rows.append(sized(e, K, gen))
        one = torch.zeros(K, dtype=BF16)
        one[(e * 37) % K] = rows[-1][0]
        rows.append(one)
        rows.append((rows[0].double() * torch.ldexp(torch.ones(K, dtype=torch.float64),
                                                    torch.randint(0, e + 134, (K,), generator=gen))).to(BF16))
    rows.append(torch.zeros(K, dtype=BF16))
    return torch.stack(rows).cuda()


def check_rstd(got, sres, eps):
    """Rounded once: half a step, and 2^-19 of one for the second-order term of the root's correction (a first root off
    by 2 units in the last place: 3/8 (2^-21)^2) and what the sum is short of.  Beyond fp32: infinity.
    A value whose own square is beyond fp32, from 2^64 on (the mixed rows reach it), makes it 0."""
    want = ref.rstd64(sres, torch.tensor(eps, dtype=torch.float32, device="cuda").double())  # (eps is an fp32 number)
    want[(sres.abs() >= 2.0 ** 64).any(1)] = 0
    _, e = torch.frexp(want)
    step = torch.ldexp(torch.ones_like(want), e - 24)
    beyond = want >= 2.0 ** 128 - 2.0 ** 103
    assert torch.isinf(got[beyond]).all()
    err = ((got.double() - want).abs() / step)[~beyond]
    assert not err.isnan().any() and err.max() <= 0.5 + 2.0 ** -18, (err.max().item(), int(err.argmax()))


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 1e-40, 2.0 ** -61, 2.0 ** -59, 1e-6, 1.0, 3e38])
@pytest.mark.parametrize("K,many", [(256, False), (256, True), (1040, False), (4096, True), (6144, False), (6144, True),
                                    (8192, True), (12288, True), (16384, True), (8208, False), (16400, False),
                                    (65536, False)])
def test_rows_of_every_size(mr, K, many, eps):
    x, g = ends(K), (0.2 * ref.rows(3, 1, K)[0].float()).to(BF16)
    if many:
        x = x.repeat(5, 1)  # (more than two rows an SM: another variant)
    out = mr.add_rms_norm(x, None, g, eps, "rms", "fp8", outputs=("sres", "rstd", "xn"))
    assert same(out["sres"], x)
    check_rstd(out["rstd"], x, eps)
    assert same(out["xn"], ref.normed(x, out["rstd"], g, "rms"))
    q, s = mr.fp8_quant(out["xn"])
    assert same(out["q"], q) and same(out["scale"], s)


@pytest.mark.parametrize("M", [3, 400])
def test_residual_that_leaves_little_or_much(mr, M):
    """The size that counts is the sum's."""
    K = 6144
    g = torch.zeros(K, dtype=BF16, device="cuda")
    x = torch.ones(M, K, device="cuda").to(BF16)
    res = (-x.float() + 2.0 ** -8).to(BF16)
    res[1] = 3e17
    res[2] = -1
    for eps in (0.0, 1e-6):
        out = mr.add_rms_norm(x, res, g, eps, "gemma", "mxfp8", outputs=("sres", "rstd", "xn"))
        sres = (x.float() + res.float()).to(BF16)
        check_rstd(out["rstd"], sres, eps)
        assert same(out["xn"], ref.normed(sres, out["rstd"], g, "gemma"))
        assert (out["xn"][1] == 1).all()


def test_squares_beyond_fp32(mr):
    """From 2^64 on a value's square is beyond fp32 and makes its row's rstd 0, an infinity too; a NaN stays one."""
    K = 2048
    for M in (7, 700):
        x = ref.rows(1, M, K)
        x[1, 5] = 2.0 ** 64
        x[2] = 3e38
        x[3, K - 1] = float("-inf")
        x[4, 0], x[4, 9] = float("nan"), float("inf")
        x[5, 5] = 2.0 ** 64 * (1 - 2.0 ** -8)
        out = mr.add_rms_norm(x, None, torch.zeros(K, dtype=BF16, device="cuda"), 0.0, outputs=("rstd", "xn"))
        r = out["rstd"]
        assert (r[1:4] == 0).all() and r[4].isnan()
        ok = torch.tensor([0, 5, *range(6, M)], device="cuda")
        check_rstd(r[ok], x[ok], 0.0)
