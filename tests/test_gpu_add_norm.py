"""The residual norm and the FP8 quantiser on the GPU, against their formulas."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    return mr


def same(a, b):
    """Equal bit for bit (a NaN equals a NaN)."""
    if a.dtype == torch.float32:
        return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
    if a.dtype == BF16:
        return same(a.float(), b.float())
    return torch.equal(a, b)


def check(mr, out, x, res, g, eps, norm, quant):
    sres = x if res is None else (x.float() + res.float()).to(BF16)
    assert same(out["sres"], sres)
    want = ref.rstd64(sres, eps)
    # rounded once: half a step, and 2^-20 of one for what the sum and the root are short of
    _, e = torch.frexp(want)
    step = torch.ldexp(torch.ones_like(want), e - 24)
    assert ((out["rstd"].double() - want).abs() <= step * (0.5 + 2.0 ** -20)).all()
    xn = ref.normed(sres, out["rstd"], g, norm)
    assert same(out["xn"], xn)
    assert same(out["xn"], mr.norm_apply(out["sres"].contiguous(), out["rstd"], g, norm))
    if quant is not None:
        q, s = {"mxfp8": mr.mxfp8_quant, "mxfp4": mr.mxfp4_quant, "fp8": mr.fp8_quant}[quant](xn)
        assert same(out["q"], q) and same(out["scale"], s)


@pytest.mark.parametrize("M,K,quant", [
    (1, 6144, "fp8"), (1, 8, None), (3, 16, "fp8"), (2, 32, "mxfp4"), (5, 2976, "fp8"), (5, 2976, "mxfp8"),
    (7, 1000, None), (33, 1008, "fp8"), (64, 3584, "mxfp4"), (17, 8192, "fp8"), (3, 8200, None), (4, 8224, "mxfp8"),
    (2, 16400, "fp8"), (2, 33024, "fp8"), (1, 65536, "mxfp8"), (2, 65520, "fp8"), (300, 256, "mxfp8"),
    (1000, 144, "fp8"), (2000, 6144, "fp8")])
@pytest.mark.parametrize("norm,with_res", [("gemma", True), ("rms", False)])
def test_values(mr, M, K, quant, norm, with_res):
    x, g = ref.rows(M + K, M, K), (0.2 * ref.rows(3, 1, K)[0].float()).to(BF16)
    res = ref.rows(5, M, K) * 3 if with_res else None
    names = ["sres", "rstd", "xn"]
    out = mr.add_rms_norm(x, res, g, 1e-6, norm, quant, outputs=names)
    assert set(out) == set(names) | ({"q", "scale"} if quant else set())
    check(mr, out, x, res, g, 1e-6, norm, quant)


@pytest.mark.parametrize("where", ["x", "residual", "strided"])
def test_strides_and_sums_in_place(mr, where):
    M, K = 9, 1040
    wide = torch.full((M, 2 * K + 16), 7.0, dtype=BF16, device="cuda")
    x, res = wide[:, 8:8 + K], ref.rows(2, M, K)
    x.copy_(ref.rows(1, M, K))
    x0, res0, g = x.clone(), res.clone(), ref.rows(3, 1, K)[0]
    sres = {"x": x, "residual": res, "strided": wide[:, K + 16:]}[where]
    out = mr.add_rms_norm(x, res, g, 1e-5, "gemma", "fp8", outputs=("rstd", "xn"), out=dict(sres=sres))
    assert out["sres"] is sres
    check(mr, out, x0, res0, g, 1e-5, "gemma", "fp8")
    untouched = wide.clone()
    untouched[:, 8:8 + K] = 7
    untouched[:, K + 16:] = 7
    assert (untouched == 7).all()


def test_each_output_alone(mr):
    x, res, g = ref.rows(1, 6, 512), ref.rows(2, 6, 512), ref.rows(3, 1, 512)[0]
    full = mr.add_rms_norm(x, res, g, quant="fp8", outputs=("sres", "rstd", "xn"))
    for name in ("sres", "rstd", "xn"):
        one = mr.add_rms_norm(x, res, g, outputs=(name,))
        assert list(one) == [name] and same(one[name], full[name])
    codes = mr.add_rms_norm(x, res, g, quant="fp8", outputs=())
    assert set(codes) == {"q", "scale"} and same(codes["q"], full["q"]) and same(codes["scale"], full["scale"])
    assert set(mr.add_rms_norm(x, res, g)) == {"sres", "rstd", "xn"}
    assert set(mr.add_rms_norm(x, res, g, quant="mxfp8")) == {"sres", "rstd", "q", "scale"}


def test_values_at_the_ends_of_the_range(mr):
    """Zeros with and without eps, subnormals, values whose squares leave fp32, infinities and NaN: each in its row."""
    K = 256
    x = torch.zeros(9, K)
    x[1] = 1
    x[2] = 2.0 ** -130
    x[3, 5] = 2.0 ** -133
    x[4] = 3e19
    x[5, 7] = float("inf")
    x[6, 9] = float("nan")
    x[7] = 2.0 ** 55
    x[8, :3] = torch.tensor([448.0, -449.0, 2.0 ** -126])
    x = x.to(BF16).cuda()
    g = torch.zeros(K, dtype=BF16, device="cuda")
    for eps in (1e-6, 0.0):
        out = mr.add_rms_norm(x, None, g, eps, quant="fp8", outputs=("sres", "rstd", "xn"))
        r = out["rstd"].cpu()
        inf = float("inf")
        assert r[0] == (torch.tensor(1e-6).double().rsqrt().float() if eps else inf)
        assert r[4] == 0 and r[5] == 0 and r[6].isnan() and r[1] == (1.0 if not eps else r[1])
        assert r[7] == 2.0 ** -55
        if not eps:  # the squares of rows 2 and 3 are below fp32's smallest number
            assert r[2] == inf and r[3] == inf
        xn = out["xn"].float().cpu()
        assert (xn[4] == 0).all() and xn[5].isnan().sum() == 1 and (xn[6].isnan()).all()
        assert same(out["xn"], ref.normed(x, out["rstd"], g, "gemma"))
        q, s = mr.fp8_quant(out["xn"])
        assert same(out["q"], q) and same(out["scale"], s)
        assert (xn[0] == 0).all() if eps else xn[0].isnan().all()


def test_rows_beyond_32_bit_offsets(mr):
    M, K = 360_000, 6144  # 2.2e9 elements
    x = torch.empty(M, K, dtype=BF16, device="cuda")
    for i in range(0, M, 60_000):
        x[i:i + 60_000].normal_()
    g = ref.rows(3, 1, K)[0]
    out = mr.add_rms_norm(x, x, g, quant="fp8", outputs=("rstd",))
    for rows in (slice(0, 64), slice(349_500, 349_600), slice(M - 64, M)):
        part = mr.add_rms_norm(x[rows], x[rows], g, quant="fp8", outputs=("rstd",))
        assert all(torch.equal(part[k], out[k][rows]) for k in part)


@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (3, 128, 8), (7, 2976, 0), (65, 6144, 16), (4096, 1536, 0)])
def test_fp8_quant(mr, M, K, pad):
    x = ref.rows(M, M, K + pad)[:, :K]
    if M > 2:
        x[2, :16] = 0
        x[1] = x[1] * 2.0 ** -126
    q, s = mr.fp8_quant(x)
    wq, ws = ref.fp8(x)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_fp8_quant_of_special_values(mr):
    x = torch.zeros(6, 256)
    x[0, 3], x[1, 200], x[2, 130] = float("nan"), float("inf"), float("-inf")
    x[3, :] = 2.0 ** -133
    x[4, :] = 3.3e38
    x = x.to(BF16).cuda()
    q, s = mr.fp8_quant(x)
    back = ref.e4m3(q) * s.double().repeat_interleave(128, 1)
    assert back[0, :128].isnan().all() and (back[0, 128:] == 0).all()
    assert back[1, 128:].isnan().all() and back[2, 128:].isnan().all() and (back[1, :128] == 0).all()
    assert (s[3] == 2.0 ** -126).all() and (back[3] == 2.0 ** -133).all()
    # half a step of e4m3 (2^-4), and the steps of fp32 on the way
    assert ((back[4] - x[4].double()).abs() <= x[4].double() * (2.0 ** -4 + 2.0 ** -21)).all()
    assert (back[5] == 0).all() and (s[5] == 2.0 ** -126).all()


def test_refusals(mr):
    x, g = ref.rows(1, 4, 256), ref.rows(2, 1, 256)[0]
    bad = [lambda: mr.add_rms_norm(x, x[:3], g), lambda: mr.add_rms_norm(x, None, g[:128]),
           lambda: mr.add_rms_norm(x, None, g, norm="layer"), lambda: mr.add_rms_norm(x, None, g, quant="int8"),
           lambda: mr.add_rms_norm(x, None, g, outputs=("q",)), lambda: mr.add_rms_norm(x, None, g, outputs=()),
           lambda: mr.add_rms_norm(x, None, g, out=dict(rstd=torch.empty(5, device="cuda"))),
           lambda: mr.add_rms_norm(x.float(), None, g), lambda: mr.add_rms_norm(x.t(), None, g),
           lambda: mr.add_rms_norm(x[:, :240], None, g[:240], quant="mxfp8"),
           lambda: mr.fp8_quant(x.float()), lambda: mr.fp8_quant(x, out=(x, x))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mr.add_rms_norm(x[:, :248], None, g[:248], quant="fp8"), lambda: mr.fp8_quant(x[:, :248]),
                 lambda: mr.add_rms_norm(x[:, :252], None, g[:252].clone())):
        with pytest.raises(mr.MoeRouteUnsupported):
            call()
    with pytest.raises(mr.MoeRouteError):
        mr.add_rms_norm(x, None, g, eps=-1.0)
    with pytest.raises(mr.MoeRouteError):  # rows that do not start on 16 bytes
        mr.add_rms_norm(x[:, 4:].clone()[:, 1:249], None, g[:248].clone())


def test_captured_prepared_and_on_another_stream(mr):
    x, res, g = ref.rows(1, 16, 6144), ref.rows(2, 16, 6144), ref.rows(3, 1, 6144)[0]
    want = mr.add_rms_norm(x, res, g, quant="mxfp8", outputs=("sres", "rstd", "xn"))
    call = mr.PreparedAddNorm(x, res, g, quant="mxfp8", outputs=("sres", "rstd", "xn"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(same(got[k], want[k]) for k in want)
    other = mr.add_rms_norm(x, res, g, quant="mxfp8", outputs=("sres", "rstd", "xn"), stream=side)
    side.synchronize()
    assert all(same(other[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(ref.rows(7, 16, 6144))
    for t in got.values():
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(mr, got, x, res, g, 1e-6, "gemma", "mxfp8")


def test_in_front_of_the_route(mr):
    """The route on the norm's scale, fed by the norm: the outputs of the norm written out and routed."""
    M, K, N = 16, 6144, 128
    x, res, g = ref.rows(1, M, K), ref.rows(2, M, K), (0.1 * ref.rows(3, 1, K)[0].float()).to(BF16)
    w = (0.02 * torch.randn(N, K, generator=torch.Generator("cpu").manual_seed(4))).to(BF16).cuda()
    h = mr.add_rms_norm(x, res, g, quant="mxfp8", outputs=("sres", "rstd", "xn"))
    a = mr.moe_route(h["sres"], w, 8, 16, rstd=h["rstd"], norm_weight=g)
    b = mr.moe_route(h["xn"], w, 8, 16)
    assert all(torch.equal(a[k], b[k]) for k in ("logits", "topk_ids", "topk_weights", "q", "scale"))
    assert torch.equal(a["q"], h["q"]) and torch.equal(a["scale"], h["scale"])
