"""The FP8 product with scales per 128 on the GPU, against its formula."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    yield mr
    assert mr.device_error() == mr.MR_OK


def padded(t, multiple=16):
    """The same rows, each starting on 16 bytes (behind them: codes of NaN)."""
    r, k = t.shape
    big = torch.full((r, -(-k // multiple) * multiple + multiple), 127, dtype=t.dtype, device=t.device)
    big[:, :k] = t
    return big[:, :k]


def operands(M, R, K, seed=1):
    kb = -(-K // 128)
    q, w = ref.codes(seed, M, K), ref.codes(seed + 1, R, K)
    if K % 16:
        q, w = padded(q), padded(w)
    return q, ref.scales(seed + 2, M, kb), w, ref.scales(seed + 3, -(-R // 128), kb)


SHAPES = [  # M, R, K
    (1, 1, 1), (1, 16, 16), (1, 200, 300), (2, 129, 128), (7, 33, 129), (8, 6144, 768), (1, 1536, 6144), (9, 500, 100),
    (16, 17, 2976), (17, 128, 256), (33, 2000, 512), (64, 1000, 1024), (65, 15, 640), (100, 255, 2048), (127, 256, 384),
    (128, 257, 400), (129, 300, 1000), (200, 2500, 528), (255, 700, 127), (256, 6144, 256), (257, 6100, 144),
    (300, 2000, 2976), (500, 9000, 272), (1001, 4100, 640), (1300, 1536, 6144),
    (17, 1536, 6144), (40, 1536, 5000), (64, 500, 6144), (100, 1536, 3000), (60, 6144, 1100)]


@pytest.mark.parametrize("M,R,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values(mr, M, R, K, dtype):
    a = operands(M, R, K)
    out = mr.fp8_gemm(*a, out_dtype=dtype)
    assert out.dtype == dtype
    want, tol = ref.product(*a, dtype)
    ref.assert_within(out, want, tol)


@pytest.mark.parametrize("M,R,K", [(3, 300, 1100), (40, 700, 260), (150, 1030, 400), (600, 6200, 300)])
def test_whole_numbers_are_exact(mr, M, R, K):
    """Small whole codes and scales that are powers of two: every sum is exact, so each row, column and block of K
    must have met its own scale."""
    gen = torch.Generator("cpu").manual_seed(M)
    kb = -(-K // 128)
    whole = lambda r: torch.randint(-3, 4, (r, K), generator=gen).float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    power = lambda r: torch.ldexp(torch.ones(r, kb), torch.randint(-2, 3, (r, kb), generator=gen)).cuda()  # noqa: E731
    q, w = whole(M), whole(R)
    if K % 16:
        q, w = padded(q), padded(w)
    xs, ws = power(M), power(-(-R // 128))
    out = mr.fp8_gemm(q, xs, w, ws, out_dtype=F32)
    assert torch.equal(out.double(), ref.product(q, xs, w, ws, F32)[0])


@pytest.mark.parametrize("M", [1, 5, 40, 130, 700])
def test_strides_and_what_lies_around(mr, M):
    R, K = 1100, 272
    q, xs, w, ws = operands(M, R, K)
    want = mr.fp8_gemm(q, xs, w, ws)
    big = torch.full((M + 2, R + 24), 7.0, dtype=BF16, device="cuda")
    wide = lambda t, left, pad: torch.nn.functional.pad(t.float() if t.dtype == F32 else t, (left, pad))[:, left:left + t.shape[1]]  # noqa: E731
    for off in (0, 8, 3):
        big.fill_(7)
        out = big[1:M + 1, off:off + R]
        got = mr.fp8_gemm(wide(q, 16, 32), wide(xs, 1, 2), wide(w, 32, 16), wide(ws, 3, 0), out=out)
        assert got is out and torch.equal(out, want)
        big[1:M + 1, off:off + R] = 7
        assert (big == 7).all()


@pytest.mark.parametrize("M", [3, 200, 600])
def test_nan_and_infinity_stay_in_their_rows_and_columns(mr, M):
    R, K = 700, 640
    q, xs, w, ws = operands(M, R, K)
    q[1, 200], w[300, 5] = 127, 255
    xs = xs.clone()
    xs[2, 4] = float("inf")
    out = mr.fp8_gemm(q, xs, w, ws, out_dtype=F32)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[1:3] = True
    want[:, 300] = True
    assert torch.equal(bad, want)


def test_one_rounding_and_no_order_of_calls(mr):
    """The bf16 result is the fp32 one rounded once, and the same on every call."""
    for M, R, K in ((1, 6144, 6144), (40, 1536, 6144), (300, 2000, 2976), (1001, 6144, 768)):
        a = operands(M, R, K)
        one = mr.fp8_gemm(*a, out_dtype=F32)
        assert torch.equal(one.to(BF16), mr.fp8_gemm(*a))
        for _ in range(5):
            assert torch.equal(mr.fp8_gemm(*a, out_dtype=F32), one)


def test_large_offsets(mr):
    """Rows of x, of the weight and of the result behind 2^31 elements."""
    K, R = 256, 70_000
    M = 33_000
    q, xs, w, ws = operands(200, R, K)
    rep = lambda t: t.repeat(M // 200, 1)  # noqa: E731
    out = mr.fp8_gemm(rep(q), rep(xs), w, ws)
    assert out.numel() > 1 << 31
    want = mr.fp8_gemm(q, xs, w, ws, out_dtype=F32).to(BF16)
    for i in (0, 77, 164):
        assert torch.equal(out[200 * i:200 * i + 200], want)
    big = torch.zeros(300, 1 << 23, dtype=torch.uint8, device="cuda")[:, :K]  # a row stride of 8 MB
    big.copy_(w[:300])
    assert torch.equal(mr.fp8_gemm(q, xs, big, ws[:3]), mr.fp8_gemm(q, xs, w[:300].clone(), ws[:3]))


def test_refusals(mr):
    q, xs, w, ws = operands(5, 300, 256)
    bad = [lambda: mr.fp8_gemm(q, xs[:4], w, ws), lambda: mr.fp8_gemm(q, xs, w[:, :128], ws),
           lambda: mr.fp8_gemm(q, xs, w, ws[:2]), lambda: mr.fp8_gemm(q, xs[:, :1], w, ws),
           lambda: mr.fp8_gemm(q, xs.double(), w, ws), lambda: mr.fp8_gemm(q.float(), xs, w, ws),
           lambda: mr.fp8_gemm(q, xs, w, ws, out_dtype=torch.float16),
           lambda: mr.fp8_gemm(q, xs, w, ws, out=torch.empty(5, 299, dtype=BF16, device="cuda")),
           lambda: mr.fp8_gemm(q, xs, w, ws, out=torch.empty(300, 5, dtype=BF16, device="cuda").t()),
           lambda: mr.fp8_gemm(q, xs, w, ws, out=torch.empty(5, 300, dtype=BF16, device="cuda"), out_dtype=F32)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    c = ref.codes(1, 5, 250)
    for call in (lambda: mr.fp8_gemm(c, xs, padded(ref.codes(2, 300, 250)), ws),       # rows not on 16 bytes
                 lambda: mr.fp8_gemm(padded(c), xs, ref.codes(2, 300, 250), ws)):
        with pytest.raises(mr.MoeRouteError):
            call()


def test_captured_prepared_and_on_another_stream(mr):
    a = operands(40, 1536, 1024)
    call = mr.PreparedFp8Gemm(*a)
    want = mr.fp8_gemm(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(mr.fp8_gemm(*a, stream=side), want)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    a[0].copy_(ref.codes(9, 40, 1024))
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, mr.fp8_gemm(*a))


def test_a_wait_that_runs_out(mr):
    """Each kernel's bounded waits (the test hook makes the first stage expect more than is copied): an error, and
    the next call is right."""
    mr.set_wait_limit_ns(2_000_000)
    try:
        for M, R, K in ((3, 500, 512), (200, 500, 512), (700, 6144, 512)):
            a = operands(M, R, K)
            mr.set_launch_flags(mr.LAUNCH_TEST_STALL)
            mr.fp8_gemm(*a)
            torch.cuda.synchronize()
            mr.set_launch_flags(0)
            assert mr.device_error(clear=True) == mr.MR_ERR_TIMEOUT
            out = mr.fp8_gemm(*a, out_dtype=F32)
            torch.cuda.synchronize()
            assert mr.device_error() == mr.MR_OK
            want, tol = ref.product(*a, F32)
            ref.assert_within(out, want, tol)
    finally:
        mr.set_launch_flags(0)
        mr.set_wait_limit_ns(1_000_000_000)
        mr.device_error(clear=True)


def test_a_layer(mr):
    """Residual and norm, the route on the norm's scale, rows to their experts, FP8 products of each, and back."""
    M, K, I, E, topk, block = 45, 512, 256, 8, 3, 16
    x, res, g = ref.rows(1, M, K), ref.rows(2, M, K), (0.1 * ref.rows(3, 1, K)[0].float()).to(BF16)
    gate = (0.05 * torch.randn(E, K, generator=torch.Generator("cpu").manual_seed(4))).to(BF16).cuda()
    w = [(ref.codes(10 + e, I, K), ref.scales(30 + e, I // 128, K // 128)) for e in range(E)]
    h = mr.add_rms_norm(x, res, g, quant="fp8", outputs=("sres", "rstd", "xn"))
    r = mr.moe_route(h["sres"], gate, topk, block, rstd=h["rstd"], norm_weight=g, quant=None)
    st, nt, ids = r["sorted_token_ids"], r["num_tokens_post_padded"], r["topk_ids"]
    q, pos = mr.moe_permute(h["q"], ids, E, st, nt)
    s, _ = mr.moe_permute(h["scale"], ids, E, st, nt)
    y = torch.zeros(st.numel(), I, dtype=BF16, device="cuda")
    for b, e in enumerate(r["expert_ids"].tolist()):
        if e >= 0:
            rows = slice(b * block, (b + 1) * block)
            mr.fp8_gemm(q[rows], s[rows], *w[e], out=y[rows])
    out = mr.moe_combine(y, pos, r["topk_weights"])
    want = torch.zeros(M, I, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(want)
    for e in range(E):
        p, t = ref.product(h["q"], h["scale"], *w[e], BF16)
        wt = (r["topk_weights"].double() * (ids == e)).sum(1, keepdim=True)
        want += wt * p
        tol += wt * (t + 2.0 ** -22 * p.abs())
    ref.assert_within(out, want, tol + 2.0 ** -8 * (want.abs() + tol))
    assert torch.equal(h["q"], mr.fp8_quant(h["xn"])[0])
