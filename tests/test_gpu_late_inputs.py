"""Operands that the kernel launched just before writes at its very end, while the call's first CTAs are already
resident: every call reads them after that kernel, not when it starts."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402
from tests import expert_ref  # noqa: E402

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
ROWS, COLS, LONG = 16, 384, 1 << 20  # of the product that writes late: 24 CTAs


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    mr.set_launch_flags(mr.LAUNCH_PDL)
    yield mr
    mr.set_launch_flags(0)


@pytest.fixture(scope="module")
def long_product(mr):
    """A product over 2^20: some 200 us on 24 SMs, its results written when all of it is summed.  Values of about one,
    and of the bytes of codes without NaN."""
    x = ref.codes(1, 16, 4096).repeat(1, LONG // 4096)
    w = ref.codes(2, COLS, 4096).repeat(1, LONG // 4096)
    one = torch.ones
    return x, one(16, LONG // 128, device="cuda"), w, one(COLS // 128, LONG // 128, device="cuda") * 2.0 ** -30


def flat(out):
    return list(out.values()) if isinstance(out, dict) else list(out) if isinstance(out, (tuple, list)) else [out]


def alike(a, b):
    return all(torch.equal(x.contiguous().view(-1).view(U8), y.contiguous().view(-1).view(U8)) for x, y in zip(a, b))


def check(mr, long_product, operand, call):
    """call reads operand, whose first rows' first columns are written late."""
    t = operand if operand.dtype in (BF16, F32) else operand.view(BF16)
    if t.dim() == 1:
        t = t[None, :]
    corner = t[:ROWS, :COLS]
    m, r = corner.shape
    x, xs, w, ws = long_product
    late = mr.PreparedFp8Gemm(x[:m], xs[:m], w[:r], ws[:-(-r // 128)], out=corner)
    late()
    want = [o.clone() for o in flat(call())]
    torch.cuda.synchronize()
    for _ in range(3):
        corner.fill_(0)
        for o in flat(call()):  # (of the stale operand)
            o.clone()
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000)  # (both launches are queued when the first one starts)
        late()
        got = [o.clone() for o in flat(call())]
        torch.cuda.synchronize()
        assert alike(got, want)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8", "mxfp4", None])
@pytest.mark.parametrize("M,K", [(1, 6144), (40, 6144), (20, 16416), (20, 40000), (500, 1024), (500, 4096), (500, 5120),
                                 (500, 6144), (400, 8192), (400, 12288), (400, 16384)])
def test_add_rms_norm(mr, long_product, M, K, quant):
    x, res, g = ref.rows(1, M, K), ref.rows(2, M, K), ref.rows(3, 1, K)[0].clone()
    call = mr.PreparedAddNorm(x, res, g, quant=quant, outputs=("sres", "rstd", "xn"))
    for operand in (x, res, g):
        check(mr, long_product, operand, call)
    check(mr, long_product, x, mr.PreparedAddNorm(x, None, g, quant=quant, outputs=("rstd", "xn")))


@pytest.mark.parametrize("M", [1, 40, 600])
def test_quantisers(mr, long_product, M):
    x, g = ref.rows(1, M, 6144), ref.rows(2, 1, 6144)[0].clone()
    rstd = torch.rand(M, device="cuda") + 0.5
    check(mr, long_product, x, lambda: mr.fp8_quant(x))
    check(mr, long_product, x, lambda: mr.mxfp8_quant(x))
    check(mr, long_product, x, lambda: mr.mxfp4_quant(x))
    for operand in (x, rstd, g):
        check(mr, long_product, operand, lambda: mr.norm_apply(x, rstd, g))


@pytest.mark.parametrize("M,R,K", [(1, 512, 6144), (16, 6144, 1024), (40, 1536, 6144), (64, 512, 2048), (200, 512, 1024),
                                   (300, 2000, 1024), (1000, 1536, 512), (2000, 1536, 512)])
def test_fp8_gemm(mr, long_product, M, R, K):
    q, xs, w, ws = ref.codes(1, M, K), ref.scales(2, M, K // 128), ref.codes(3, R, K), ref.scales(4, -(-R // 128), K // 128)
    call = mr.PreparedFp8Gemm(q, xs, w, ws)
    for operand in (q, xs, w, ws):
        check(mr, long_product, operand, call)


@pytest.mark.parametrize("M,K,topk", [(16, 6144, 8), (300, 6144, 8), (300, 6143, 3), (300, 1001, 4), (300, 6140, 4)])
def test_rows(mr, long_product, M, K, topk):
    ids, wts = ref.routed(M, 64, topk, 1, 0.1)
    st, _, nt = mr.moe_sort(ids, 64, 16)
    cap = st.numel()
    x, y = ref.rows(1, M, K), ref.rows(2, cap, K)
    pos = ref.positions(st, int(nt), M * topk).view(M, topk).int().contiguous()
    zero = lambda: torch.zeros(cap, K, dtype=BF16, device="cuda")  # noqa: E731
    check(mr, long_product, x, mr.PreparedPermute(x, ids, 64, st, nt, out=zero()))
    for operand in (y, wts, x):
        check(mr, long_product, operand, mr.PreparedCombine(y, pos, wts, x))
        check(mr, long_product, operand, mr.PreparedCombineGrad(x, y, pos, wts, st, nt, out=zero()))


@pytest.mark.parametrize("M", [1, 8, 16, 40, 64])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route(mr, long_product, M, scoring):
    N, K = 128, 6144
    x, g, w = ref.rows(1, M, K), ref.rows(2, 1, K)[0].clone(), ref.rows(3, N, K)
    bias = torch.rand(N, device="cuda") if scoring == "sigmoid" else None
    rstd = torch.rand(M, device="cuda") + 0.5
    plain = mr.PreparedRoute(x, w, 8, 16, scoring, bias)
    normed = mr.PreparedRoute(x, w, 8, 16, scoring, bias, rstd=rstd, norm_weight=g)
    n = lambda call: lambda: [call()[k] for k in ("logits", "topk_ids", "topk_weights", "q", "scale")]  # noqa: E731
    check(mr, long_product, x, n(plain))
    for operand in (x, rstd, g):
        check(mr, long_product, operand, n(normed))
    if bias is not None:
        check(mr, long_product, bias, n(plain))


@pytest.mark.parametrize("M", [8, 100, 300])
def test_router_gemv_and_gate(mr, long_product, M):
    x, w = ref.rows(1, M, 6144), ref.rows(3, 128, 6144)
    check(mr, long_product, x, lambda: mr.router_gemv(x, w))
    logits, bias = torch.randn(M, 384, device="cuda"), torch.rand(384, device="cuda")
    for operand in (logits, bias):
        check(mr, long_product, operand, lambda: mr.route_topk(logits, 8, "sigmoid", bias))


@pytest.mark.parametrize("M", [16, 300])
def test_expert_products(mr, long_product, M):
    K, I, E, topk, block = 1024, 512, 8, 4, 16
    ids, wts = ref.routed(M, E, topk, 1)
    st, ex, _ = mr.moe_sort(ids, E, block)
    q, s = expert_ref.random_mx((M, K), "mxfp8", 3)
    w13 = mr.MxWeight(*expert_ref.random_mx((E, 2 * I, K), "mxfp8", 4, 112, 116), gate_up=True)
    w2 = mr.MxWeight(*expert_ref.random_mx((E, K, I), "mxfp8", 5, 112, 116))
    a, sa = expert_ref.random_mx((st.numel(), I), "mxfp8", 6)
    act = torch.zeros(st.numel(), I, dtype=BF16, device="cuda")  # (rows behind the last are left as they were)
    for operand in (q, s):
        check(mr, long_product, operand, lambda: mr.moe_gate_up(q, s, w13, st, ex, topk, block, out=act))
    for operand in (a, sa, wts):
        check(mr, long_product, operand, lambda: mr.moe_down(a, sa, w2, ids, wts, st, ex, block))
    W = mr.MxWeight(*expert_ref.random_mx((K, K), "mxfp8", 7, 112, 116))
    for operand in (q, s):
        check(mr, long_product, operand, lambda: mr.mx_gemm(q, s, W))
