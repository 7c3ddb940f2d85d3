"""The norm, the FP8 products and the rows to the experts and back in the orders, streams and sizes of a program:
back to back on the same buffers, on several streams at once, captured; every variant of the product."""

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


def operands(M, R, K, seed=1):
    kb = -(-K // 128)
    xs, ws = ref.scales(seed + 2, M, kb), ref.scales(seed + 3, -(-R // 128), kb)
    return ref.codes(seed, M, K), xs, ref.codes(seed + 1, R, K), ws


# one of each: pairs of CTAs of both widths; tiles whose K range 2, 4 or 8 CTAs share; 64- and 128-row products; one,
# two and four blocks a stage; few rows of x in wide and narrow grids
VARIANTS = [
    (4096, 700, 6144), (2048, 2000, 4096), (1000, 6144, 6144), (2048, 2500, 1104), (4096, 300, 4096), (4096, 100, 4096),
    (1300, 100, 16384), (129, 12000, 112), (17, 12000, 8192), (1300, 2500, 112), (1000, 2000, 16384), (100, 15, 112),
    (100, 15, 8192), (1300, 100, 4096), (64, 2000, 16384), (65, 6144, 4096), (50, 2500, 6144), (65, 16384, 112),
    (33, 9000, 8192), (17, 15, 16384), (17, 6144, 112), (17, 2500, 6144), (17, 1536, 8192), (200, 6144, 6144),
    (40, 6144, 6144), (16, 6144, 6144), (16, 100, 16384), (9, 10000, 112), (8, 16384, 2048), (3, 40, 8192),
    (2048, 300, 6144), (4096, 100, 6144), (129, 2500, 112), (50, 6144, 112), (65, 15, 112), (17, 15, 112)]


@pytest.mark.parametrize("M,R,K", VARIANTS)
def test_every_variant_of_the_product(mr, M, R, K):
    a = operands(M, R, K)
    out = mr.fp8_gemm(*a, out_dtype=F32)
    want, tol = ref.product(*a, F32)
    ref.assert_within(out, want, tol)
    for _ in range(3):
        assert torch.equal(mr.fp8_gemm(*a, out_dtype=F32), out)


def test_a_pair_whose_wait_runs_out(mr):
    """A pair's bounded waits: an error, and the next call is right."""
    a = operands(2048, 2000, 4096)
    want = mr.fp8_gemm(*a)
    torch.cuda.synchronize()
    mr.set_wait_limit_ns(2_000_000)
    try:
        mr.set_launch_flags(mr.LAUNCH_TEST_STALL)
        mr.fp8_gemm(*a)
        torch.cuda.synchronize()
        mr.set_launch_flags(0)
        assert mr.device_error(clear=True) == mr.MR_ERR_TIMEOUT
        assert torch.equal(mr.fp8_gemm(*a), want)
        torch.cuda.synchronize()
        assert mr.device_error() == mr.MR_OK
    finally:
        mr.set_launch_flags(0)
        mr.set_wait_limit_ns(1_000_000_000)
        mr.device_error(clear=True)


class Layers:
    """Layers of norm, route, rows to the experts, a product, rows back; all on the same buffers, so that a call that
    read early or wrote before the one before it had ended would change a value."""

    def __init__(self, mr, M, K=1024, E=16, topk=4, block=16):
        self.mr, self.n = mr, 8
        self.x0, self.r0 = ref.rows(1, M, K), ref.rows(2, M, K)
        g = (0.1 * ref.rows(3, 1, K)[0].float()).to(BF16)
        gate = (0.05 * torch.randn(E, K, generator=torch.Generator("cpu").manual_seed(4))).to(BF16).cuda()
        self.wb = [(0.05 * ref.rows(20 + i, K, K).float()).to(BF16) for i in range(self.n)]
        e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        self.x, self.res = e(M, K), e(M, K)
        self.w, self.wsr = e(K, K, dt=torch.uint8), e(K, K // 128, dt=F32)
        self.ws = torch.full((K // 128, K // 128), 2.0 ** -9, device="cuda")
        self.norm = mr.PreparedAddNorm(self.x, self.res, g, quant="fp8", outputs=("sres", "rstd", "xn"),
                                       out={"sres": self.res})
        h = self.norm.out
        self.route = None
        if M <= 64:
            self.route = mr.PreparedRoute(h["sres"], gate, topk, block, rstd=h["rstd"], norm_weight=g, quant=None)
            r = self.route.out
            st, nt = r["sorted_token_ids"], r["num_tokens_post_padded"]
            ids, wts = r["topk_ids"], r["topk_weights"]
        else:
            ids, wts = ref.routed(M, E, topk, 5, 0.1)
            st, _, nt = mr.moe_sort(ids, E, block)
        self.perm = mr.PreparedPermute(h["q"], ids, E, st, nt)
        self.perm_s = mr.PreparedPermute(h["scale"], ids, E, st, nt)
        self.perm.out[0].zero_()
        self.perm_s.out[0].zero_()
        self.dense = mr.PreparedFp8Gemm(h["q"], h["scale"], self.w, self.ws)
        self.gemm = mr.PreparedFp8Gemm(self.perm.out[0], self.perm_s.out[0], self.w, self.ws)
        self.back = mr.PreparedCombine(self.gemm.out, self.perm.out[1], wts, add=h["xn"], out=self.x)
        # (backwards: of the rows' way, by the gradient of the sum)
        self.grad = mr.PreparedCombineGrad(self.x, self.gemm.out, self.perm.out[1], wts, st, nt)
        self.grad.out[0].zero_()
        self.gx = mr.PreparedPermuteGrad(self.grad.out[0], self.perm.out[1])

    def run(self, between=lambda: None):
        self.x.copy_(self.x0)
        self.res.copy_(self.r0)
        kept = []
        for i in range(self.n):
            self.mr.fp8_quant(self.wb[i], out=(self.w, self.wsr))  # the weight, written just before
            between()
            self.norm()
            between()
            if self.route is not None:
                self.route()
                between()
            for call in (self.dense, self.perm, self.perm_s, self.gemm, self.back, self.grad, self.gx):
                call()
                between()
            kept.append((self.x.clone(), self.dense.out.clone(), self.gx.out.clone(), self.grad.out[1].clone()))
        return kept


@pytest.mark.parametrize("M", [1, 3, 16, 40, 64, 300, 1500])
@pytest.mark.parametrize("pdl", [False, True])
def test_layers_back_to_back(mr, M, pdl):
    layers = Layers(mr, M)
    want = layers.run(torch.cuda.synchronize)
    try:
        mr.set_launch_flags(mr.LAUNCH_PDL if pdl else 0)
        for _ in range(3):
            got = layers.run()
            for a, b in zip(want, got):
                assert all(torch.equal(s, t) for s, t in zip(a, b))
                assert torch.isfinite(a[0].float()).all()
    finally:
        mr.set_launch_flags(0)


@pytest.mark.parametrize("M", [3, 40, 300])
def test_captured_layers(mr, M):
    layers = Layers(mr, M)
    want = layers.run(torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layers.run()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_several_streams_at_once(mr):
    """Calls of every kind on three streams, some of them on the same inputs: the values of one after the other."""
    shapes = [(3, 2000, 2048), (16, 6144, 768), (40, 1536, 2048), (64, 500, 4096), (300, 2000, 1024),
              (2048, 2000, 4096)]
    prods = [operands(*s, seed=5 * i) for i, s in enumerate(shapes)]
    want = [mr.fp8_gemm(*a) for a in prods]
    x, res, g = ref.rows(1, 700, 2048), ref.rows(2, 700, 2048), ref.rows(3, 1, 2048)[0].contiguous()
    norm = mr.add_rms_norm(x, res, g, quant="fp8")
    ids, wts = ref.routed(700, 32, 4, 7, 0.1)
    st, ex, nt = mr.moe_sort(ids, 32, 16)
    torch.cuda.synchronize()
    n = int(nt)
    rows, pos = mr.moe_permute(x, ids, 32, st, nt)
    y = torch.zeros(st.numel(), 2048, dtype=BF16, device="cuda")
    y[:n] = rows[:n]
    back = mr.moe_combine(y, pos, wts)
    gy, gw = mr.moe_combine_grad(x, y, pos, wts, st, nt)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                order = prods[(turn + i) % 6:] + prods[:(turn + i) % 6]
                results.append(([mr.fp8_gemm(*a) for a in order], (turn + i) % 6,
                                mr.add_rms_norm(x, res, g, quant="fp8"), mr.moe_permute(x, ids, 32, st, nt),
                                mr.moe_combine(y, pos, wts), mr.moe_combine_grad(x, y, pos, wts, st, nt)))
    torch.cuda.synchronize()
    for outs, first, h, (r, p), b, (a, w) in results:
        assert all(torch.equal(o, q) for o, q in zip(outs, want[first:] + want[:first]))
        assert all(torch.equal(h[k], norm[k]) for k in norm)
        assert torch.equal(r[:n], rows[:n]) and torch.equal(p, pos) and torch.equal(b, back)
        assert torch.equal(a[:n], gy[:n]) and torch.equal(w, gw)


@pytest.mark.parametrize("M", [3, 17, 40, 100, 300, 2048])
def test_a_scale_beyond_the_range_stays_where_it_is(mr, M):
    """An infinite scale of the last, ragged block of K, NaN behind the scales and codes of NaN behind K."""
    R, K = 2500, 1104
    q, xs, w, ws = operands(M, R, K)

    def wide(t, fill):
        return torch.cat([t, torch.full((t.shape[0], 16), fill, dtype=t.dtype, device="cuda")], 1)[:, :t.shape[1]]

    want, tol = ref.product(q, xs, w, ws, F32)
    xs, ws = wide(xs, float("nan")), wide(ws, float("nan"))
    xs[M - 1, -1] = float("inf")
    out = mr.fp8_gemm(wide(q, 127), xs, wide(w, 255), ws, out_dtype=F32)
    assert not torch.isfinite(out[M - 1]).any()
    ref.assert_within(out[:M - 1], want[:M - 1], tol[:M - 1])


@pytest.mark.parametrize("topk,K", [(32, 2056), (9, 4104), (1, 6144), (17, 2564)])
def test_many_tokens_of_many_slots(mr, topk, K):
    """Thousands of tokens, slots beyond eight, an expert taken twice by a token."""
    M, E = 4000 // topk * 2 + 1000, 64
    ids, wts = ref.routed(M, E, topk, 3, 0.05)
    ids[5::7, -1] = ids[5::7, 0]
    st, ex, nt = mr.moe_sort(ids, E, 16)
    x = ref.rows(4, M, K)
    rows, pos = mr.moe_permute(x, ids, E, st, nt)
    n, f = int(nt), st[:int(nt)].long()
    real = f < M * topk
    want = torch.zeros(n, K, dtype=BF16, device="cuda")
    want[real] = x[f[real] // topk]
    assert torch.equal(rows[:n], want)
    there = pos.view(-1)[f[real]].long()
    assert torch.equal(there, torch.arange(n, device="cuda")[real])
    assert int((pos >= 0).sum()) == int(real.sum())
    out = mr.moe_combine(rows, pos, wts, add=x)
    s = (wts * (pos >= 0)).double().sum(1, keepdim=True)
    size = (wts.abs() * (pos >= 0)).double().sum(1, keepdim=True)
    val = x.double() * (1 + s)
    # topk fused multiply-adds in fp32, then bf16
    tol = (topk * 2.0 ** -24) * x.double().abs() * (1 + size)
    ref.assert_within(out, val, tol + 2.0 ** -8 * (val.abs() + tol))


@pytest.mark.parametrize("K", [1, 3, 8, 9, 33, 100, 1001])
@pytest.mark.parametrize("dtype", [BF16, F32, torch.uint8])
def test_rows_that_start_anywhere(mr, K, dtype):
    """Operands and results that start at any element of their memory, in place too: the values of aligned ones, and
    nothing beside them changed.  (Memory beside the operands holds NaN.)"""
    M, E, topk = 37, 8, 3
    ids, wts = ref.routed(M, E, topk, 2, 0.2)
    st, _, nt = mr.moe_sort(ids, E, 8)
    n, cap = int(nt), st.numel()
    codes = dtype == torch.uint8

    def within(t, off):
        fill = 77 if codes else float("nan")
        flat = torch.full((t.numel() + 48,), fill, dtype=t.dtype, device="cuda")
        view = flat[off:off + t.numel()].view(t.shape)
        view.copy_(t)
        return flat, view

    def beside(flat, off, count):
        left = torch.cat([flat[:off], flat[off + count:]])
        return (left == 77).all() if codes else torch.isnan(left).all()

    x = ref.codes(1, M, K) if codes else ref.rows(1, M, K, dtype)
    rows, pos = mr.moe_permute(x, ids, E, st, nt, out=torch.zeros(cap, K, dtype=dtype, device="cuda"))
    for off in (1, 2, 5, 8, 15):
        flat, out = within(torch.zeros_like(rows), 16 - off)
        got, p = mr.moe_permute(within(x, off)[1], ids, E, st, nt, out=out)
        assert torch.equal(got, rows) and torch.equal(p, pos) and beside(flat, 16 - off, cap * K)
        if codes:
            continue
        y, add = ref.rows(3, cap, K, dtype), ref.rows(4, M, K, dtype)
        want = mr.moe_combine(y, pos, wts, add=add)
        flat, out = within(add, off)
        assert torch.equal(mr.moe_combine(within(y, 17 - off)[1], pos, wts, add=out, out=out), want)
        assert beside(flat, off, M * K)
        assert torch.equal(mr.moe_permute_grad(within(y, off)[1], pos), mr.moe_permute_grad(y, pos))
        gy, gw = mr.moe_combine_grad(x, y, pos, wts, st, nt, out=torch.zeros_like(y))
        flat, out = within(y, off)
        gy2, gw2 = mr.moe_combine_grad(within(x, 16 - off)[1], out, pos, wts, st, nt, out=out)
        assert torch.equal(gy2[:n], gy[:n]) and torch.equal(gy2[n:], y[n:]) and beside(flat, off, cap * K)
        # (fp32 sums over K in another order)
        tol = K * 2.0 ** -23 * (x.double().abs().max() * y[:n].double().abs().max()) * K
        assert ((gw2 - gw).double().abs() <= tol).all()
