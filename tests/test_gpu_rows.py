"""Rows to the experts and back, and their gradients, on the GPU."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32

SHAPES = [  # M, K, topk, E, block, drop
    (1, 1, 1, 1, 1, 0.0), (1, 6144, 8, 128, 16, 0.0), (3, 65, 2, 8, 16, 0.3), (16, 3584, 16, 896, 16, 0.0),
    (37, 1000, 7, 100, 16, 0.5), (100, 2049, 5, 32, 64, 0.125), (129, 130, 32, 64, 8, 0.2), (64, 7, 3, 4, 64, 1.0),
    (1001, 516, 8, 128, 64, 0.1)]


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    return mr


class Case:
    def __init__(self, mr, shape, dtype, seed=1):
        self.M, self.K, self.topk, self.E, self.block, drop = shape
        self.ids, self.w = ref.routed(self.M, self.E, self.topk, seed, drop)
        self.st, self.ex, self.nt = mr.moe_sort(self.ids, self.E, self.block)
        self.cap, self.n, self.mk = self.st.numel(), int(self.nt), self.M * self.topk
        self.pos = ref.positions(self.st, self.n, self.mk)
        self.real = self.pos >= 0
        self.x = ref.rows(seed, self.M, self.K, dtype)
        self.y = ref.rows(seed + 1, self.cap, self.K, dtype)
        self.tok = torch.arange(self.mk, device="cuda") // self.topk


def out_rows(c, dtype, fill=3):
    return torch.full((c.cap, c.K), fill, dtype=dtype, device="cuda")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32, torch.uint8])
def test_permute(mr, shape, dtype):
    c = Case(mr, shape, BF16 if dtype == torch.uint8 else dtype)
    x = c.x if dtype != torch.uint8 else torch.randint(0, 256, c.x.shape, dtype=dtype, device="cuda")
    out = out_rows(c, dtype)
    rows, pos = mr.moe_permute(x, c.ids, c.E, c.st, c.nt, out=out)
    assert rows is out and torch.equal(pos.view(-1).long(), c.pos)
    want = out_rows(c, dtype)
    want[:c.n] = 0
    want[c.pos[c.real]] = x[c.tok[c.real]]
    assert torch.equal(rows, want)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("weighted,add", [(True, True), (True, False), (False, False)])
def test_combine(mr, shape, dtype, weighted, add):
    c = Case(mr, shape, dtype)
    bad = torch.ones(c.cap, dtype=torch.bool, device="cuda")
    bad[c.pos[c.real]] = False
    y = c.y.clone()
    y[bad] = float("nan")  # what no assignment asks for counts for nothing
    pos = c.pos.view(c.M, c.topk).int()
    w = c.w if weighted else None
    a = ref.rows(9, c.M, c.K, dtype) if add else None
    out = mr.moe_combine(y, pos, w, a)
    g = torch.where(c.real[:, None], c.y.double()[c.pos.clamp(min=0)], 0.0).unflatten(0, (c.M, c.topk))
    w64 = (c.w.double() if weighted else torch.ones_like(c.w).double())[..., None]
    terms = g * w64
    want, mag = terms.sum(1), terms.abs().sum(1)
    if add:
        want, mag = want + a.double(), mag + a.double().abs()
    # each of the topk fused multiply-adds rounds a partial sum to fp32, then one rounding to the type
    tol = (c.topk + 1) * 2.0 ** -24 * mag
    tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + torch.finfo(dtype).smallest_normal * 2.0 ** -10
    ref.assert_within(out, want, tol)
    if add:
        again = a.clone()
        assert mr.moe_combine(y, pos, w, again, out=again) is again and torch.equal(again, out)
    if not weighted and not add:
        assert torch.equal(mr.moe_permute_grad(y, pos), out)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(mr, shape, dtype, weighted):
    c = Case(mr, shape, dtype)
    w = c.w if weighted else None
    pos = c.pos.view(c.M, c.topk).int()
    out = out_rows(c, dtype)
    gy, gw = mr.moe_combine_grad(c.x, c.y, pos, w, c.st, c.nt, out=out)
    f = c.real.nonzero()[:, 0]
    w64 = (c.w.double().view(-1) if weighted else torch.ones(c.mk, dtype=torch.float64, device="cuda"))
    want = out_rows(c, torch.float64)
    want[:c.n] = 0
    want[c.pos[f]] = w64[f, None] * c.x.double()[c.tok[f]]
    tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + torch.finfo(dtype).smallest_normal * 2.0 ** -10
    tol[c.n:] = 0
    ref.assert_within(gy, want, tol, "grad_y")
    terms = c.x.double()[c.tok[f]] * c.y.double()[c.pos[f]]
    wgw, mag = torch.zeros(c.mk, dtype=torch.float64, device="cuda"), torch.zeros(c.mk, dtype=torch.float64, device="cuda")
    wgw[f], mag[f] = terms.sum(1), terms.abs().sum(1)
    # (as many roundings as terms at most)
    ref.assert_within(gw.view(-1), wgw, (c.K + 1) * 2.0 ** -24 * mag, "grad_weights")
    same = c.y.clone()
    gy2, gw2 = mr.moe_combine_grad(c.x, same, pos, w, c.st, c.nt, out=same)
    assert torch.equal(gy2[:c.n], gy[:c.n]) and torch.equal(gy2[c.n:], c.y[c.n:]) and torch.equal(gw2, gw)


def test_gradients_by_differences(mr):
    """On small whole numbers every sum is exact and both calls are linear in each argument, so the differences are
    the gradients."""
    M, K, topk, E, block = 5, 12, 3, 6, 4
    c = Case(mr, (M, K, topk, E, block, 0.3), F32)
    gen = torch.Generator("cpu").manual_seed(2)
    whole = lambda *s: torch.randint(-4, 5, s, generator=gen).float().cuda()  # noqa: E731
    x, y, w, g, gr = whole(M, K), whole(c.cap, K), whole(M, topk), whole(M, K), whole(c.cap, K)
    pos = c.pos.view(M, topk).int()
    live = torch.zeros(c.cap, 1, device="cuda")
    live[c.pos[c.real]] = 1

    loss = lambda y, w: (mr.moe_combine(y, pos, w) * g).sum().item()  # noqa: E731
    gy, gw = mr.moe_combine_grad(g, y, pos, w, c.st, c.nt, out=torch.zeros_like(y))
    base = loss(y, w)
    for p, k in [(int(p), int(k)) for p, k in zip(torch.randint(0, c.cap, (30,)), torch.randint(0, K, (30,)))]:
        d = y.clone()
        d[p, k] += 1
        assert loss(d, w) - base == gy[p, k].item()
    for m in range(M):
        for j in range(topk):
            d = w.clone()
            d[m, j] += 1
            assert loss(y, d) - base == gw[m, j].item()

    spread = lambda x: (mr.moe_permute(x, c.ids, E, c.st, c.nt, out=torch.zeros_like(gr))[0] * gr).sum().item()  # noqa: E731
    gx = mr.moe_permute_grad(gr, pos)
    base = spread(x)
    for m in range(M):
        for k in range(K):
            d = x.clone()
            d[m, k] += 1
            assert spread(d) - base == gx[m, k].item()


def test_infinities_and_nan_stay_in_their_rows(mr):
    c = Case(mr, (8, 256, 2, 4, 16, 0.0), BF16)
    x, y = c.x.clone(), c.y.clone()
    x[3, 5], y[int(c.pos[2]), 9] = float("inf"), float("nan")
    pos = c.pos.view(8, 2).int()
    rows, _ = mr.moe_permute(x, c.ids, c.E, c.st, c.nt)
    bad = (~torch.isfinite(rows[:c.n])).any(1).nonzero()[:, 0].tolist()
    assert bad == sorted(c.pos[6:8].tolist())
    out = mr.moe_combine(y, pos, c.w)
    assert (~torch.isfinite(out)).nonzero().tolist() == [[1, 9]]
    gy, gw = mr.moe_combine_grad(x, y, pos, c.w, c.st, c.nt)
    assert sorted((~torch.isfinite(gw)).view(-1).nonzero()[:, 0].tolist()) == [2, 6, 7]


def test_strided_and_unaligned_operands(mr):
    c = Case(mr, (19, 120, 3, 8, 16, 0.2), BF16)
    pos = c.pos.view(c.M, c.topk).int()

    def view(t, off, pad):
        big = torch.full((t.shape[0], t.shape[1] + pad), 5, dtype=t.dtype, device="cuda")
        v = big[:, off:off + t.shape[1]]
        v.copy_(t)
        return v

    want = mr.moe_permute(c.x, c.ids, c.E, c.st, c.nt)[0][:c.n]
    comb = mr.moe_combine(c.y, pos, c.w, c.x)
    gy, gw = mr.moe_combine_grad(c.x, c.y, pos, c.w, c.st, c.nt)
    for off, pad in ((8, 8), (4, 12), (2, 6), (1, 9), (3, 3)):
        x, y = view(c.x, off, pad), view(c.y, off, pad)
        assert torch.equal(mr.moe_permute(x, c.ids, c.E, c.st, c.nt)[0][:c.n], want)
        assert torch.equal(mr.moe_combine(y, pos, c.w, x), comb)
        gy2, gw2 = mr.moe_combine_grad(x, y, pos, c.w, c.st, c.nt)
        assert torch.equal(gy2[:c.n], gy[:c.n])
        # (another word size sums in another order)
        ref.assert_within(gw2, gw.double(), 2 * 121 * 2.0 ** -24 * (c.x.abs().max() * c.y.abs().max() * 120).double().expand(gw.shape))


def test_offsets_beyond_32_bits(mr):
    """Rows behind 2^31 elements of the sorted positions, moved there and back."""
    M, K, topk, E, block = 90_000, 3136, 8, 16, 64
    ids = torch.stack([(torch.arange(topk) * 2 + (m & 1)) for m in range(2)]).int().repeat(M // 2, 1).cuda()
    st, ex, nt = mr.moe_sort(ids, E, block)
    x = torch.empty(M, K, dtype=torch.uint8, device="cuda").random_(0, 256)
    rows, pos = mr.moe_permute(x, ids, E, st, nt)
    assert rows.numel() > 1 << 31
    assert torch.equal(pos.view(-1).long(), ref.positions(st, int(nt), M * topk))
    for p in (0, 1, int(nt) - 1, int(nt) // 2, 700_001):
        f = int(st[p])
        assert torch.equal(rows[p], x[f // topk] if f < M * topk else torch.zeros_like(x[0]))


def test_refusals(mr):
    c = Case(mr, (4, 64, 2, 8, 16, 0.0), BF16)
    pos = c.pos.view(4, 2).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [lambda: mr.moe_permute(c.x, c.ids[:3], c.E, c.st, c.nt), lambda: mr.moe_permute(c.x.t(), c.ids, c.E, c.st, c.nt),
           lambda: mr.moe_permute(c.x.double(), c.ids, c.E, c.st, c.nt),
           lambda: mr.moe_permute(c.x, c.ids.long(), c.E, c.st, c.nt),
           lambda: mr.moe_permute(c.x, c.ids, c.E, c.st.long(), c.nt),
           lambda: mr.moe_permute(c.x, c.ids, c.E, c.st, c.nt, out=c.x),
           lambda: mr.moe_permute(c.x, c.ids, c.E, c.st, c.nt, positions=torch.empty(4, 3, **i32)),
           lambda: mr.moe_combine(c.y, pos.long()), lambda: mr.moe_combine(c.y, pos, c.w[:, :1]),
           lambda: mr.moe_combine(c.y, pos, c.w.double()), lambda: mr.moe_combine(c.y, pos, c.w, c.x[:3]),
           lambda: mr.moe_combine(c.y, pos, c.w, c.x.float()), lambda: mr.moe_combine(c.y.to(torch.uint8), pos),
           lambda: mr.moe_combine(c.y, pos, out=c.x[:, :32]),
           lambda: mr.moe_combine_grad(c.x, c.y[:5], pos, c.w, c.st, c.nt),
           lambda: mr.moe_combine_grad(c.x, c.y.float(), pos, c.w, c.st, c.nt),
           lambda: mr.moe_combine_grad(c.x, c.y, pos, c.w, c.st, c.nt, grad_weights=c.w[:, :1]),
           lambda: mr.moe_permute_grad(c.y, pos.view(-1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mr.MoeRouteUnsupported):
        mr.moe_combine(c.y, torch.zeros(2, 33, **i32))
    with pytest.raises(mr.MoeRouteError):  # rows that lie over one another
        mr.moe_combine(c.y[:1].expand(c.cap, 64), pos)


def test_captured_prepared_and_on_another_stream(mr):
    c = Case(mr, (33, 520, 4, 16, 16, 0.1), BF16)
    pos = c.pos.view(c.M, c.topk).int()
    perm = mr.PreparedPermute(c.x, c.ids, c.E, c.st, c.nt, out=out_rows(c, BF16, 0))
    comb = mr.PreparedCombine(c.y, pos, c.w, c.x)
    grad = mr.PreparedCombineGrad(c.x, c.y, pos, c.w, c.st, c.nt, out=out_rows(c, BF16, 0))
    back = mr.PreparedPermuteGrad(c.y, pos)
    calls = (perm, comb, grad, back)

    def flat(outs):
        return [t.clone() for o in outs for t in (o if isinstance(o, tuple) else (o,))]

    want = flat([f() for f in calls])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [f(side) for f in calls]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(got), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f in calls:
            f()
    x2 = ref.rows(77, c.M, c.K)
    c.x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    again = flat([f.out for f in calls])
    assert torch.equal(again[0], mr.moe_permute(x2, c.ids, c.E, c.st, c.nt, out=out_rows(c, BF16, 0))[0])
    assert torch.equal(again[2], mr.moe_combine(c.y, pos, c.w, x2))
    assert torch.equal(again[4], mr.moe_combine_grad(x2, c.y, pos, c.w, c.st, c.nt)[1])
