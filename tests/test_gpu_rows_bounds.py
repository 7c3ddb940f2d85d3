"""Rows to the experts and back: gradients of rows that start anywhere, held to the bound of their sums, and rows and
operands behind 2^31 elements."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import block_ref as ref  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def mr():
    import decode_expert_routing_gb300 as mr
    mr.load_library()
    return mr


def within(t, off):
    """t at element off of memory that holds NaN beside it."""
    flat = torch.full((t.numel() + 48,), float("nan"), dtype=t.dtype, device="cuda")
    view = flat[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return flat, view


def check_gradients(gy, gw, x, y, pos, w, n, dtype):
    """The formula's: grad_y by its two roundings, grad_weights by as many as it has terms."""
    M, topk = pos.shape
    f = (pos.view(-1) >= 0).nonzero()[:, 0]
    p, tok = pos.view(-1)[f].long(), f // topk
    want = torch.zeros(n, x.shape[1], dtype=torch.float64, device="cuda")
    want[p] = w.double().view(-1)[f, None] * x.double()[tok]
    tol = want.abs() * (torch.finfo(dtype).eps / 2 + 2.0 ** -23) + torch.finfo(dtype).smallest_normal * 2.0 ** -10
    ref.assert_within(gy[:n], want, tol, "grad_y")
    terms = x.double()[tok] * y.double()[p]
    wgw, mag = torch.zeros(M * topk, dtype=torch.float64, device="cuda"), torch.zeros(M * topk, dtype=torch.float64, device="cuda")
    wgw[f], mag[f] = terms.sum(1), terms.abs().sum(1)
    ref.assert_within(gw.view(-1), wgw, (x.shape[1] + 1) * 2.0 ** -24 * mag, "grad_weights")


@pytest.mark.parametrize("K", [1, 3, 8, 9, 33, 100, 130, 1001, 2050])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_gradients_of_rows_that_start_anywhere(mr, K, dtype):
    """grad_out, y and grad_y start at elements of their own each, in place and not."""
    M, E, topk = 37, 8, 3
    ids, w = ref.routed(M, E, topk, 2, 0.2)
    st, _, nt = mr.moe_sort(ids, E, 8)
    n, cap = int(nt), st.numel()
    pos = ref.positions(st, n, M * topk).view(M, topk).int()
    x, y = ref.rows(1, M, K, dtype), ref.rows(3, cap, K, dtype)
    for off in (0, 1, 2, 5, 8, 15):
        for there in (0, 3, 4, 7):
            flat, out = within(torch.zeros_like(y), 16 - off)
            gy, gw = mr.moe_combine_grad(within(x, off)[1], within(y, there)[1], pos, w, st, nt, out=out)
            check_gradients(gy, gw, x, y, pos, w, n, dtype)
            assert (gy[n:] == 0).all() and flat.isnan().sum() == 48
        flat, out = within(y, off)
        gy, gw = mr.moe_combine_grad(within(x, 16 - off)[1], out, pos, w, st, nt, out=out)
        check_gradients(gy, gw, x, y, pos, w, n, dtype)
        assert torch.equal(gy[n:], y[n:]) and flat.isnan().sum() == 48


@pytest.mark.parametrize("K", [120, 121, 514])
@pytest.mark.parametrize("off,pad", [(0, 0), (8, 8), (4, 12), (2, 6), (1, 9), (3, 3), (0, 1)])
def test_gradients_of_strided_rows(mr, K, off, pad):
    M, E, topk = 19, 8, 3
    ids, w = ref.routed(M, E, topk, 4, 0.2)
    st, _, nt = mr.moe_sort(ids, E, 16)
    n, cap = int(nt), st.numel()
    pos = ref.positions(st, n, M * topk).view(M, topk).int()
    x, y = ref.rows(1, M, K), ref.rows(3, cap, K)

    def view(t):
        big = torch.full((t.shape[0], K + off + pad), float("nan"), dtype=t.dtype, device="cuda")
        big[:, off:off + K] = t
        return big[:, off:off + K]

    gy, gw = mr.moe_combine_grad(view(x), view(y), pos, w, st, nt)
    check_gradients(gy, gw, x, y, pos, w, n, BF16)


@pytest.mark.parametrize("K", [30_000, 30_001])
def test_rows_behind_2_to_the_31_elements(mr, K):
    """There, back and the gradients, of rows that are moved by 16-byte words and of rows that start anywhere."""
    M, topk, E, block = 9000, 8, 8, 16
    gen = torch.Generator("cpu").manual_seed(1)
    ids = torch.argsort(torch.rand(M, E, generator=gen), 1).int().cuda()  # every token at every expert
    w = (torch.rand(M, topk, generator=gen) * 2 - 0.5).cuda()
    st, _, nt = mr.moe_sort(ids, E, block)
    n, cap = int(nt), st.numel()
    pos = ref.positions(st, n, M * topk).view(M, topk).int()
    assert (n - 20) * K > 1 << 31
    x = torch.empty(M, K, dtype=BF16, device="cuda").normal_()
    rows, got = mr.moe_permute(x, ids, E, st, nt)
    assert torch.equal(got, pos)
    some = torch.tensor([0, 1, 8, 4500, 8520, 8530, *range(8980, 9000)], device="cuda")
    p = pos[some].long()
    assert p.max() * K > 1 << 31
    assert torch.equal(rows[p.view(-1)], x[some].repeat_interleave(topk, 0))
    for i in range(0, cap, 8000):
        rows[i:i + 8000].normal_()
    y64, w64 = rows[p.view(-1)].double().unflatten(0, (-1, topk)), w[some].double()[..., None]

    def check(out, add):
        want, mag = (y64 * w64).sum(1), (y64 * w64).abs().sum(1)
        if add is not None:
            want, mag = want + add.double(), mag + add.double().abs()
        tol = (topk + 1) * 2.0 ** -24 * mag
        ref.assert_within(out, want, tol + 2.0 ** -8 * (want.abs() + tol) + 2.0 ** -133)

    check(mr.moe_combine(rows, pos, w, x)[some], x[some])
    check(mr.moe_combine(rows, pos[some].clone(), w[some].clone()), None)  # (few tokens: another kernel)
    last = rows[n:].clone()
    want_rows = rows[p.view(-1)].clone()
    gy, gw = mr.moe_combine_grad(x, rows, pos, w, st, nt, out=rows)
    assert torch.equal(gy[n:], last)
    want = w64 * x[some].double()[:, None]
    ref.assert_within(gy[p.view(-1)].view(want.shape), want, want.abs() * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133)
    terms = x[some].double().repeat_interleave(topk, 0) * want_rows.double()
    ref.assert_within(gw[some].view(-1), terms.sum(1), (K + 1) * 2.0 ** -24 * terms.abs().sum(1))


@pytest.mark.parametrize("K", [96, 97])
def test_row_strides_whose_offsets_pass_2_to_the_31(mr, K):
    M, topk, E, block, ld = 9000, 8, 8, 16, 32_776
    ids = torch.arange(E).int().repeat(M, 1).cuda()
    w = torch.rand(M, topk, generator=torch.Generator("cpu").manual_seed(2)).cuda()
    st, _, nt = mr.moe_sort(ids, E, block)
    n, cap = int(nt), st.numel()
    pos = ref.positions(st, n, M * topk).view(M, topk).int()
    x, y = ref.rows(1, M, K), ref.rows(2, cap, K)
    wide = torch.empty(cap, ld, dtype=BF16, device="cuda")[:, :K]
    wide.copy_(y)
    assert (n - 20) * ld > 1 << 31
    assert torch.equal(mr.moe_combine(wide, pos, w, x), mr.moe_combine(y, pos, w, x))
    zero = torch.zeros_like(y)
    gy, gw = mr.moe_combine_grad(x, wide, pos, w, st, nt, out=zero)
    check_gradients(gy, gw, x, y, pos, w, n, BF16)


@pytest.mark.parametrize("M,ld", [(16, 1 << 28), (40, 1 << 26), (300, 1 << 23), (2000, 1 << 21)])
@pytest.mark.parametrize("R", [70, 700])
def test_fp8_rows_whose_offsets_pass_2_to_the_31(mr, M, ld, R):
    """Rows of x far apart (and in the first two the weight's too), every variant of the product."""
    K = 400
    q, xs, w, ws = ref.codes(1, M, K), ref.scales(2, M, 4), ref.codes(3, R, K), ref.scales(4, -(-R // 128), 4)
    far = torch.empty(M, ld, dtype=torch.uint8, device="cuda")[:, :K]
    far.copy_(q)
    assert M * ld > (1 << 31) - 1
    want = mr.fp8_gemm(q, xs, w, ws, out_dtype=F32)
    ref.assert_within(want, *ref.product(q, xs, w, ws, F32))
    assert torch.equal(mr.fp8_gemm(far, xs, w, ws, out_dtype=F32), want)
    del far
    if M <= 40:
        far = torch.empty(R, (1 << 32) // R // 16 * 16, dtype=torch.uint8, device="cuda")[:, :K]
        far.copy_(w)
        assert torch.equal(mr.fp8_gemm(q, xs, far, ws, out_dtype=F32), want)
        far = torch.empty(M, (1 << 31) // M, dtype=F32, device="cuda")[:, :R]
        assert torch.equal(mr.fp8_gemm(q, xs, w, ws, out=far), want)
