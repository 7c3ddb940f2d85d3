"""mx_gemm, moe_gate_up and moe_down on the GPU against the definitions in 64
bits (expert_ref.py holds them with their error bounds)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402

FMTS = ["mxfp8", "mxfp4"]
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def mr():
    from decode_expert_routing_gb300 import build
    build.build()
    import decode_expert_routing_gb300 as m
    m.load_library()
    m.set_launch_flags(0)
    yield m
    assert m.device_error(clear=True) == m.MR_OK


def quant(mr, x, fmt):
    return (mr.mxfp8_quant if fmt == "mxfp8" else mr.mxfp4_quant)(x)


# ------------------------------------------------------------------ mx_gemm

GEMM = [  # M, R, K: one row and column, odd sizes, K inside a stage, tiles of one and several row groups
    (1, 1, 32), (1, 128, 128), (1, 130, 768), (3, 100, 96), (15, 128, 256), (16, 64, 512), (17, 257, 160),
    (33, 128, 1024), (100, 192, 2080), (128, 128, 256), (129, 384, 512), (240, 128, 384), (255, 128, 512),
    (256, 256, 640), (257, 128, 512), (700, 520, 1056), (1, 6144, 768), (5, 40000, 64),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,R,K", GEMM)
def test_mx_gemm(mr, fmt, M, R, K):
    x, w = ref.random_mx((M, K), fmt, M + K), ref.random_mx((R, K), fmt, R)
    W = mr.MxWeight(*w, fmt)
    xv, wv = ref.value64(*x, fmt), ref.value64(*w, fmt)
    for dtype in (torch.float32, BF16):
        out = mr.mx_gemm(*x, W, out_dtype=dtype)
        ref.assert_close(out, *ref.product(xv, wv, dtype), f"{fmt} {dtype}")


@pytest.mark.parametrize("fmt", FMTS)
def test_mx_gemm_small_integers_are_exact(mr, fmt):
    """Values of a few bits with scales 2^-2 .. 2^2: every sum fits fp32, so
    any misplaced element or scale shows as a wrong integer."""
    M, R, K = 150, 300, 768
    x, w = ref.random_mx((M, K), fmt, 1, 125, 130), ref.random_mx((R, K), fmt, 2, 125, 130)
    if fmt == "mxfp8":  # codes of 0, 1, 1.5, 2, 3, 4, 6, 8 and their negatives
        lut = torch.tensor([0x00, 0x38, 0x3C, 0x40, 0x44, 0x48, 0x4C, 0x50], dtype=torch.uint8, device="cuda")
        x = ((lut[(x[0] & 7).long()] | (x[0] & 128)), x[1])
        w = ((lut[(w[0] & 7).long()] | (w[0] & 128)), w[1])
    out = mr.mx_gemm(*x, mr.MxWeight(*w, fmt), out_dtype=torch.float32)
    assert torch.equal(out.double(), ref.value64(*x, fmt) @ ref.value64(*w, fmt).T)


@pytest.mark.parametrize("fmt", FMTS)
def test_mx_gemm_strides_and_extreme_scales(mr, fmt):
    M, R, K = 37, 200, 512
    x, w = ref.random_mx((M, K), fmt, 3, 0, 40), ref.random_mx((R, K), fmt, 4, 200, 254)
    qb = torch.empty(M, x[0].shape[1] + 48, dtype=torch.uint8, device="cuda")
    sb = torch.empty(M, K // 32 + 5, dtype=torch.uint8, device="cuda")
    ob = torch.full((M + 2, R + 7), 7.0, device="cuda")
    q, s, out = qb[:, 16:16 + x[0].shape[1]], sb[:, 3:3 + K // 32], ob[1:-1, 2:2 + R]
    q.copy_(x[0])
    s.copy_(x[1])
    mr.mx_gemm(q, s, mr.MxWeight(*w, fmt), out=out)
    ref.assert_close(out, *ref.product(ref.value64(*x, fmt), ref.value64(*w, fmt), torch.float32))
    assert (ob[0] == 7).all() and (ob[-1] == 7).all() and (ob[:, :2] == 7).all() and (ob[:, 2 + R:] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_mx_gemm_nan_stays_in_its_row(mr, fmt):
    """A scale byte 255 (NaN) reaches the results that use it and no others."""
    M, R, K = 20, 140, 256
    x, w = ref.random_mx((M, K), fmt, 5), ref.random_mx((R, K), fmt, 6)
    clean = mr.mx_gemm(*x, mr.MxWeight(*w, fmt), out_dtype=torch.float32)
    x[1][7, 3] = 255
    w[1][131, 0] = 255
    out = mr.mx_gemm(*x, mr.MxWeight(*w, fmt), out_dtype=torch.float32)
    bad = torch.zeros(M, R, dtype=torch.bool, device="cuda")
    bad[7] = True
    bad[:, 131] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad])


# ------------------------------------------------------------------ the experts

def routed(M, E, topk, seed, invalid=0.0, skew=0.0):
    g = torch.Generator("cpu").manual_seed(seed)
    logits = torch.randn(M, E, generator=g) + skew * torch.randn(E, generator=g)
    ids = logits.topk(topk, 1).indices.int()
    ids[torch.rand(M, topk, generator=g) < invalid] = -1
    wts = torch.rand(M, topk, generator=g)
    return ids.cuda(), (wts / wts.sum(1, keepdim=True)).cuda()


EXPERTS = [  # M, E, topk, K, I, block, share of slots without an expert, skew of the choice
    (1, 8, 2, 128, 32, 16, 0.0, 0), (1, 1, 1, 32, 32, 1, 0.0, 0), (7, 16, 4, 256, 64, 16, 0.0, 0),
    (16, 128, 8, 512, 96, 16, 0.2, 0), (33, 5, 3, 416, 160, 8, 0.3, 1), (64, 8, 8, 384, 64, 32, 0.0, 0),
    (100, 3, 2, 640, 32, 5, 0.1, 2), (300, 2, 2, 256, 128, 64, 0.0, 0), (513, 9, 3, 288, 64, 64, 0.05, 2),
    (40, 1024, 16, 128, 32, 16, 0.0, 0), (257, 4, 1, 768, 192, 256, 0.0, 3),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,K,I,block,invalid,skew", EXPERTS)
def test_gate_up(mr, fmt, M, E, topk, K, I, block, invalid, skew):
    ids, _ = routed(M, E, topk, M + E, invalid, skew)
    st, ex, _ = mr.moe_sort(ids, E, block)
    w = ref.random_mx((E, 2 * I, K), fmt, I, 117, 122)
    W = mr.MxWeight(*w, fmt, gate_up=True)
    wv = ref.value64(*w, fmt)
    x = torch.randn(M, K, generator=torch.Generator("cpu").manual_seed(M)).to(BF16).cuda()
    q = quant(mr, x, fmt)
    xv = ref.value64(*q, fmt)
    act, tol = ref.gate_up(xv, wv, st, ex, topk, block, M * topk, False)
    real = (st < M * topk)
    out = torch.full((st.numel(), I), 5.0, dtype=BF16, device="cuda")
    mr.moe_gate_up(*q, W, st, ex, topk, block, out=out)
    half = ref.half_step(BF16)
    ref.assert_close(out[real], act[real], (tol + half * (act.abs() + tol))[real], "token order")
    assert (out[~real] == 5).all(), "rows without an assignment were written"
    # the rows in sorted order: the same bits
    _, _, _, qs, ss = mr.moe_sort_quant(ids, x, E, block, quant=fmt, sorted_rows=True)
    out2 = torch.full_like(out, 5.0)
    mr.moe_gate_up(qs, ss, W, st, ex, topk, block, num_tokens=M, sorted_rows=True, out=out2)
    assert torch.equal(out, out2)
    # quantised in the epilogue: the bits of the quantiser on the bf16 rows
    for qf in FMTS:
        c, s = mr.moe_gate_up(*q, W, st, ex, topk, block, quant=qf)
        rc, rs = quant(mr, out, qf)
        assert torch.equal(c[real], rc[real]) and torch.equal(s[real], rs[real]), qf


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,R,I,block,invalid,skew", EXPERTS + [(9, 16, 4, 130, 64, 16, 0.3, 0),
                                                                      (70, 6, 2, 33, 96, 16, 0.0, 0)])
def test_down(mr, fmt, M, E, topk, R, I, block, invalid, skew):
    ids, wts = routed(M, E, topk, M + E, invalid, skew)
    st, ex, _ = mr.moe_sort(ids, E, block)
    w = ref.random_mx((E, R, I), fmt, I, 117, 122)
    a = ref.random_mx((st.numel(), I), fmt, R)
    add = torch.randn(M, R, generator=torch.Generator("cpu").manual_seed(R)).to(BF16).cuda()
    W = mr.MxWeight(*w, fmt)
    av, wv = ref.value64(*a, fmt), ref.value64(*w, fmt)
    half = ref.half_step(BF16)
    scratch = mr.ExpertScratch(M, topk, R)
    for extra in (None, add):
        want, tol = ref.down(av, wv, st, ex, ids, wts, block, E, extra)
        out = mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra, scratch=scratch)
        ref.assert_close(out, want, tol + half * (want.abs() + tol))
        again = mr.moe_down(*a, W, ids, wts, st, ex, block, add=extra, scratch=scratch)
        assert torch.equal(out, again)
    inplace = add.clone()
    mr.moe_down(*a, W, ids, wts, st, ex, block, add=inplace, out=inplace, scratch=scratch)
    assert torch.equal(inplace, out)


def test_down_tokens_without_experts(mr):
    M, E, topk, R, I, block = 6, 4, 2, 256, 64, 16
    ids = torch.full((M, topk), -1, dtype=torch.int32, device="cuda")
    ids[2, 1] = 3
    ids[4] = 7  # past the last expert
    wts = torch.full((M, topk), float("nan"), device="cuda")  # a weight nobody uses may be anything
    wts[2] = 0.5
    st, ex, _ = mr.moe_sort(ids, E, block)
    a, w = ref.random_mx((st.numel(), I), "mxfp8", 1), ref.random_mx((E, R, I), "mxfp8", 2)
    out = mr.moe_down(*a, mr.MxWeight(*w), ids, wts, st, ex, block)
    rest = [m for m in range(M) if m != 2]
    assert (out[rest] == 0).all() and (out[2] != 0).any()
    # no token has an expert: nothing but add
    ids[2, 1] = -1
    st, ex, _ = mr.moe_sort(ids, E, block)
    add = torch.ones(M, R, dtype=BF16, device="cuda")
    assert torch.equal(mr.moe_down(*a, mr.MxWeight(*w), ids, wts, st, ex, block, add=add), add)


def test_the_same_expert_twice(mr):
    """Every slot of every token on one expert: 8 M rows in its run."""
    M, E, topk, K, I, block = 45, 4, 8, 256, 64, 16
    ids = torch.full((M, topk), 2, dtype=torch.int32, device="cuda")
    wts = torch.rand(M, topk, generator=torch.Generator("cpu").manual_seed(0)).cuda()
    st, ex, _ = mr.moe_sort(ids, E, block)
    w13, w2 = ref.random_mx((E, 2 * I, K), "mxfp8", 1, 117, 122), ref.random_mx((E, K, I), "mxfp8", 2, 117, 122)
    q = mr.mxfp8_quant(torch.randn(M, K, generator=torch.Generator("cpu").manual_seed(3)).to(BF16).cuda())
    act, tol = ref.gate_up(ref.value64(*q, "mxfp8"), ref.value64(*w13, "mxfp8"), st, ex, topk, block, M * topk, False)
    out = mr.moe_gate_up(*q, mr.MxWeight(*w13, gate_up=True), st, ex, topk, block)
    real = st < M * topk
    ref.assert_close(out[real], act[real], (tol + ref.half_step(BF16) * (act.abs() + tol))[real])
    a = mr.moe_gate_up(*q, mr.MxWeight(*w13, gate_up=True), st, ex, topk, block, quant="mxfp8")
    a[0][~real], a[1][~real] = 0, 0  # (the reference reads every row)
    want, tol = ref.down(ref.value64(*a, "mxfp8"), ref.value64(*w2, "mxfp8"), st, ex, ids, wts, block, E)
    got = mr.moe_down(*a, mr.MxWeight(*w2), ids, wts, st, ex, block)
    ref.assert_close(got, want, tol + ref.half_step(BF16) * (want.abs() + tol))


def layer(mr, M, E, topk, K, I, block, fmt, seed):
    """One MoE layer as a decode step runs it: route, gate/up, down."""
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(BF16).cuda()
    gate = (torch.randn(E, K, generator=g) * 0.02).to(BF16).cuda()
    w13 = ref.random_mx((E, 2 * I, K), fmt, seed + 1, 116, 120)
    w2 = ref.random_mx((E, K, I), fmt, seed + 2, 116, 120)
    W13, W2 = mr.MxWeight(*w13, fmt, gate_up=True), mr.MxWeight(*w2, fmt)
    route = mr.PreparedRoute(x, gate, topk, block, quant=fmt)
    r = route.out
    up = mr.PreparedGateUp(r["q"], r["scale"], W13, r["sorted_token_ids"], r["expert_ids"], topk, block, quant=fmt)
    down = mr.PreparedDown(*up.out, W2, r["topk_ids"], r["topk_weights"], r["sorted_token_ids"], r["expert_ids"], block)
    return x, w13, w2, route, up, down


def check_layer(mr, x, w13, w2, route, up, down, topk, block, E, fmt):
    r = route.out
    st, ex = r["sorted_token_ids"], r["expert_ids"]
    M = x.shape[0]
    q = quant(mr, x, fmt)
    act, tol = ref.gate_up(ref.value64(*q, fmt), ref.value64(*w13, fmt), st, ex, topk, block, M * topk, False)
    real = st < M * topk
    # stage 1 quantises: within its bound plus a whole code step of the block's scale (a sum near the border of
    # two codes may fall on either side; a block whose largest element crosses a power of two takes twice the step)
    got = torch.zeros_like(act)
    got[real] = ref.value64(up.out[0][real], up.out[1][real], fmt)
    amax = act.abs().unflatten(1, (-1, 32)).amax(2, keepdim=True)
    step = amax.expand(-1, -1, 32).flatten(1) * (2.0 ** -3 if fmt == "mxfp8" else 2.0 ** -1)
    ref.assert_close(got[real], act[real], (tol * 2 + 2.0 ** -8 * act.abs() + step)[real])
    want, tol = ref.down(got, ref.value64(*w2, fmt), st, ex, r["topk_ids"], r["topk_weights"], block, E)
    ref.assert_close(down.out, want, tol + ref.half_step(BF16) * (want.abs() + tol))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 16, 40])
def test_route_then_experts(mr, fmt, M):
    E, topk, K, I, block = 64, 4, 1024, 128, 16
    x, w13, w2, route, up, down = layer(mr, M, E, topk, K, I, block, fmt, M)
    for call in (route, up, down):
        call()
    check_layer(mr, x, w13, w2, route, up, down, topk, block, E, fmt)


def test_captured_layer_replays_on_new_inputs(mr):
    E, topk, K, I, block, M, fmt = 64, 4, 1024, 128, 16, 24, "mxfp8"
    x, w13, w2, route, up, down = layer(mr, M, E, topk, K, I, block, fmt, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for call in (route, up, down):
            call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for call in (route, up, down):
            call()
    for seed in range(3):
        x.copy_(torch.randn(M, K, generator=torch.Generator("cpu").manual_seed(seed)).to(BF16))
        g.replay()
        torch.cuda.synchronize()
        got = down.out.clone()
        check_layer(mr, x, w13, w2, route, up, down, topk, block, E, fmt)
        for call in (route, up, down):  # the same bits outside the graph
            call()
        assert torch.equal(down.out, got)


def test_two_streams_with_their_own_scratch(mr):
    E, topk, K, I, block, fmt = 32, 4, 1024, 128, 16, "mxfp4"
    layers = [layer(mr, M, E, topk, K, I, block, fmt, M) for M in (8, 31)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (_, _, _, route, up, down) in zip(streams, layers):
            for call in (route, up, down):
                call(s)
    torch.cuda.synchronize()
    for x, w13, w2, route, up, down in layers:
        check_layer(mr, x, w13, w2, route, up, down, topk, block, E, fmt)


def test_pdl_flag_gives_the_same_bits(mr):
    E, topk, K, I, block, fmt, M = 32, 4, 1024, 128, 16, "mxfp8", 16
    _, _, _, route, up, down = layer(mr, M, E, topk, K, I, block, fmt, 9)
    for call in (route, up, down):
        call()
    want = down.out.clone()
    mr.set_launch_flags(mr.LAUNCH_PDL)
    try:
        for _ in range(20):
            for call in (route, up, down):
                call()
        assert torch.equal(down.out, want)
    finally:
        mr.set_launch_flags(0)


@pytest.mark.parametrize("fmt", FMTS)
def test_one_expert_of_many_takes_all(mr, fmt):
    """The largest tables beside the widest tiles."""
    M, E, topk, K, I, block = 601, 1024, 1, 416, 64, 64
    ids = torch.full((M, topk), 1000, dtype=torch.int32, device="cuda")
    wts = torch.full((M, topk), 0.5, device="cuda")
    st, ex, _ = mr.moe_sort(ids, E, block)
    w13, w2 = ref.random_mx((E, 2 * I, K), fmt, 1, 117, 122), ref.random_mx((E, K, I), fmt, 2, 117, 122)
    q = quant(mr, torch.randn(M, K, generator=torch.Generator("cpu").manual_seed(3)).to(BF16).cuda(), fmt)
    one = [t[1000:1001].contiguous() for t in w13], [t[1000:1001].contiguous() for t in w2]
    act, tol = ref.swiglu(ref.value64(*q, fmt), ref.value64(one[0][0][0], one[0][1][0], fmt))
    out = mr.moe_gate_up(*q, mr.MxWeight(*w13, fmt, gate_up=True), st, ex, topk, block)
    ref.assert_close(out[:M], act, tol + ref.half_step(BF16) * (act.abs() + tol))
    c, s = mr.moe_gate_up(*q, mr.MxWeight(*w13, fmt, gate_up=True), st, ex, topk, block, quant=fmt)
    want = ref.value64(c[:M], s[:M], fmt) @ ref.value64(one[1][0][0], one[1][1][0], fmt).T
    got = mr.moe_down(c, s, mr.MxWeight(*w2, fmt), ids, wts, st, ex, block)
    d = ref.sum_bound(I) * (ref.value64(c[:M], s[:M], fmt).abs() @ ref.value64(one[1][0][0], one[1][1][0], fmt).abs().T)
    half = ref.half_step(BF16)
    tol = 0.5 * (d + half * (want.abs() + d)) + 2.0 ** -23 * want.abs()
    ref.assert_close(got, 0.5 * want, tol + half * (0.5 * want.abs() + tol))


def test_offsets_past_32_bits(mr):
    """420 000 assignments: more column tiles than the kernel lists, and rows
    of y and of the gate/up output past 2^31 elements."""
    fmt, M, E, topk, K, I, block = "mxfp4", 70000, 4, 6, 32, 5216, 64
    g = torch.Generator("cuda").manual_seed(1)
    ids = torch.randint(0, E, (M, topk), generator=g, device="cuda", dtype=torch.int32)
    wts = torch.rand(M, topk, generator=g, device="cuda")
    st, ex, _ = mr.moe_sort(ids, E, block)
    assert st.numel() * I > 1 << 31
    w13 = ref.random_mx((E, 2 * I, K), fmt, 1, 117, 122)
    q = quant(mr, torch.randn(M, K, generator=g, device="cuda").to(BF16), fmt)
    out = mr.moe_gate_up(*q, mr.MxWeight(*w13, fmt, gate_up=True), st, ex, topk, block)
    pos = torch.cat([torch.arange(40, device="cuda"), torch.nonzero(st < M * topk)[-40:, 0]])
    f, e = st[pos].long(), ex[pos // block].long()
    xv, wv = ref.value64(*q, fmt), ref.value64(*w13, fmt)
    for i in range(pos.numel()):
        act, tol = ref.swiglu(xv[f[i] // topk][None], wv[e[i]])
        ref.assert_close(out[pos[i]][None], act, tol + ref.half_step(BF16) * (act.abs() + tol))
    del out
    I, R = 32, 5216  # the other way round: y has M * topk rows of R
    w2 = ref.random_mx((E, R, I), fmt, 2, 117, 122)
    a = torch.randint(0, 256, (st.numel(), I // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(120, 126, (st.numel(), 1), generator=g, device="cuda", dtype=torch.uint8)
    got = mr.moe_down(a, s, mr.MxWeight(*w2, fmt), ids, wts, st, ex, block)
    place = torch.empty(M * topk, dtype=torch.long, device="cuda")
    real = torch.nonzero(st < M * topk)[:, 0]
    place[st[real].long()] = real
    wv = ref.value64(*w2, fmt)
    for m in (0, 1, 777, M // 2, M - 2, M - 1):
        p = place[m * topk:(m + 1) * topk]
        rows = ref.value64(a[p], s[p], fmt)
        y = torch.stack([rows[j] @ wv[int(ids[m, j])].T for j in range(topk)])
        d = ref.sum_bound(I) * torch.stack([rows[j].abs() @ wv[int(ids[m, j])].abs().T for j in range(topk)])
        d = d + ref.half_step(BF16) * (y.abs() + d)
        w = wts[m].double()[:, None]
        want, tol = (w * y).sum(0), (w * d).sum(0) + (topk + 1) * 2.0 ** -24 * (w * y.abs()).sum(0)
        ref.assert_close(got[m], want, tol + ref.half_step(BF16) * (want.abs() + tol))


def test_weights_past_32_bits(mr):
    """Weight codes of more than 4 GB: the last expert's."""
    fmt, M, E, topk, K, I, block = "mxfp8", 5, 700, 2, 4096, 768, 16
    g = torch.Generator("cuda").manual_seed(2)
    codes = torch.randint(0, 120, (E, 2 * I, K), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.randint(112, 116, (E, 2 * I, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    assert codes.numel() > 1 << 32
    W = mr.MxWeight(codes, scale, fmt, gate_up=True)
    ids = torch.tensor([[699, 3], [698, 699], [0, 699], [350, 698], [699, 1]], dtype=torch.int32, device="cuda")
    st, ex, _ = mr.moe_sort(ids, E, block)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16) * 0.1
    q = quant(mr, x, fmt)
    out = mr.moe_gate_up(*q, W, st, ex, topk, block)
    xv = ref.value64(*q, fmt)
    pos, f = ref.used_positions(st, M * topk)
    for p, a in zip(pos.tolist(), f.tolist()):
        e = int(ex[p // block])
        act, tol = ref.swiglu(xv[a // topk][None], ref.value64(codes[e], scale[e], fmt))
        ref.assert_close(out[p][None], act, tol + ref.half_step(BF16) * (act.abs() + tol))


def test_scales_at_any_alignment(mr):
    """Scale rows whose length, stride and first byte are odd, at the ends of their array."""
    for fmt in FMTS:
        for K, extra, first in ((2976, 0, 0), (2976, 2, 1), (160, 0, 3), (32, 0, 1), (1056, 5, 2)):
            M, R = 37, 130
            x, w = ref.random_mx((M, K), fmt, K), ref.random_mx((R, K), fmt, 4)
            kb = K // 32
            buf = torch.full((first + M * (kb + extra),), 255, dtype=torch.uint8, device="cuda")
            s = buf[first:].view(M, kb + extra)[:, :kb]
            s.copy_(x[1])
            out = mr.mx_gemm(x[0], s, mr.MxWeight(*w, fmt), out_dtype=torch.float32)
            ref.assert_close(out, *ref.product(ref.value64(*x, fmt), ref.value64(*w, fmt), torch.float32), f"{fmt} {K}")


@pytest.mark.parametrize("M", [8, 300])
def test_a_wait_that_runs_out_is_reported(mr, M):
    """The first stage expects bytes that nobody sends: the call ends, the flag tells, and the next call is right."""
    x, w = ref.random_mx((M, 512), "mxfp8", 1), ref.random_mx((256, 512), "mxfp8", 2)
    W = mr.MxWeight(*w)
    want = mr.mx_gemm(*x, W)
    torch.cuda.synchronize()
    try:
        mr.set_wait_limit_ns(20_000_000)
        mr.set_launch_flags(mr.LAUNCH_TEST_STALL)
        mr.mx_gemm(*x, W)
        torch.cuda.synchronize()
    finally:
        mr.set_launch_flags(0)
        mr.set_wait_limit_ns(1_000_000_000)
    assert mr.device_error(clear=True) == mr.MR_ERR_TIMEOUT
    assert torch.equal(mr.mx_gemm(*x, W), want)
    assert mr.device_error() == mr.MR_OK


# ------------------------------------------------------------------ few tiles of a long K: several CTAs to a tile

LONG = [  # M, R, K: one row of tiles and several, odd numbers of k-blocks, several column tiles
    (1, 128, 6144), (8, 256, 6144), (33, 1000, 6144), (33, 6144, 6144), (64, 500, 4128), (129, 130, 12320),
    (250, 300, 2976), (256, 100, 20480), (600, 200, 8192), (1, 1, 16416),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,R,K", LONG)
def test_mx_gemm_of_few_tiles(mr, fmt, M, R, K):
    test_mx_gemm(mr, fmt, M, R, K)
    x, W = ref.random_mx((M, K), fmt, 1), mr.MxWeight(*ref.random_mx((R, K), fmt, 2), fmt)
    assert torch.equal(mr.mx_gemm(*x, W), mr.mx_gemm(*x, W))


@pytest.mark.parametrize("fmt,M,R,K", [
    ("mxfp8", 895, 1420, 4736), ("mxfp4", 895, 1420, 9472), ("mxfp8", 520, 1700, 6144), ("mxfp8", 400, 700, 8192)])
def test_mx_gemm_of_few_tiles_of_many_rows(mr, fmt, M, R, K):
    """Where narrower tiles would fill the CTAs, but not the clusters that share a tile's K range."""
    test_mx_gemm(mr, fmt, M, R, K)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,E,topk,K,I,block,invalid,skew", [
    (1, 8, 2, 6144, 64, 16, 0.0, 0), (5, 4, 2, 4128, 96, 16, 0.3, 0), (40, 2, 2, 5152, 32, 8, 0.0, 0),
    (130, 3, 1, 12320, 160, 64, 0.1, 2), (3, 1, 1, 8192, 32, 1, 0.0, 0), (300, 1, 1, 6176, 64, 128, 0.0, 0)])
def test_experts_of_few_tiles(mr, fmt, M, E, topk, K, I, block, invalid, skew):
    test_gate_up(mr, fmt, M, E, topk, K, I, block, invalid, skew)
    test_down(mr, fmt, M, E, topk, I + 5, K, block, invalid, skew)


def test_a_wait_of_one_slice_that_runs_out_is_reported(mr):
    """As above where the CTAs of a cluster share a tile's K range."""
    M, E, topk, K, I, block = 8, 2, 1, 6144, 64, 16
    x, w = ref.random_mx((M, K), "mxfp8", 1), ref.random_mx((256, K), "mxfp8", 2)
    ids, wts = routed(M, E, topk, 1)
    st, ex, _ = mr.moe_sort(ids, E, block)
    gemm = mr.PreparedMxGemm(*x, mr.MxWeight(*w))
    up = mr.PreparedGateUp(*x, mr.MxWeight(*ref.random_mx((E, 2 * I, K), "mxfp8", 3, 117, 122), gate_up=True), st, ex,
                           topk, block)
    a = ref.random_mx((st.numel(), K), "mxfp8", 4)
    down = mr.PreparedDown(*a, mr.MxWeight(*ref.random_mx((E, I, K), "mxfp8", 5)), ids, wts, st, ex, block)
    up.out.zero_()
    for call in (gemm, up, down):
        want = call().clone()
        torch.cuda.synchronize()
        try:
            mr.set_wait_limit_ns(20_000_000)
            mr.set_launch_flags(mr.LAUNCH_TEST_STALL)
            call()
            torch.cuda.synchronize()
        finally:
            mr.set_launch_flags(0)
            mr.set_wait_limit_ns(1_000_000_000)
        assert mr.device_error(clear=True) == mr.MR_ERR_TIMEOUT
        assert torch.equal(call(), want)
        assert mr.device_error() == mr.MR_OK


# ------------------------------------------------------------------ streams and graphs

def test_down_on_another_stream_without_scratch(mr):
    """The scratch that the call makes itself stays its own until that stream is done with it."""
    M, E, topk, R, I, block = 64, 8, 4, 1024, 256, 16
    ids, wts = routed(M, E, topk, 3)
    st, ex, _ = mr.moe_sort(ids, E, block)
    a, W = ref.random_mx((st.numel(), I), "mxfp8", 1), mr.MxWeight(*ref.random_mx((E, R, I), "mxfp8", 2))
    want = mr.moe_down(*a, W, ids, wts, st, ex, block)
    n = mr.ExpertScratch(M, topk, R).nbytes
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        out = torch.zeros_like(want)
        torch.cuda.current_stream().synchronize()
        mr.moe_down(*a, W, ids, wts, st, ex, block, out=out, stream=stream)
        other = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((o == 255).all() for o in other), "the call's scratch was handed on before it ran"


@pytest.mark.parametrize("R", [64, 1024, 1032, 130])
def test_down_touches_its_own_rows_of_the_scratch_only(mr, R):
    """A call of fewer tokens than the scratch is made for, again and again beside other uses of its rest."""
    M, E, topk, I, block = 19, 8, 3, 256, 16
    ids, wts = routed(M, E, topk, 3, invalid=0.2)
    st, ex, _ = mr.moe_sort(ids, E, block)
    a, W = ref.random_mx((st.numel(), I), "mxfp4", 1), mr.MxWeight(*ref.random_mx((E, R, I), "mxfp4", 2), "mxfp4")
    want = mr.moe_down(*a, W, ids, wts, st, ex, block)
    scratch = mr.ExpertScratch(4 * M, topk, R)
    rest = scratch.tensor[M * topk * R * 2:]
    for i in range(20):
        rest.fill_(i)
        assert torch.equal(mr.moe_down(*a, W, ids, wts, st, ex, block, scratch=scratch), want)
        assert (rest == i).all()


def test_captured_after_copies_and_a_fork(mr):
    """In a graph the calls follow a copy, another stream's work and each other."""
    M, E, topk, K, I, block, fmt = 12, 8, 2, 512, 64, 16, "mxfp8"
    ids, wts = routed(M, E, topk, 5)
    st, ex, _ = mr.moe_sort(ids, E, block)
    xs = [ref.random_mx((M, K), fmt, i) for i in range(3)]
    q, sc = torch.zeros_like(xs[0][0]), torch.zeros_like(xs[0][1])
    src = [torch.zeros_like(q), torch.zeros_like(sc)]
    w13 = mr.MxWeight(*ref.random_mx((E, 2 * I, K), fmt, 7, 112, 116), gate_up=True)
    w2, wg = mr.MxWeight(*ref.random_mx((E, K, I), fmt, 8)), mr.MxWeight(*ref.random_mx((200, K), fmt, 9))
    up = mr.PreparedGateUp(q, sc, w13, st, ex, topk, block, quant=fmt)
    down = mr.PreparedDown(*up.out, w2, ids, wts, st, ex, block)
    gemm = mr.PreparedMxGemm(q, sc, wg)
    side = torch.cuda.Stream()
    main = torch.cuda.Stream()

    def step():
        now = torch.cuda.current_stream()
        q.copy_(src[0])
        sc.copy_(src[1])
        side.wait_stream(now)
        gemm(side)
        up()
        down()
        now.wait_stream(side)
        gemm.out.mul_(2.0)
        down.out.add_(1.0)

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        step()
    for x in xs:
        src[0].copy_(x[0])
        src[1].copy_(x[1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = gemm.out.clone(), down.out.clone()
        assert torch.equal(got[0], mr.mx_gemm(*x, wg) * 2.0)
        act = mr.moe_gate_up(*x, w13, st, ex, topk, block, quant=fmt)
        assert torch.equal(got[1], mr.moe_down(*act, w2, ids, wts, st, ex, block) + 1.0)


def test_beside_the_router_on_another_stream(mr):
    """Both kinds of kernel that take tensor memory at once."""
    N, K, M = 256, 2048, 512
    g = torch.Generator("cpu").manual_seed(0)
    x, w = torch.randn(M, K, generator=g).to(BF16).cuda(), (torch.randn(N, K, generator=g) * 0.02).to(BF16).cuda()
    mx, W = ref.random_mx((300, K), "mxfp4", 1), mr.MxWeight(*ref.random_mx((1000, K), "mxfp4", 2), "mxfp4")
    gemm, scratch = mr.PreparedMxGemm(*mx, W), mr.Scratch(M, N, K, 8)
    want = gemm().clone(), mr.router_gemv(x, w, scratch=scratch)
    out = torch.empty_like(want[1])
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(200):
        gemm(s[0])
        mr.router_gemv(x, w, out=out, scratch=scratch, stream=s[1])
    torch.cuda.synchronize()
    assert torch.equal(gemm.out, want[0]) and torch.equal(out, want[1])


# ------------------------------------------------------------------ refusals

def test_python_refusals(mr):
    fmt, M, E, topk, K, I, block = "mxfp8", 4, 8, 2, 256, 64, 16
    ids, wts = routed(M, E, topk, 0)
    st, ex, _ = mr.moe_sort(ids, E, block)
    q = ref.random_mx((M, K), fmt, 0)
    w13, w2 = ref.random_mx((E, 2 * I, K), fmt, 1), ref.random_mx((E, K, I), fmt, 2)
    W13, W2 = mr.MxWeight(*w13, gate_up=True), mr.MxWeight(*w2)
    Wd = mr.MxWeight(w2[0][0], w2[1][0])
    a = ref.random_mx((st.numel(), I), fmt, 3)
    bad = pytest.raises(ValueError)
    with bad:
        mr.MxWeight(*w13, format="bf16")
    with bad:
        mr.MxWeight(w13[0], w13[1][:, :, 1:])
    with bad:
        mr.MxWeight(w13[0].transpose(0, 1), w13[1].transpose(0, 1))
    with pytest.raises(mr.MoeRouteUnsupported):  # I % 32
        mr.MxWeight(*ref.random_mx((E, 2 * 40, K), fmt, 1), gate_up=True)
    with bad:
        mr.mx_gemm(*a, W13)
    with bad:
        mr.mx_gemm(q[0], q[1], Wd)  # another K
    with bad:
        mr.mx_gemm(a[0], a[1].cpu(), Wd)
    with bad:
        mr.mx_gemm(*a, Wd, out_dtype=torch.float16)
    with bad:
        mr.moe_gate_up(*q, W2, st, ex, topk, block)
    with bad:
        mr.moe_gate_up(*q, W13, st, ex, topk, block, quant="fp8")
    with bad:
        mr.moe_gate_up(*q, W13, st, ex, topk, block, sorted_rows=True)
    with bad:
        mr.moe_gate_up(*q, W13, st, ex, topk, block, sorted_rows=True, num_tokens=M)  # q has M rows
    with bad:
        mr.moe_gate_up(*q, W13, st.long(), ex, topk, block)
    with bad:
        mr.moe_down(a[0][:8], a[1][:8], W2, ids, wts, st, ex, block)
    with bad:
        mr.moe_down(*a, W2, ids, wts.double(), st, ex, block)
    with bad:
        mr.moe_down(*a, W2, ids, wts, st, ex, block, out=torch.empty(M, K, device="cuda"))
    with pytest.raises(mr.MoeRouteError) as e:  # a scratch of fewer rows
        mr.moe_down(*a, W2, ids, wts, st, ex, block, scratch=mr.ExpertScratch(1, 1, 32))
    assert e.value.status == mr.MR_ERR_SCRATCH_TOO_SMALL
    odd = torch.empty(M * K + 16, dtype=torch.uint8, device="cuda")[8:8 + M * K].view(M, K)
    with pytest.raises(mr.MoeRouteError) as e:  # misaligned codes
        mr.moe_gate_up(odd, q[1], W13, st, ex, topk, block)
    assert e.value.status == mr.MR_ERR_INVALID_ARG
