"""Stream order of the expert products' calls and of the memory they make."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests import expert_ref as ref  # noqa: E402
from tests.test_gpu_experts import mr, quant, routed  # noqa: E402, F401

BF16 = torch.bfloat16


def _rows(seed, m, k):
    return torch.randn(m, k, generator=torch.Generator("cpu").manual_seed(seed)).to(BF16).cuda()


def _with_flags(mr, flags, run, times):
    mr.set_launch_flags(flags)
    try:
        out = [run() for _ in range(times)]
        torch.cuda.synchronize()
        return out
    finally:
        mr.set_launch_flags(0)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_scales_are_laid_out_in_stream_order(mr, fmt):
    """Under MR_LAUNCH_PDL: a weight quantised just before its scales are laid
    out, products just before and after they are laid out again, and a product
    of the call before the layout."""
    M, R, K = 300, 4096, 2048
    w, w2 = _rows(1, R, K), _rows(2, R, K) * 8
    x = quant(mr, _rows(3, M, K), fmt)
    E, topk, I, block = 4, 2, 512, 64
    ids, wts = routed(M, E, topk, 1)
    st, ex, _ = mr.moe_sort(ids, E, block)
    w13 = mr.MxWeight(*ref.random_mx((E, 2 * I, K), fmt, 6, 112, 116), fmt, gate_up=True)
    down = mr.MxWeight(*ref.random_mx((E, K, I), fmt, 7, 112, 116), fmt)
    torch.cuda.synchronize()

    def run():
        codes, scale = quant(mr, w, fmt)
        W = mr.MxWeight(codes, scale, fmt)  # (scale is being written by the kernel before)
        first = mr.mx_gemm(*x, W)
        W.scale = quant(mr, w2, fmt)[1]
        again = mr.mx_gemm(*x, W)
        W.refresh()  # (the product before still reads the scales as they were)
        last = mr.mx_gemm(*x, W)
        act = mr.moe_gate_up(*x, w13, st, ex, topk, block, quant=fmt)
        W.refresh()
        out = mr.moe_down(*act, down, ids, wts, st, ex, block)
        return first, again, last, out

    want = _with_flags(mr, 0, run, 1)[0]
    assert torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2])
    for got in _with_flags(mr, mr.LAUNCH_PDL, run, 20):
        for g, o in zip(got, want):
            assert torch.equal(g, o)


# ------------------------------------------------------------------ memory that the calls make themselves

SLEEP = 20_000_000  # cycles of a queued wait: some 10 ms


class Pending:
    """A block of the current stream given back while work on it is still queued there: it is written late, and read
    into keep after that."""

    def __init__(self, nbytes):
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.keep = torch.zeros_like(block)
        self.ptr = block.data_ptr()
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        block.fill_(171)
        torch.cuda._sleep(SLEEP)
        self.keep.copy_(block)

    def check(self):
        torch.cuda.synchronize()
        assert (self.keep == 171).all(), "queued work on the block given back was overwritten"


def experts(mr, M, E, topk, K, I, block, seed=1):
    ids, wts = routed(M, E, topk, seed)
    st, ex, _ = mr.moe_sort(ids, E, block)
    x = ref.random_mx((M, K), "mxfp8", seed)
    w13 = mr.MxWeight(*ref.random_mx((E, 2 * I, K), "mxfp8", seed + 1, 112, 116), gate_up=True)
    a = ref.random_mx((st.numel(), I), "mxfp8", seed + 2)
    w2 = mr.MxWeight(*ref.random_mx((E, K, I), "mxfp8", seed + 3))
    return dict(ids=ids, wts=wts, st=st, ex=ex, x=x, w13=w13, a=a, w2=w2, topk=topk, block=block)


def up(mr, s, **kw):
    return mr.moe_gate_up(*s["x"], s["w13"], s["st"], s["ex"], s["topk"], s["block"], **kw)


def down(mr, s, **kw):
    return mr.moe_down(*s["a"], s["w2"], s["ids"], s["wts"], s["st"], s["ex"], s["block"], **kw)


@pytest.mark.parametrize("raw", [False, True])
def test_calls_on_another_stream_take_that_streams_memory(mr, raw):
    """No synchronisation before the calls: the current stream's work on memory that it has given back is queued."""
    M, topk, K, I = 64, 4, 1024, 256
    s = experts(mr, M, 8, topk, K, I, 16)
    gw = mr.MxWeight(*ref.random_mx((K, K), "mxfp8", 9))
    codes, scale = ref.random_mx((4096, 4096), "mxfp8", 8)
    want = down(mr, s), up(mr, s), up(mr, s, quant="mxfp8"), mr.mx_gemm(*s["x"], gw), mr.MxWeight(codes, scale).packed
    rows = s["st"] < M * topk
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    cap = s["st"].numel()
    calls = [(lambda: down(mr, s, stream=stream), mr.ExpertScratch(M, topk, K).nbytes),
             (lambda: up(mr, s, stream=stream), cap * I * 2), (lambda: up(mr, s, quant="mxfp8", stream=stream), cap * I),
             (lambda: mr.mx_gemm(*s["x"], gw, stream=stream), M * K * 2),
             (lambda: mr.MxWeight(codes, scale, stream=stream).packed, want[4].numel())]
    torch.cuda.synchronize()
    for (call, nbytes), w in zip(calls, want):
        p = Pending(nbytes)
        got = call()
        assert all(t.data_ptr() != p.ptr for t in (got if isinstance(got, tuple) else (got,)))
        side.synchronize()
        got = tuple(t.clone() for t in got) if isinstance(got, tuple) else got.clone()
        p.check()
        if isinstance(w, tuple):
            assert all(torch.equal(g[rows], o[rows]) for g, o in zip(got, w))
        elif w.shape[0] == cap:
            assert torch.equal(got[rows], w[rows])
        else:
            assert torch.equal(got, w)


def test_the_scratch_is_the_calls_own_streams(mr, monkeypatch):
    s = experts(mr, 64, 8, 4, 1024, 256, 16)
    made = []

    class Log(mr.ExpertScratch):
        def __init__(self, *a, **kw):
            super().__init__(*a, **kw)
            made.append((self.tensor.data_ptr(), torch.cuda.current_stream().cuda_stream))

    monkeypatch.setattr(mr, "ExpertScratch", Log)
    side = torch.cuda.Stream()
    down(mr, s)
    down(mr, s, stream=side)
    down(mr, s, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert [m[1] for m in made] == [torch.cuda.current_stream().cuda_stream, side.cuda_stream, side.cuda_stream]
    assert made[0][0] != made[1][0]
    assert torch.equal(down(mr, s, stream=0), down(mr, s))  # (the default stream's handle)


def test_prepared_calls_on_another_stream(mr):
    """Their buffers come from the stream of their making: the first call on another one comes after what is queued
    there, and the memory is not handed on before that stream is done."""
    M, topk, K = 64, 4, 1024
    s = experts(mr, M, 8, topk, K, 256, 16)
    want = down(mr, s)
    out = torch.zeros_like(want)
    n = mr.ExpertScratch(M, topk, K).nbytes
    side = torch.cuda.Stream()
    for made_out in (True, False):
        torch.cuda.synchronize()
        p = Pending(n)
        call = mr.PreparedDown(*s["a"], s["w2"], s["ids"], s["wts"], s["st"], s["ex"], s["block"],
                               out=None if made_out else out)
        got = call(side)
        got = got if made_out else out
        side.synchronize()
        p.check()
        assert torch.equal(got, want)
        # dropped while its call waits on the side stream
        out.zero_()
        call = mr.PreparedDown(*s["a"], s["w2"], s["ids"], s["wts"], s["st"], s["ex"], s["block"], out=out)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        call(side)
        del call
        other = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all((o == 255).all() for o in other), "the call's scratch was handed on before it ran"


def test_a_weight_dropped_while_its_product_waits(mr):
    codes, scale = ref.random_mx((2048, 1024), "mxfp8", 1)
    x = ref.random_mx((32, 1024), "mxfp8", 2)
    want = mr.mx_gemm(*x, mr.MxWeight(codes, scale))
    side = torch.cuda.Stream()
    for prepared in (False, True):
        out = torch.zeros_like(want)
        W = mr.MxWeight(codes, scale)
        n = W.packed.numel()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(SLEEP)
        if prepared:
            mr.PreparedMxGemm(*x, W, out=out)(side)
        else:
            mr.mx_gemm(*x, W, out=out, stream=side)
        del W
        other = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all((o == 255).all() for o in other)


def test_a_result_dropped_while_the_current_stream_reads_it(mr):
    W = mr.MxWeight(*ref.random_mx((2048, 1024), "mxfp8", 1))
    x, y = ref.random_mx((512, 1024), "mxfp8", 2), ref.random_mx((512, 1024), "mxfp8", 3)
    want = mr.mx_gemm(*x, W)
    keep = torch.zeros_like(want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mr.mx_gemm(*x, W, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    keep.copy_(got)
    del got
    others = [mr.mx_gemm(*y, W, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(keep, want)
    assert all(torch.equal(o, mr.mx_gemm(*y, W)) for o in others)


def test_made_and_called_inside_a_capture(mr):
    """Prepared calls made while a graph is captured, and called on a stream that joined it earlier."""
    s = experts(mr, 24, 8, 4, 1024, 256, 16)
    want = down(mr, s), up(mr, s, quant="mxfp8")
    rows = s["st"] < 24 * 4
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        side.wait_stream(main)
        tmp = torch.full((4 << 20,), 3, dtype=torch.uint8, device="cuda")
        sums = tmp.long().sum()
        del tmp
        a = mr.PreparedDown(*s["a"], s["w2"], s["ids"], s["wts"], s["st"], s["ex"], s["block"])
        b = mr.PreparedGateUp(*s["x"], s["w13"], s["st"], s["ex"], s["topk"], s["block"], quant="mxfp8")
        b(side)
        a(side)
        c = down(mr, s, stream=side)
        main.wait_stream(side)
    # the same objects in another capture, on a third stream, and outside
    third = torch.cuda.Stream()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2, stream=main):
        third.wait_stream(main)
        a(third)
        b(third)
        main.wait_stream(third)
    for graph in (g, g2, g):
        a.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(c, want[0]) and int(sums) == 3 * (4 << 20)
        assert all(torch.equal(o[rows], w[rows]) for o, w in zip(b.out, want[1]))
    a.out.zero_()
    a()
    assert torch.equal(a.out, want[0])


def test_streams_of_other_kinds(mr):
    """Raw handles and the default stream's for laying out scales; a CPU operand is refused whatever the stream."""
    codes, scale = ref.random_mx((256, 512), "mxfp8", 1)
    x = ref.random_mx((8, 512), "mxfp8", 2)
    side = torch.cuda.Stream()
    W = mr.MxWeight(codes, scale)
    want = mr.mx_gemm(*x, W)
    torch.cuda.synchronize()
    for stream in (0, side, side.cuda_stream):
        V = mr.MxWeight(codes, scale, stream=stream)
        V.refresh(stream)
        got = mr.mx_gemm(*x, V, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(V.packed, W.packed) and torch.equal(got, want)
    with pytest.raises(ValueError):
        mr.mx_gemm(x[0].cpu(), x[1], W, stream=side)
