"""The operators around the routed experts, as cases to measure.

* norm: the residual's addition and the root-mean-square norm in front of the
  router, with the normalised rows in 8 bits: E4M3 with one fp32 scale per 128
  elements, or MXFP8.
* gemm: the product of E4M3 operands with fp32 scales, one per 128 elements of
  an activation's row and one per 128 x 128 of the weight.
* permute: rows of tokens to the sorted positions of their assignments, and
  (permute_grad) its gradient.
* combine: rows at the sorted positions back to their tokens, weighted, and
  (combine_grad) its gradients.

run() takes the plain form (elementary torch operations in fp32, one rounding
at the end) or, with own set, the calls of the framework.  exact() is the
definition in fp64.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the norm of one token's residual in front of a layer's FP8 products
        dict(name="norm_m1_fp8", op="norm", M=1, K=6144, quant="fp8"),
        # a decode batch in front of the route and of MXFP8 experts
        dict(name="norm_m48_mxfp8", op="norm", M=48, K=6144, quant="mxfp8"),
        # a prompt
        dict(name="norm_m4096_fp8", op="norm", M=4096, K=6144, quant="fp8"),
        # a dense projection of one token: the weight once
        dict(name="gemm_m1_n6144_k6144", op="gemm", M=1, N=6144, K=6144, out="bf16"),
        # the shared expert's gate/up projection of a decode batch
        dict(name="gemm_m40_n1536_k6144", op="gemm", M=40, N=1536, K=6144, out="bf16"),
        # ragged in every direction (rows, columns, a last block of 32), unrounded sums
        dict(name="gemm_m300_n2000_k2976_fp32", op="gemm", M=300, N=2000, K=2976, out="fp32"),
        # a dense projection of a prompt
        dict(name="gemm_m4096_n6144_k6144", op="gemm", M=4096, N=6144, K=6144, out="bf16"),
        # a prompt's tokens to their experts
        dict(name="permute_m4096", op="permute", M=4096, K=6144, E=128, topk=8, block=64, drop=0.0, type="bf16"),
        # the gradient of the same in a small training step, an odd batch
        dict(name="permute_grad_m1001", op="permute_grad", M=1001, K=6144, E=128, topk=8, block=64, drop=0.0,
             type="bf16"),
        # many small experts (896, top-16) of a decode batch, back to the tokens
        dict(name="combine_m16_e896", op="combine", M=16, K=3584, E=896, topk=16, block=16, drop=0.0, type="bf16"),
        # a prompt, an eighth of the assignments to experts of another process
        dict(name="combine_m4096", op="combine", M=4096, K=6144, E=128, topk=8, block=64, drop=0.125, type="bf16"),
        # the gradients of a training step
        dict(name="combine_grad_m2048", op="combine_grad", M=2048, K=6144, E=128, topk=8, block=64, drop=0.0,
             type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "permute", "permute_grad", "combine", "combine_grad"])
    M = _log(rng, 1, 4096)
    if op == "norm":
        quant = rng.choice(["fp8", "fp8", "mxfp8"])
        return dict(op=op, M=M, K=32 * _log(rng, 4, 192) if quant == "mxfp8" else 16 * _log(rng, 8, 384), quant=quant)
    if op == "gemm":
        return dict(op=op, M=M, N=_log(rng, 33, 6144), K=16 * _log(rng, 8, 384), out=rng.choice(["bf16", "fp32"]))
    K = 8 * _log(rng, 9, 768) if rng.random() < 0.7 else _log(rng, 65, 6144)
    return dict(op=op, M=min(M, 2048) if op == "combine_grad" else M, K=K,
                E=rng.choice([8, 32, 64, 100, 128] + [896] * (M <= 256)), topk=rng.randint(1, 8),
                block=16 if M <= 128 else 64, drop=rng.choice([0.0, 0.0, 0.125, 0.5]),
                type=rng.choice(["bf16", "bf16", "fp16"]))


# ------------------------------------------------------------------ inputs

def _rows(gen, m, k, dtype=torch.bfloat16):
    """Activations: unit scale, a few large channels."""
    x = torch.randn(m, k, device=DEV, generator=gen)
    x *= 1 + 7 * (torch.rand(k, device=DEV, generator=gen) < 0.01)
    return x.to(dtype)


def _groups(x, n):
    """[M, K] -> [M, ceil(K / n), n], zeros behind the row's end."""
    K = x.shape[1]
    return torch.nn.functional.pad(x, (0, -K % n)).unflatten(1, (-1, n))


def _fp8(x):
    """E4M3 codes (as values) and fp32 scales per 128 of bf16 rows."""
    g = _groups(x.float(), 128)
    s = (g.abs().amax(-1) / torch.full((), 448.0, device=DEV)).clamp(min=2.0 ** -126)
    v = g * (1.0 / s)[..., None]
    return v.clamp(-448, 448).flatten(1)[:, :x.shape[1]].to(torch.float8_e4m3fn), s


def _mxfp8(x):
    """E4M3 codes (as values) and E8M0 scales per 32 of bf16 rows: X = floor(log2(amax)) - 8."""
    g = x.float().unflatten(1, (-1, 32))
    amax = g.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    X = torch.where(amax > 0, e - 8, torch.full_like(e, -127)).clamp(-127, 127)
    v = torch.ldexp(g, -X[..., None]).flatten(1)
    return v.clamp(-448, 448).to(torch.float8_e4m3fn), (X + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _sort(ids, E, block):
    """The route's sort of ids [M, topk] (those outside [0, E) left out):
    sorted_token_ids padded with M * topk, expert_ids, num_tokens_post_padded."""
    M, k = ids.shape
    mk = M * k
    cap = (mk + min(E, mk) * (block - 1) + block - 1) // block * block
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, E)
    count = torch.bincount(flat, minlength=E + 1)[:E]
    padded = (count + block - 1) // block * block
    end = padded.cumsum(0)
    order = torch.argsort(flat, stable=True)[:int(count.sum())]
    first = torch.cumsum(count, 0) - count
    e = flat[order]
    pos = (end - padded)[e] + torch.arange(order.numel(), device=DEV) - first[e]
    st = torch.full((cap,), mk, dtype=torch.int32, device=DEV)
    st[pos] = order.int()
    b0 = torch.arange(cap // block, device=DEV) * block
    ex = torch.searchsorted(end, b0, right=True)
    ex = torch.where(b0 < end[-1], ex, -1).int()
    return st, ex, end[-1:].int()


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    c = dict(case)
    s = dict(c=c)
    M, K = c["M"], c["K"]
    if c["op"] == "norm":
        s["x"] = _rows(gen, M, K)
        s["res"] = _rows(gen, M, K) * 4
        s["g"] = (0.1 * torch.randn(K, device=DEV, generator=gen)).bfloat16()
        if own:
            import decode_expert_routing_gb300 as mr
            s["call"] = mr.PreparedAddNorm(s["x"], s["res"], s["g"], eps=EPS, norm="gemma", quant=c["quant"])
        return s
    if c["op"] == "gemm":
        N = c["N"]
        s["q"], s["xs"] = _fp8(_rows(gen, M, K))
        # any code but NaN of the exponent field 4..11, and scales that make values of about 0.01
        b = torch.randint(0, 256, (N, K), dtype=torch.uint8, device=DEV, generator=gen)
        s["w"] = ((b & 0x87) | (4 + (b >> 4 & 7) << 3)).view(torch.float8_e4m3fn)
        s["ws"] = torch.rand(-(-N // 128), -(-K // 128), device=DEV, generator=gen) * 0.003 + 0.001
        if own:
            import decode_expert_routing_gb300 as mr
            s["call"] = mr.PreparedFp8Gemm(s["q"].view(torch.uint8), s["xs"], s["w"].view(torch.uint8), s["ws"],
                                           out_dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16)
        return s
    E, k, dt = c["E"], c["topk"], TYPES[c["type"]]
    # a router's choice: some experts are asked for more often than others; experts of other processes have no id here
    logits = torch.randn(M, E, device=DEV, generator=gen) + 0.4 * torch.randn(E, device=DEV, generator=gen)
    top = torch.softmax(logits, 1).topk(k, 1)
    s["wts"] = top.values / top.values.sum(1, keepdim=True)
    gone = torch.rand(M, k, device=DEV, generator=gen) < c["drop"]
    s["ids"] = top.indices.int().masked_fill_(gone, -1)
    st, ex, nt = _sort(s["ids"], E, c["block"])
    s["sorted"], s["nt"] = st, nt
    cap = st.numel()
    # sorted positions of the assignments, -1 for those that have none
    pos = torch.full((M * k + 1,), -1, dtype=torch.int32, device=DEV)
    pos[st.long()] = torch.arange(cap, dtype=torch.int32, device=DEV)
    s["pos"] = pos[:-1].view(M, k).masked_fill(gone, -1)
    if c["op"] in ("permute", "combine_grad"):
        s["x"] = _rows(gen, M, K, dt)
    if c["op"] != "permute":
        s["y"] = _rows(gen, cap, K, dt)  # what the padding's rows hold is of no account
    if c["op"] == "combine":
        s["add"] = _rows(gen, M, K, dt)
    if own:
        import decode_expert_routing_gb300 as mr
        if c["op"] == "permute":
            # rows behind the last expert's are left as they were
            out = torch.zeros(cap, K, dtype=dt, device=DEV)
            s["call"] = mr.PreparedPermute(s["x"], s["ids"], E, st, nt, out=out)
        elif c["op"] == "permute_grad":
            s["call"] = mr.PreparedPermuteGrad(s["y"], s["pos"])
        elif c["op"] == "combine":
            s["call"] = mr.PreparedCombine(s["y"], s["pos"], s["wts"], add=s["add"])
        else:
            out = torch.zeros(cap, K, dtype=dt, device=DEV)
            s["call"] = mr.PreparedCombineGrad(s["x"], s["y"], s["pos"], s["wts"], st, nt, out=out)
    return s


# ------------------------------------------------------------------ the plain form

def _deq(q, s):
    """fp32 values of E4M3 codes [R, K] with scales [R, K / 128] (one row of scales per row of codes)."""
    return q.float() * s.repeat_interleave(128, 1)[:, :q.shape[1]]


def _norm(s):
    c = s["c"]
    sres = (s["x"].float() + s["res"].float()).bfloat16()
    f = sres.float()
    # the sum in 64 bits: what follows rounds to bf16, and one step of rstd decides on values next to a border
    rstd = (f.double().square().mean(1) + EPS).rsqrt().float()
    xn = ((f * rstd[:, None]) * (1 + s["g"].float())).bfloat16()
    q, sc = _fp8(xn) if c["quant"] == "fp8" else _mxfp8(xn)
    return dict(sres=sres, rstd=rstd, q=q, scale=sc)


def _gather(y, pos):
    """The rows of y at pos [M, k] in fp32, zeros where there is none: [M, k, K]."""
    return y[pos.clamp(min=0).long()].float().masked_fill_((pos < 0)[..., None], 0)


def run(s):
    c = s["c"]
    if own:
        r = s["call"]()
        if c["op"] == "norm":
            e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
            return dict(sres=r["sres"], rstd=r["rstd"], q=r["q"].view(e4),
                        scale=r["scale"] if c["quant"] == "fp8" else r["scale"].view(e8))
        return r
    if c["op"] == "norm":
        return _norm(s)
    if c["op"] == "gemm":
        w = _deq(s["w"], s["ws"].repeat_interleave(128, 0)[:c["N"]])
        out = _deq(s["q"], s["xs"]) @ w.T
        return out if c["out"] == "fp32" else out.bfloat16()
    dt, k = TYPES[c["type"]], c["topk"]
    if c["op"] == "permute_grad":
        return _gather(s["y"], s["pos"]).sum(1).to(dt)
    if c["op"] == "combine":
        return ((_gather(s["y"], s["pos"]) * s["wts"][..., None]).sum(1) + s["add"].float()).to(dt)
    st = s["sorted"].long()
    pad = (st >= c["M"] * k)[:, None]
    tok = (st // k).clamp(max=c["M"] - 1)
    if c["op"] == "permute":
        return s["x"][tok].masked_fill_(pad, 0), s["pos"]
    w = s["wts"].reshape(-1)[st.clamp(max=c["M"] * k - 1)]
    gy = (s["x"][tok].float() * w[:, None]).masked_fill_(pad, 0).to(dt)
    gw = (_gather(s["y"], s["pos"]) * s["x"].float()[:, None]).sum(2)
    return gy, gw


def work(c):
    M, K = c["M"], c["K"]
    if c["op"] == "norm":
        scales = M * -(-K // 128) * 4 if c["quant"] == "fp8" else M * K // 32
        return {"bytes": 7 * M * K + scales + 4 * M + 2 * K, "flops": 8 * M * K}
    if c["op"] == "gemm":
        N, kb = c["N"], -(-K // 128)
        out = (4 if c["out"] == "fp32" else 2) * M * N
        return {"bytes": (M + N) * K + 4 * kb * (M + -(-N // 128)) + out, "flops": 2 * M * N * K}
    E, mk, b = c["E"], c["M"] * c["topk"], TYPES[c["type"]].itemsize
    rows = mk * (1 - c["drop"])
    hit = E * (1 - (1 - (1 - c["drop"]) / E) ** mk)  # experts that some assignment asks for
    padded = rows + hit * (c["block"] - 1) / 2       # with the rows of their last blocks
    idx = 4 * mk
    if c["op"] == "permute":
        return {"bytes": (M + padded) * K * b + 4 * padded + 2 * idx, "flops": 0}
    if c["op"] == "permute_grad":
        return {"bytes": (M + rows) * K * b + idx, "flops": rows * K}
    if c["op"] == "combine":
        return {"bytes": (2 * M + rows) * K * b + 2 * idx, "flops": 2 * rows * K}
    return {"bytes": (M + rows + padded) * K * b + 4 * padded + 3 * idx, "flops": 3 * rows * K}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(codes):
    """E4M3 values in fp64 from the bits of the format."""
    b = codes.view(torch.uint8).int()
    e, m = b >> 3 & 15, (b & 7).double() / 8
    v = torch.ldexp(torch.where(e > 0, 1 + m, m), torch.where(e > 0, e, 1) - 7)
    return torch.where(b >> 7 > 0, -v, v)


def _scaled(codes, scale, rows):
    """codes [R, K] times scale [R / rows, K / 128]."""
    r = torch.arange(codes.shape[0], device=DEV) // rows
    b = torch.arange(codes.shape[1], device=DEV) // 128
    return _e4m3(codes) * scale.double()[r][:, b]


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        total = s["x"].double() + s["res"].double()
        f = total.bfloat16().double()  # the norm is that of the rounded sum, by definition
        rstd = 1 / torch.sqrt((f * f).sum(1) / K + EPS)
        xn = (f * rstd[:, None] * (1 + s["g"].double())).bfloat16().double()  # and is handed over in bf16
        n = 128 if case["quant"] == "fp8" else 32
        last = -(-K // n)
        big = torch.zeros(M, last, dtype=torch.float64, device=DEV)
        big.scatter_reduce_(1, (torch.arange(K, device=DEV) // n).expand(M, K), xn.abs(), "amax")
        if n == 128:
            sc = (big / 448).clamp(min=2.0 ** -126)
        else:
            sc = torch.ldexp(torch.ones_like(big), torch.where(big > 0, torch.frexp(big).exponent - 9, -127).clamp(min=-127))
        return dict(sres=total, rstd=rstd, q=xn / sc.repeat_interleave(n, 1)[:, :K], scale=sc)
    if case["op"] == "gemm":
        return _scaled(s["q"], s["xs"], 1) @ _scaled(s["w"], s["ws"], 128).T
    k = case["topk"]
    pos, ids = s["pos"].long(), s["ids"]
    if case["op"] in ("permute", "combine_grad"):
        x = s["x"].double()
        tok, slot = (ids >= 0).nonzero(as_tuple=True)
        rows = torch.zeros(s["sorted"].numel(), K, dtype=torch.float64, device=DEV)
        w = s["wts"].double()[tok, slot, None] if case["op"] == "combine_grad" else 1.0
        rows[pos[tok, slot]] = x[tok] * w
        if case["op"] == "permute":
            return rows, None
        gw = torch.zeros(M, k, dtype=torch.float64, device=DEV)
        gw[tok, slot] = (x[tok] * s["y"].double()[pos[tok, slot]]).sum(1)
        return rows, gw
    out = s["add"].double() if case["op"] == "combine" else torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for j in range(k):
        tok = (ids[:, j] >= 0).nonzero()[:, 0]
        w = s["wts"].double()[tok, j, None] if case["op"] == "combine" else 1.0
        out[tok] += s["y"].double()[pos[tok, j]] * w
    return out
