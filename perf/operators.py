"""The expert products that follow the route, as cases to measure.

Three operators and one run of two of them:

* mx_gemm: the product of a microscaled activation and a microscaled weight
  (MXFP8: E4M3 codes, MXFP4: E2M1 codes, one E8M0 scale per 32 elements of k).
* moe_gate_up: the experts' gate/up products over the sorted assignments, with
  SwiGLU; rows at the sorted positions, bf16.
* moe_down: the experts' down products and the combination over a token's
  top-k experts, bf16.
* experts: moe_gate_up with its output quantised to the same MX format, then
  moe_down (the two calls of one MoE layer).

run() takes the plain form (elementary torch operations in fp32, one rounding
at the end; the sort's padded blocks as one batch of small products) or, with
own set, the calls of the framework.  exact() is the definition in fp64.
"""

import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one token of a decode step: 8 experts' weights once, latency of a short launch
        dict(name="gate_up_m1_fp8", op="gate_up", fmt="mxfp8", M=1, E=128, topk=8, K=6144, I=768, block=16,
             sorted_rows=False),
        # a decode batch on 4-bit weights
        dict(name="gate_up_m16_fp4", op="gate_up", fmt="mxfp4", M=16, E=128, topk=8, K=6144, I=768, block=16,
             sorted_rows=False),
        # many small experts (896, top-16), an odd batch
        dict(name="gate_up_m37_e896_fp8", op="gate_up", fmt="mxfp8", M=37, E=896, topk=16, K=3584, I=256, block=16,
             sorted_rows=False),
        # prefill: 32768 assignments, the quantised rows in sorted order
        dict(name="gate_up_m4096_fp8", op="gate_up", fmt="mxfp8", M=4096, E=128, topk=8, K=6144, I=768, block=64,
             sorted_rows=True),
        # the second half of the same decode steps and of the prefill
        dict(name="down_m1_fp8", op="down", fmt="mxfp8", M=1, E=128, topk=8, K=6144, I=768, block=16),
        dict(name="down_m64_fp4", op="down", fmt="mxfp4", M=64, E=128, topk=8, K=6144, I=768, block=16),
        dict(name="down_m4096_fp8", op="down", fmt="mxfp8", M=4096, E=128, topk=8, K=6144, I=768, block=64),
        # both halves: a decode batch, and a ragged prompt on 4-bit weights
        dict(name="experts_m8_fp8", op="experts", fmt="mxfp8", M=8, E=128, topk=8, K=6144, I=768, block=16),
        dict(name="experts_m1001_fp4", op="experts", fmt="mxfp4", M=1001, E=128, topk=8, K=6144, I=768, block=64),
        # the shared expert's down projection for one token
        dict(name="gemm_m1_n6144_k768_fp8", op="gemm", fmt="mxfp8", M=1, N=6144, K=768),
        # a dense projection of a decode batch, and of a prompt
        dict(name="gemm_m33_n6144_k6144_fp8", op="gemm", fmt="mxfp8", M=33, N=6144, K=6144),
        dict(name="gemm_m4096_n6144_k6144_fp4", op="gemm", fmt="mxfp4", M=4096, N=6144, K=6144),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fmt = rng.choice(["mxfp8", "mxfp4"])
    op = rng.choice(["gate_up", "down", "experts", "gemm"])
    M = _log(rng, 1, 4096)
    if op == "gemm":
        return dict(op=op, fmt=fmt, M=M, N=_log(rng, 33, 6144), K=32 * _log(rng, 4, 192))
    case = dict(op=op, fmt=fmt, M=M, E=rng.choice([8, 32, 64, 100, 128]), topk=rng.randint(1, 8),
                K=32 * _log(rng, 8, 192), I=32 * _log(rng, 2, 16 if op == "experts" else 24),
                block=16 if M <= 128 else 64)
    if op == "gate_up":
        case["sorted_rows"] = rng.random() < 0.5
    return case


# ------------------------------------------------------------------ inputs

def _elems(codes, fmt, dtype):
    """The values of MX codes, without their scales: [..., K]."""
    if fmt == "mxfp8":
        return codes.view(torch.float8_e4m3fn).to(dtype)
    mag = torch.tensor(E2M1, dtype=dtype, device=codes.device)
    one = torch.cat([mag, -mag])
    pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # byte -> (low nibble, high nibble)
    return pair[codes.int()].flatten(-2)


def _dequant(codes, scale, fmt, dtype=torch.float32):
    v = _elems(codes, fmt, dtype)
    s = torch.exp2(scale.to(dtype) - 127)
    return v.unflatten(-1, (-1, 32)).mul_(s[..., None]).flatten(-2)


def _quant(x, fmt):
    """MX codes and scales of bf16 rows, per the OCP formats: X = floor(log2(amax)) - emax."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1
    X = torch.where(amax > 0, e - (8 if fmt == "mxfp8" else 2), torch.full_like(e, -127)).clamp(-127, 127)
    v = torch.ldexp(b, -X[..., None]).flatten(-2)
    scale = (X + 127).to(torch.uint8)
    if fmt == "mxfp8":
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    a = v.abs().clamp(max=6)
    step = torch.where(a >= 4, 2.0, torch.where(a >= 2, 1.0, 0.5))
    a = torch.round(a / step) * step  # ties to even
    idx = torch.bucketize(a, torch.tensor(E2M1, device=x.device)).to(torch.uint8)
    idx = idx | (torch.signbit(v).to(torch.uint8) << 3)
    return idx[..., 0::2] | (idx[..., 1::2] << 4), scale


def _weight(gen, shape, fmt):
    """Random codes [..., K] and scales: values of about 0.01, as trained weights have."""
    K = shape[-1]
    if fmt == "mxfp8":
        # any code but NaN: the exponent field 4..11
        b = torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)
        codes = (b & 0x87) | (4 + (b >> 4 & 7) << 3)
    else:
        codes = torch.randint(0, 256, (*shape[:-1], K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    lo = 115 if fmt == "mxfp8" else 117
    scale = torch.randint(lo, lo + 5, (*shape[:-1], K // 32), dtype=torch.uint8, device=DEV, generator=gen)
    return codes, scale


def _sort(ids, E, block):
    """The route's sort: (sorted_token_ids, expert_ids), padded with M * topk and -1."""
    M, k = ids.shape
    mk = M * k
    cap = (mk + min(E, mk) * (block - 1) + block - 1) // block * block
    flat = ids.reshape(-1).long()
    count = torch.bincount(flat, minlength=E)
    padded = (count + block - 1) // block * block
    end = padded.cumsum(0)
    order = torch.argsort(flat, stable=True)
    first = torch.cumsum(count, 0) - count
    e = flat[order]
    pos = (end - padded)[e] + torch.arange(mk, device=DEV) - first[e]
    st = torch.full((cap,), mk, dtype=torch.int32, device=DEV)
    st[pos] = order.int()
    b0 = torch.arange(cap // block, device=DEV) * block
    ex = torch.searchsorted(end, b0, right=True)
    ex = torch.where(b0 < end[-1], ex, -1).int()
    return st, ex


def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    c = dict(case)
    s = dict(c=c)
    M, K, fmt = c["M"], c["K"], c["fmt"]

    def rows(m, k):
        # activations after a norm: unit scale, a few large channels
        x = torch.randn(m, k, device=DEV, generator=gen)
        x *= 1 + 7 * (torch.rand(k, device=DEV, generator=gen) < 0.01)
        return x.bfloat16()

    if c["op"] == "gemm":
        s["x"] = _quant(rows(M, K), fmt)
        s["w"] = _weight(gen, (c["N"], K), fmt)
        if own:
            import decode_expert_routing_gb300 as mr
            s["call"] = mr.PreparedMxGemm(*s["x"], mr.MxWeight(*s["w"], fmt))
        return s
    E, k, I, block = c["E"], c["topk"], c["I"], c["block"]
    # a router's choice: some experts are asked for more often than others
    logits = torch.randn(M, E, device=DEV, generator=gen) + 0.4 * torch.randn(E, device=DEV, generator=gen)
    top = torch.softmax(logits, 1).topk(k, 1)
    s["ids"] = top.indices.int()
    s["wts"] = top.values / top.values.sum(1, keepdim=True)
    st, ex = s["sort"] = _sort(s["ids"], E, block)
    cap = st.numel()
    if c["op"] != "down":
        q, sc = _quant(rows(M, K), fmt)
        if c.get("sorted_rows"):
            tok = (st // k).clamp(max=M - 1).long()
            pad = (st == M * k)[:, None]
            q, sc = q[tok].masked_fill_(pad, 0), sc[tok].masked_fill_(pad, 0)
        s["x"] = q, sc
        s["w13"] = _weight(gen, (E, 2 * I, K), fmt)
    else:
        a = rows(cap, I).masked_fill_((st == M * k)[:, None], 0)
        s["act"] = _quant(a, fmt)
    if c["op"] != "gate_up":
        s["w2"] = _weight(gen, (E, K, I), fmt)
    if own:
        import decode_expert_routing_gb300 as mr
        if c["op"] != "down":
            quant = fmt if c["op"] == "experts" else None
            out = None if quant else torch.zeros(cap, I, dtype=torch.bfloat16, device=DEV)
            s["up"] = mr.PreparedGateUp(*s["x"], mr.MxWeight(*s["w13"], fmt, gate_up=True), st, ex, k, block,
                                        num_tokens=M, sorted_rows=bool(c.get("sorted_rows")), quant=quant, out=out)
            if quant:
                s["act"] = s["up"].out
        if c["op"] != "gate_up":
            s["down"] = mr.PreparedDown(*s["act"], mr.MxWeight(*s["w2"], fmt), s["ids"], s["wts"], st, ex, block)
    return s


# ------------------------------------------------------------------ the plain form

def _blocks(rows, w, ex, block, fmt):
    """rows [cap, K] fp32 times each block's expert's weight: [cap, R] fp32 (blocks without an expert: of expert 0)."""
    codes, scale = w
    e = ex.clamp(min=0).long()
    wf = _dequant(codes[e], scale[e], fmt)
    return torch.bmm(rows.unflatten(0, (-1, block)), wf.transpose(1, 2)).flatten(0, 1)


def _gate_up(s):
    c = s["c"]
    st, ex = s["sort"]
    M, k, I = c["M"], c["topk"], c["I"]
    x = _dequant(*s["x"], c["fmt"])
    if not c.get("sorted_rows"):
        x = x[(st // k).clamp(max=M - 1).long()]
    h = _blocks(x, s["w13"], ex, c["block"], c["fmt"])
    g, u = h[:, :I], h[:, I:]
    act = g / (1 + torch.exp(-g)) * u
    return act.masked_fill_((st == M * k)[:, None], 0).bfloat16()


def _down(s, act):
    c = s["c"]
    st, ex = s["sort"]
    M, k, K = c["M"], c["topk"], c["K"]
    y = _blocks(_dequant(*act, c["fmt"]), s["w2"], ex, c["block"], c["fmt"])
    f = torch.zeros(M * k + 1, K, device=DEV)
    f[st.long()] = y  # the padding positions share the last row
    return (f[:-1].unflatten(0, (M, k)) * s["wts"][..., None]).sum(1).bfloat16()


def run(s):
    if own:
        if "call" in s:
            return s["call"]()
        if "up" in s:
            act = s["up"]()
        return s["down"]() if "down" in s else act
    c = s["c"]
    if c["op"] == "gemm":
        return (_dequant(*s["x"], c["fmt"]) @ _dequant(*s["w"], c["fmt"]).T).bfloat16()
    if c["op"] == "gate_up":
        return _gate_up(s)
    if c["op"] == "down":
        return _down(s, s["act"])
    return _down(s, _quant(_gate_up(s), c["fmt"]))


def work(c):
    per = 33 / 32 if c["fmt"] == "mxfp8" else 17 / 32  # bytes of one element with its share of the scale
    M, K = c["M"], c["K"]
    if c["op"] == "gemm":
        N = c["N"]
        return {"bytes": (M + N) * K * per + 2 * M * N, "flops": 2 * M * N * K}
    E, k, I = c["E"], c["topk"], c["I"]
    mk = M * k
    hit = E * (1 - (1 - k / E) ** M)  # experts that some token asks for
    up = hit * 2 * I * K * per + (mk if c.get("sorted_rows") else M) * K * per + 4 * mk
    down = hit * K * I * per + 12 * mk + 2 * M * K
    act8, act16 = mk * I * per, mk * I * 2
    if c["op"] == "gate_up":
        return {"bytes": up + act16, "flops": 4 * mk * I * K}
    if c["op"] == "down":
        return {"bytes": down + act8, "flops": 2 * mk * I * K}
    return {"bytes": up + down + 2 * act8, "flops": 6 * mk * I * K}


# ------------------------------------------------------------------ the definition in 64 bits

def _value64(codes, scale, fmt):
    """code * 2^(scale - 127) in fp64 from the bits of the formats."""
    b = codes.to(torch.int32)
    if fmt == "mxfp4":
        b = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        sign, e, m, bias, mant = b >> 3, b >> 1 & 3, b & 1, 1, 2
    else:
        sign, e, m, bias, mant = b >> 7, b >> 3 & 15, b & 7, 7, 8
    frac = torch.where(e > 0, 1.0, 0.0).double() + m.double() / mant
    p = torch.where(e > 0, e, torch.ones_like(e)) - bias + scale.repeat_interleave(32, -1).int() - 127
    return torch.ldexp(torch.where(sign > 0, -frac, frac), p)


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    c, fmt = s["c"], case["fmt"]
    if c["op"] == "gemm":
        return _value64(*s["x"], fmt) @ _value64(*s["w"], fmt).T
    E, k, I, M, K = c["E"], c["topk"], c["I"], c["M"], c["K"]
    ids = s["ids"].long()
    place = torch.empty(M * k, dtype=torch.long, device=DEV)  # sorted position of assignment f
    st = s["sort"][0].long()
    real = (st < M * k).nonzero()[:, 0]
    place[st[real]] = real
    out = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    acts = torch.zeros(st.numel(), I, dtype=torch.float64, device=DEV)
    for e in range(E):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if tok.numel() == 0:
            continue
        pos = place[tok * k + slot]
        if c["op"] != "down":
            src = pos if c.get("sorted_rows") else tok
            x = _value64(s["x"][0][src], s["x"][1][src], fmt)
            h = x @ _value64(s["w13"][0][e], s["w13"][1][e], fmt).T
            g, u = h[:, :I], h[:, I:]
            acts[pos] = act = g * torch.sigmoid(g) * u
        if c["op"] == "gate_up":
            continue
        if c["op"] == "experts":  # the hand-over is in bf16 and the MX format by definition
            a = _value64(*_quant(act.bfloat16(), fmt), fmt)
        else:
            a = _value64(s["act"][0][pos], s["act"][1][pos], fmt)
        y = a @ _value64(s["w2"][0][e], s["w2"][1][e], fmt).T
        out.index_add_(0, tok, y * s["wts"][tok, slot].double()[:, None])
    return acts if c["op"] == "gate_up" else out
