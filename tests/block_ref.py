"""The residual norm, the FP8 product with scales per 128 and the rows to the
experts and back, written out with torch (not a test module)."""

import torch

BF16 = torch.bfloat16


def rows(seed, m, k, dtype=BF16, device="cuda"):
    """Unit values with a few large columns."""
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(m, k, generator=g) * (1 + 7 * (torch.rand(k, generator=g) < 0.05))
    return x.to(dtype).to(device)


# ------------------------------------------------------------------ norm

def rstd64(sres, eps):
    return 1 / torch.sqrt(sres.double().square().sum(1) / sres.shape[1] + eps)


def normed(sres, rstd, g, norm):
    s = g.float() if norm == "rms" else 1 + g.float()
    return ((sres.float() * rstd[:, None]) * s).to(BF16)


def fp8(x):
    """(codes uint8, scales fp32 per 128) by the formula, every fp32 step rounded to nearest."""
    K = x.shape[1]
    g = torch.nn.functional.pad(x.float(), (0, -K % 128)).unflatten(1, (-1, 128))
    a = g.abs().amax(-1)
    s = a / torch.tensor(448.0, device=x.device)
    s = torch.where(s < 2.0 ** -126, torch.full_like(s, 2.0 ** -126), s)
    one = torch.ones((), device=x.device)
    v = (g * (one / s)[..., None]).flatten(1)[:, :K]
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


# ------------------------------------------------------------------ FP8 product

def e4m3(codes):
    """E4M3 values in fp64 from the format's bits."""
    b = codes.to(torch.int32)
    e, m = (b >> 3) & 15, (b & 7).double() / 8
    v = torch.ldexp(torch.where(e > 0, 1 + m, m), torch.where(e > 0, e, torch.ones_like(e)) - 7)
    v = torch.where((b & 127) == 127, torch.full_like(v, float("nan")), v)
    return torch.where(b >> 7 > 0, -v, v)


def codes(seed, r, k, device="cuda"):
    """Random codes, any but NaN."""
    c = torch.randint(0, 256, (r, k), generator=torch.Generator("cpu").manual_seed(seed), dtype=torch.uint8)
    return torch.where((c & 127) == 127, torch.zeros_like(c), c).to(device)


def scales(seed, r, k, device="cuda"):
    return (0.001 + 0.01 * torch.rand(r, k, generator=torch.Generator("cpu").manual_seed(seed))).to(device)


def product(q, xs, w, ws, dtype):
    """(out, bound) in fp64.  A block's sum: its up to 128 terms are exact and each of its additions is off by at most
    2^-23 of a partial sum (truncation); the scale's product rounds once, the scaled block and each addition of it
    once, also where shares of K are added: K / 128 + 16 additions at most; then one rounding to dtype."""
    M, K = q.shape
    R, kb = w.shape[0], xs.shape[1]
    x64, w64 = e4m3(q), e4m3(w)
    ref = torch.zeros(M, R, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(ref)
    for b in range(kb):
        s = xs[:, b, None].double() * ws[:, b].double().repeat_interleave(128)[None, :R]
        xb, wb = x64[:, 128 * b:128 * b + 128], w64[:, 128 * b:128 * b + 128]
        ref += s * (xb @ wb.T)
        mag += s.abs() * (xb.abs() @ wb.abs().T)
    tol = (128 * 2.0 ** -23 + (kb + 18) * 2.0 ** -24) * mag
    half = torch.finfo(dtype).eps / 2
    return ref, tol + half * (ref.abs() + tol) + 2.0 ** -149


# ------------------------------------------------------------------ rows

def routed(M, E, topk, seed, drop=0.0, device="cuda"):
    g = torch.Generator("cpu").manual_seed(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:topk] for _ in range(M)]).to(torch.int32)
    if drop:
        gone = torch.rand(M, topk, generator=g) < drop
        ids = torch.where(gone, torch.where(torch.rand(M, topk, generator=g) < 0.5, -1, E + 3).to(torch.int32), ids)
    w = torch.rand(M, topk, generator=g) * 2 - 0.5
    return ids.contiguous().to(device), w.to(device)


def positions(st, nt, mk):
    """Sorted position of every assignment, -1 for those that have none."""
    pos = torch.full((mk,), -1, dtype=torch.int64, device=st.device)
    p = (st[:nt] < mk).nonzero()[:, 0]
    pos[st[p].long()] = p
    return pos


def assert_within(got, ref, tol, what=""):
    err = (got.double() - ref).abs() - tol
    worst = err.max().item() if err.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} past the bound; error {(got.double() - ref).abs().max().item():.3e}"
