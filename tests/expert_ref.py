"""The expert products in 64 bits, from the formats' bits (not a test module)."""

import torch


def value64(codes, scale, fmt):
    """code * 2^(scale - 127) of MX rows, [..., K] float64 (no NaN codes)."""
    b = codes.to(torch.int32)
    if fmt == "mxfp4":
        b = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        sign, e, m, bias, mant = b >> 3, (b >> 1) & 3, b & 1, 1, 2
    else:
        sign, e, m, bias, mant = b >> 7, (b >> 3) & 15, b & 7, 7, 8
    frac = (e > 0).double() + m.double() / mant
    p = torch.where(e > 0, e, torch.ones_like(e)) - bias + scale.repeat_interleave(32, -1).to(torch.int32) - 127
    return torch.ldexp(torch.where(sign > 0, -frac, frac), p)


def random_mx(shape, fmt, seed, lo=120, hi=130, device="cuda"):
    """Random codes (any but NaN) and scale bytes in [lo, hi)."""
    g = torch.Generator("cpu").manual_seed(seed)
    K = shape[-1]
    if fmt == "mxfp4":
        c = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, dtype=torch.uint8)
    else:
        c = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
        c = torch.where((c & 127) == 127, torch.zeros_like(c), c)
    s = torch.randint(lo, hi, (*shape[:-1], K // 32), generator=g, dtype=torch.uint8)
    return c.to(device), s.to(device)


def sum_bound(K):
    """Error of a K-term sum of exact products over sum |term|: every one of
    the K additions is off by at most 2^-23 of a partial sum (truncation)."""
    return K * 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def product(x, w, dtype):
    """(x @ w^T, its bound) in 64 bits: the sum's error, then one rounding."""
    ref = x @ w.T
    tol = sum_bound(x.shape[-1]) * (x.abs() @ w.abs().T)
    tiny = torch.finfo(dtype).smallest_normal
    return ref, tol + half_step(dtype) * (ref.abs() + tol) + tiny * half_step(dtype) * 2


def swiglu(x, w13):
    """(act, bound) of rows x [m, K] and w13 [2I, K] before the rounding to bf16."""
    I = w13.shape[0] // 2
    h = x @ w13.T
    d = sum_bound(x.shape[-1]) * (x.abs() @ w13.abs().T)
    g, u, dg, du = h[:, :I], h[:, I:], d[:, :I], d[:, I:]
    s = torch.sigmoid(g)
    act = g * s * u
    # |silu'| <= 1.1; e^-g, the sum, the quotient and the product each round:
    # expf is good to 2 ulps, so the factors are off by 8 half steps in all
    tol = 1.1 * dg * (u.abs() + du) + (g * s).abs() * du + 8 * 2.0 ** -23 * act.abs() + 2.0 ** -120
    return act, tol


def assert_close(got, ref, tol, what=""):
    err = (got.double() - ref).abs() - tol
    worst = err.max().item()
    assert worst <= 0, f"{what}: {worst:.3e} past the bound; error {(got.double() - ref).abs().max().item():.3e}"


def used_positions(st, mk):
    """(position, assignment) of every placed assignment."""
    pos = (st < mk).nonzero()[:, 0]
    return pos, st[pos].long()


def gate_up(x, w13, st, ex, topk, block, mk, sorted_rows):
    """act [cap, I] and bound (zero rows where no assignment is placed)."""
    cap, I = st.numel(), w13.shape[1] // 2
    act = torch.zeros(cap, I, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(act)
    pos, f = used_positions(st, mk)
    e = ex[pos // block].long()
    src = pos if sorted_rows else f // topk
    for k in e.unique().tolist():
        m = e == k
        act[pos[m]], tol[pos[m]] = swiglu(x[src[m]], w13[k])
    return act, tol


def down(a, w2, st, ex, ids, wts, block, E, add=None):
    """out [M, R] and bound before the last rounding."""
    M, topk = ids.shape
    R = w2.shape[1]
    y = torch.zeros(M * topk, R, dtype=torch.float64, device=a.device)
    d = torch.zeros_like(y)
    pos, f = used_positions(st, M * topk)
    e = ex[pos // block].long()
    for k in e.unique().tolist():
        m = e == k
        rows = a[pos[m]]
        y[f[m]] = rows @ w2[k].T
        d[f[m]] = sum_bound(rows.shape[1]) * (rows.abs() @ w2[k].abs().T)
    w = (wts.double() * ((ids >= 0) & (ids < E)))[..., None]
    # a product is rounded to bf16 before it is weighted: half a step of a value within d of y
    d = d + half_step(torch.bfloat16) * (y.abs() + d)
    y, d = y.unflatten(0, (M, topk)), d.unflatten(0, (M, topk))
    out = (w * y).sum(1)
    mag = (w * y).abs().sum(1)
    if add is not None:
        out = out + add.double()
        mag = mag + add.double().abs()
    return out, (w.abs() * d).sum(1) + (topk + 1) * 2.0 ** -24 * mag
