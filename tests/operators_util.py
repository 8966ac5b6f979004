"""Plain 64-bit forms of cross attention and layer norm, and how far a kernel's results may be from them.

The bounds count roundings.  A value of type t is off by at most half a step, H[t] of itself; a sum of n
fp32 products by n 2^-24 of the sum of their magnitudes.  On the tensor cores the softmax weights and dS
are rounded to bf16 before the second product.  Every bound is an array: one for each element.
"""
from __future__ import annotations

import math

import torch

H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24


def tokens(gen, b, h, n, d, dtype, layout="bhnd", device="cuda", scale=1.0, shift=0.0):
    """A [b, h, n, d] tensor; bnhd: heads inside the token; fused: a slice of a wider projection's output."""
    shape = {"bhnd": (b, h, n, d), "bnhd": (b, n, h, d), "fused": (b, n, 3, h, d)}[layout]
    x = (torch.randn(shape, generator=gen, dtype=torch.float32) * scale + shift).to(device).to(dtype)
    if layout == "bnhd":
        return x.transpose(1, 2)
    return x[:, :, 1].transpose(1, 2) if layout == "fused" else x


def valid_keys(b, nk, kv_len, key_mask):
    ok = torch.ones(b, nk, dtype=torch.bool)
    if kv_len is not None:
        ok &= torch.arange(nk) < kv_len.cpu().clamp(0, nk)[:, None]
    if key_mask is not None:
        ok &= key_mask.cpu() != 0
    return ok


def cross_reference(q, k, v, ok, scale, dO=None):
    """The formulas in 64 bits on the CPU, with the bounds: {name: (value, bound)}."""
    t = q.dtype
    half = H[t]
    b, h, nq, d = q.shape
    hk, nk = k.shape[1], k.shape[2]
    g = h // hk
    bad = ~ok[:, None, :, None]
    q = q.cpu().double()
    k = k.cpu().double().masked_fill(bad, 0).repeat_interleave(g, 1)
    v = v.cpu().double().masked_fill(bad, 0).repeat_interleave(g, 1)
    z = (q @ k.mT) * scale
    z = z.masked_fill(~ok[:, None, None, :], -math.inf)
    lse = torch.logsumexp(z, -1)
    ref = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)[..., None]
    p = torch.exp(z - ref)
    o = p @ v
    # a logit: d products, the scale, the change of base, the difference from the maximum or the lse
    dz = (d + 4) * U * scale * (q.abs() @ k.abs().mT) + 4 * U * (z.masked_fill(z == -math.inf, 0).abs() + ref.abs())
    dz = dz.masked_fill(~ok[:, None, None, :], 0)
    dp_ = p * (dz + (p * dz).sum(-1, keepdim=True) + (nk + 16) * U)       # a weight: its logit, 2^x, the sum, the quotient
    w = half if t == torch.bfloat16 else 0.0                              # the weights as bf16 operands
    pv = p @ v.abs()
    out = {"o": (o, half * o.abs() + w * pv + (dp_ @ v.abs()) + (nk + 8) * U * pv),
           "lse": (lse, (p * dz).sum(-1) + (nk + 16) * U + 4 * U * ref[..., 0].abs())}
    if dO is None:
        return out
    go = dO.cpu().double()
    dP = go @ v.mT
    D = (go * o).sum(-1, keepdim=True)
    ds = p * (dP - D) * scale
    # D is formed from the rounded O
    eD = (go.abs() * out["o"][1]).sum(-1, keepdim=True) + (d + 2) * U * (go.abs() * o.abs()).sum(-1, keepdim=True)
    edP = (d + 2) * U * (go.abs() @ v.abs().mT)
    e_ds = scale * (dp_ * (dP - D).abs() + p * (edP + eD)) + 4 * U * ds.abs()
    e_ds2 = e_ds + w * (ds.abs() + e_ds)
    e_p = dp_ + w * (p + dp_)

    def over_group(x):
        return x.view(b, hk, g, nk, d).sum(2)

    dq = ds @ k
    dk, dv = over_group(ds.mT @ q), over_group(p.mT @ go)
    out["dq"] = (dq, half * dq.abs() + e_ds2 @ k.abs() + (nk + 8) * U * (ds.abs() @ k.abs()))
    n = nq * g + 8
    out["dk"] = (dk, half * dk.abs() + over_group(e_ds2.mT @ q.abs() + n * U * (ds.abs().mT @ q.abs())))
    out["dv"] = (dv, half * dv.abs() + over_group(e_p.mT @ go.abs() + n * U * (p.mT @ go.abs())))
    return out


def norm_reference(x, w, b, eps, dtype, param_dtype, per_batch, dy=None):
    half, phalf = H[dtype], H[param_dtype]
    x = x.cpu().double()
    c = x.shape[-1]
    shape = (x.shape[0], 1, 1, c) if per_batch else (1, 1, 1, c)
    w = (torch.ones(shape) if w is None else w.cpu().reshape(shape)).double()
    b = (torch.zeros(shape) if b is None else b.cpu().reshape(shape)).double()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    xhat = xc * rstd
    y = xhat * w + b
    # the mean of c values, the deviation from it (its error enters the variance in second order
    # and through the deviations' own roundings)
    e_mean = (c + 2) * U * x.abs().mean(-1, keepdim=True)
    e_xc = e_mean + U * xc.abs()
    e_rel = (c + 8) * U + (2 * xc.abs() * e_xc + e_xc * e_xc).mean(-1, keepdim=True) * rstd * rstd
    e_xhat = rstd * e_xc + xhat.abs() * (e_rel + 2 * U)
    out = {"y": (y, half * y.abs() + (1 + half) * (e_xhat * w.abs() + 2 * U * (xhat * w).abs() + U * y.abs()))}
    if dy is None:
        return out
    dy = dy.cpu().double()
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xhat).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xhat * c2)
    e_c1 = (c + 2) * U * g.abs().mean(-1, keepdim=True)
    e_c2 = (c + 4) * U * (g * xhat).abs().mean(-1, keepdim=True) + (g.abs() * e_xhat).mean(-1, keepdim=True)
    e_dx = rstd * (4 * U * (g.abs() + c1.abs() + (xhat * c2).abs()) + e_c1 + xhat.abs() * e_c2 + e_xhat * c2.abs()) \
        + (e_rel + 4 * U) * dx.abs()
    out["dx"] = (dx, half * dx.abs() + (1 + half) * e_dx)
    dims = (1, 2) if per_batch else (0, 1, 2)
    rows = x[..., 0].numel()
    dw, db = (dy * xhat).sum(dims), dy.sum(dims)
    e_dw = (dy.abs() * e_xhat).sum(dims) + (rows + 4) * U * (dy * xhat).abs().sum(dims)
    out["dweight"] = (dw, phalf * dw.abs() + (1 + phalf) * e_dw)
    out["dbias"] = (db, phalf * db.abs() + (1 + phalf) * (rows + 4) * U * dy.abs().sum(dims))
    return out


def check(name, got, want, bound):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin], want[~fin]), f"{name}: infinities differ"
    off = (got - want).abs()[fin]
    allowed = bound[fin] + 1e-30
    assert torch.isfinite(off).all(), f"{name}: not finite where the formula is"
    if off.numel():
        i = int((off / allowed).argmax())
        assert bool((off <= allowed).all()), \
            f"{name}: off by {off[i]:.3g} at {want[fin][i]:.6g}, allowed {allowed[i]:.3g}; " \
            f"{int((off > allowed).sum())} of {off.numel()} outside"
