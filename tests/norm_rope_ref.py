"""Norm, rotation and their gradients in 64 bits (plain torch on the CPU),
and the error that fp32 arithmetic and one bf16 rounding may add.

Bounds.  The kernels read bf16 (exact), compute in fp32 and round once.  With
u = 2^-24 (half a step of fp32) every intermediate is a short chain of
roundings: at most 7 + 4 additions and 3 operations around the reciprocal
root for rstd, and fewer than 12 products and sums for a value, so a value is
off by at most 32 u times the sum of the magnitudes of its terms, before the
final rounding of half a bf16 step (2^-8 of the rounded value).  The gradient
adds a second row sum and a product with it: 64 u.  A weight gradient is a sum
over rows: its longest chain is (rows per thread) + 40 additions, on top of
each term's 32 u.
"""
import torch

U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
EPS = 1e-6


def table(rows, rope_dim, base=10000.0):
    inv = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv
    return torch.stack((ang.cos(), ang.sin()), -1).float()


def pairs(d, rope_dim, interleaved):
    """Index of every value's pair partner, and the sign of the sine for it."""
    partner, sign = torch.arange(d), torch.zeros(d, dtype=torch.float64)
    for i in range(rope_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rope_dim // 2)
        partner[a], partner[b], sign[a], sign[b] = b, a, -1.0, 1.0
    return partner, sign


def spread(tab, d, interleaved):
    """(cos, sin) [..., d] of every value of a row, from table rows [..., rope/2, 2]."""
    half = tab.shape[-2]
    tab = tab.double()
    cos = torch.ones(tab.shape[:-2] + (d,), dtype=torch.float64)
    sin = torch.zeros_like(cos)
    for i in range(half):
        for e in ((2 * i, 2 * i + 1) if interleaved else (i, i + half)):
            cos[..., e], sin[..., e] = tab[..., i, 0], tab[..., i, 1]
    return cos, sin


def forward(x, w, eps, tab, interleaved):
    """(y, bound) for x [..., H, d]; tab [..., rope/2, 2] or None; w [d] or None."""
    x = x.double()
    d = x.shape[-1]
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    terms = x.abs()
    if tab is not None:
        partner, sign = pairs(d, 2 * tab.shape[-2], interleaved)
        cos, sin = (t[..., None, :] for t in spread(tab, d, interleaved))
        terms = (x * cos).abs() + (x[..., partner] * sin).abs()
        x = x * cos + sign * x[..., partner] * sin
    err = 32 * U * terms
    return x, err + HALF_BF16 * (x.abs() + err)


def backward(dy, x, w, eps, tab, interleaved):
    """(dx, bound, dw, its terms' magnitudes summed) for dy, x [..., H, d]."""
    g = dy.double()
    d = g.shape[-1]
    mag = g.abs()
    if tab is not None:
        partner, sign = pairs(d, 2 * tab.shape[-2], interleaved)
        cos, sin = (t[..., None, :] for t in spread(tab, d, interleaved))
        mag = (g * cos).abs() + (g[..., partner] * sin).abs()
        g = g * cos - sign * g[..., partner] * sin
    if w is None:
        err = 32 * U * mag
        return g, err + HALF_BF16 * (g.abs() + err), None, None
    x, w = x.double(), w.double()
    rstd = 1 / ((x * x).mean(-1, keepdim=True) + eps).sqrt()
    xh = x * rstd
    dw = (g * xh).flatten(0, -2).sum(0)
    dw_mag = (mag * xh.abs()).flatten(0, -2).sum(0)
    dx = rstd * (g * w - xh * (g * w * xh).mean(-1, keepdim=True))
    terms = rstd * (mag * w.abs() + xh.abs() * (mag * w.abs() * xh.abs()).mean(-1, keepdim=True))
    err = 64 * U * terms
    return dx, err + HALF_BF16 * (dx.abs() + err), dw, dw_mag


def check(got, want, bound):
    got = got.detach().cpu().double()
    assert got.shape == want.shape
    assert torch.isfinite(got).all()
    worst = ((got - want).abs() - bound).max().item()
    assert worst <= 0, f"beyond the bound by {worst}"
