"""Attention over a paged cache behind a shared prefix in 64 bits (plain torch
on the CPU), and the error that the kernels' roundings may add.

Bounds, with u = 2^-24 (half a step of fp32) and h = 2^-8 (half a step of
bf16).  A score is a sum of d exact products, accumulated in fp32 with steps
that may truncate (2u each): off by at most 2 d u times the magnitudes of its
terms.  Scaling it and subtracting the maximum round twice at its magnitude,
exp2 adds less than 4 u, the merges of partial results (at most 16 of them,
each a weight, a product and a sum) less than 16 * 8 u.  So every weight is
off by a relative D = 2 d u X + 4 u X + 160 u, X being the row's largest sum
of |q k| * scale, in the weight as in the sum that divides it: 2 D for O, D
for the log-sum-exp.  Rounding the weights to bf16 adds h (the sum that
divides takes the rounded ones, so that O moves by at most
sum w |v - O| * h / (1 - h)).  Sums over n keys in fp32 add 2 n u of their
terms' magnitudes, and O is rounded once more on the way out.
"""
import math

import torch

U = 2.0 ** -24
H = 2.0 ** -8


def make(new, lens, P, Hq, Hkv, d, page, seed, pad=0, lead=0, fill=float("nan"), spare=3):
    """Inputs on the CPU.  Rows of the pages that hold no key are `fill`; table
    entries that name no page are -7."""
    gen = torch.Generator().manual_seed(seed)
    S, T = len(new), lead + sum(new) + pad
    need = [-(-n // page) for n in lens]
    shared = -(-P // page)
    pages = sum(need) + shared + spare
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((S, max(1, max(need)) + 2), -7, dtype=torch.int32)
    k = torch.full((pages, Hkv, page, d), fill, dtype=torch.bfloat16)
    v = k.clone()

    def put(ids, count):
        for i, p in enumerate(ids):
            n = min(page, count - i * page)
            k[p, :, :n] = torch.randn(Hkv, n, d, generator=gen).bfloat16()
            v[p, :, :n] = torch.randn(Hkv, n, d, generator=gen).bfloat16()

    put(order[:shared].tolist(), P)
    at = shared
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        put(order[at:at + n].tolist(), lens[s])
        at += n
    start = torch.tensor([lead + sum(new[:i]) for i in range(S + 1)], dtype=torch.int32)
    return dict(q=torch.randn(T, Hq, d, generator=gen).bfloat16(), k=k, v=v, table=table,
                start=start, len=torch.tensor(lens, dtype=torch.int32),
                prefix=order[:shared].clone(), P=P, new=new, lens=lens, page=page,
                heads=(Hq, Hkv, d), scale=d ** -0.5)


def _keys(pages, ids, count):
    return pages[ids.long()].double().transpose(0, 1).flatten(1, 2)[:, :count]


def exact(c):
    """(O, its bound, LSE, its bound) of every token, in 64 bits; a row that
    sees nothing has O = 0 and LSE = -inf, one of no sequence is left NaN."""
    Hq, Hkv, d = c["heads"]
    G = Hq // Hkv
    T = c["q"].shape[0]
    out = torch.full((T, Hq, d), float("nan"), dtype=torch.float64)
    bound = torch.zeros_like(out)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64)
    lse_bound = torch.zeros_like(lse)
    pk, pv = _keys(c["k"], c["prefix"], c["P"]), _keys(c["v"], c["prefix"], c["P"])
    for s, n in enumerate(c["new"]):
        m = c["lens"][s]
        ids = c["table"][s, :-(-m // c["page"])]
        k = torch.cat((pk, _keys(c["k"], ids, m)), 1)
        v = torch.cat((pv, _keys(c["v"], ids, m)), 1)
        for i in range(n):
            t = int(c["start"][s]) + i
            seen = c["P"] + max(0, m - n + i + 1)
            if seen == 0:
                out[t], lse[t] = 0.0, -math.inf
                continue
            q = c["q"][t].double().view(Hkv, G, d)
            ks, vs = k[:, :seen], v[:, :seen]
            x = c["scale"] * (q @ ks.transpose(1, 2))
            w = torch.softmax(x, -1)
            o = w @ vs
            top = (c["scale"] * (q.abs() @ ks.abs().transpose(1, 2))).amax(-1, keepdim=True)
            delta = (2 * d + 4) * U * top + 160 * U
            apart = torch.einsum("hgk,hgkd->hgd", w, (vs[:, None] - o[:, :, None]).abs())
            err = (H / (1 - H) + 2 * delta) * apart + 2 * (seen + 64) * U * (w @ vs.abs())
            out[t] = o.reshape(Hq, d)
            bound[t] = (err + H * (o.abs() + err)).reshape(Hq, d)
            lse[t] = torch.logsumexp(x, -1).reshape(Hq)
            lse_bound[t] = (delta[..., 0] + 2 * seen * U
                            + 4 * U * torch.logsumexp(x, -1).abs()).reshape(Hq)
    return out, bound, lse, lse_bound


def check(c, o, lse, rows=None):
    """Every row of a sequence (or the given ones) within its bound."""
    want, bound, want_lse, lse_bound = exact(c)
    o, lse = o.cpu().double(), lse.cpu().double()
    first = int(c["start"][0])
    rows = list(range(first, first + sum(c["new"]))) if rows is None else rows
    for t in rows:
        assert torch.isfinite(o[t]).all(), f"row {t}"
        worst = ((o[t] - want[t]).abs() - bound[t]).max().item()
        assert worst <= 0, f"row {t}: O beyond the bound by {worst}"
        if torch.isinf(want_lse[t]).all():
            assert torch.equal(lse[t], want_lse[t])
            continue
        worst = ((lse[t] - want_lse[t]).abs() - lse_bound[t]).max().item()
        assert worst <= 0, f"row {t}: LSE beyond the bound by {worst}"
