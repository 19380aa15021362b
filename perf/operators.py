"""Measured cases of the operators around attention: norms and rotation of
queries and keys (forward and backward), appending to a paged cache, and
attention of a batch over a paged cache behind a shared prefix.

``run`` computes each operator in elementary torch operations when ``own`` is
false, and through this repository's entry points when it is true.
"""
import math
import random

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # The projection of a training step of 2 x 8192 tokens, 16 heads of 128.
        dict(name="norm_rope_16k", op="norm_rope", B=2, N=8192, Hq=16, Hkv=16, d=128, rope=128,
             interleaved=False, w32=False, packed=False),
        # A ragged small batch: grouped heads of 64, half of each row rotated in
        # neighbouring pairs, positions that restart inside a row of documents.
        dict(name="norm_rope_odd", op="norm_rope", B=3, N=517, Hq=32, Hkv=8, d=64, rope=32,
             interleaved=True, w32=True, packed=True),
        # The gradients of the training step above.
        dict(name="norm_rope_grad_16k", op="norm_rope_grad", B=2, N=8192, Hq=16, Hkv=16, d=128,
             rope=128, interleaved=False, w32=False, packed=False),
        # The gradients of a short odd sequence with grouped heads.
        dict(name="norm_rope_grad_odd", op="norm_rope_grad", B=1, N=1023, Hq=16, Hkv=4, d=64,
             rope=64, interleaved=True, w32=True, packed=True),
        # One token of one conversation: latency.
        dict(name="append_one", op="append", S=1, new_min=1, new_max=1, cached=1000, Hq=16, Hkv=16,
             d=128, rope=128, interleaved=False, page=16, norm=False, lens=1),
        # One token for each of 64 conversations, grouped heads with norms.
        dict(name="append_batch", op="append", S=64, new_min=1, new_max=1, cached=2000, Hq=32,
             Hkv=8, d=128, rope=128, interleaved=False, page=64, norm=True, lens=2),
        # Thirteen prompts of different lengths brought in at once.
        dict(name="append_prompts", op="append", S=13, new_min=90, new_max=1500, cached=100, Hq=16,
             Hkv=16, d=128, rope=64, interleaved=True, page=32, norm=True, lens=3),
        # One conversation behind a short system prompt: latency.
        dict(name="prefix_one", op="paged", S=1, new_min=1, new_max=1, own_min=37, own_max=37,
             P=1024, Hq=16, Hkv=16, d=128, page=16, lens=4),
        # A batch of conversations behind one long system prompt, grouped heads.
        dict(name="prefix_chat", op="paged", S=64, new_min=1, new_max=1, own_min=1, own_max=1024,
             P=16384, Hq=32, Hkv=8, d=128, page=64, lens=5),
        # Up to four drafted tokens a sequence, heads of 64, an odd prefix.
        dict(name="prefix_drafts", op="paged", S=16, new_min=1, new_max=4, own_min=200,
             own_max=2900, P=8191, Hq=32, Hkv=32, d=64, page=16, lens=6),
        # Many short answers about one long document: the tensor cores count.
        dict(name="prefix_document", op="paged", S=128, new_min=1, new_max=1, own_min=64,
             own_max=512, P=65536, Hq=32, Hkv=4, d=128, page=128, lens=7),
        # No common prefix: sixteen long conversations, each over its own pages.
        dict(name="paged_16x8192", op="paged", S=16, new_min=1, new_max=1, own_min=8192,
             own_max=8192, P=0, Hq=16, Hkv=16, d=128, page=64, lens=8),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "append", "paged", "paged"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    if op in ("norm_rope", "norm_rope_grad"):
        return dict(op=op, B=_spread(rng, 1, 8), N=_spread(rng, 16, 16384), Hq=Hq, Hkv=Hkv, d=d,
                    rope=rng.choice([16, 32, 48, d // 2, d]), interleaved=rng.random() < 0.5,
                    w32=rng.random() < 0.5, packed=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    S = _spread(rng, 1, 128)
    if op == "append":
        most = _spread(rng, 1, 1500)
        return dict(op=op, S=S, new_min=rng.choice([1, (most + 1) // 2]), new_max=most,
                    cached=_spread(rng, 1, 4000), Hq=Hq, Hkv=Hkv, d=d,
                    rope=rng.choice([16, 32, 48, d // 2, d]), interleaved=rng.random() < 0.5,
                    page=page, norm=rng.random() < 0.5, lens=rng.randrange(1 << 20))
    most = _spread(rng, 8, 8192)
    new = rng.choice([1, 1, 2, 4])
    return dict(op=op, S=S, new_min=rng.choice([1, new]), new_max=new,
                own_min=max(new, rng.choice([1, most // 4, most])), own_max=max(new, most),
                P=rng.choice([0, _spread(rng, 64, 65536), _spread(rng, 64, 65536)]), Hq=Hq,
                Hkv=Hkv, d=d, page=page, lens=rng.randrange(1 << 20))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        top = [work(c) for c in listed() if c["op"] == case["op"]]
        if w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top):
            return case


def _counts(case):
    """New tokens and lengths of every sequence: part of the case, not of the seed."""
    rng = random.Random(case["lens"])
    new = [rng.randint(case["new_min"], case["new_max"]) for _ in range(case["S"])]
    if case["op"] == "append":
        return new, [rng.randint(0, case["cached"]) for _ in new]
    return new, [max(n, rng.randint(case["own_min"], case["own_max"])) for n in new]


def work(case):
    d, heads = case["d"], case["Hq"] + 2 * case["Hkv"]
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        tokens = case["B"] * case["N"]
        table = case["N"] * case["rope"] * 4
        normed = case["Hq"] + case["Hkv"]
        if case["op"] == "norm_rope":
            return dict(bytes=tokens * heads * d * 4 + table, flops=tokens * normed * d * 7)
        return dict(bytes=tokens * (heads * 2 + normed) * d * 2 + table,
                    flops=tokens * normed * d * 14)
    new, lens = _counts(case)
    tokens = sum(new)
    if case["op"] == "append":
        return dict(bytes=tokens * (heads * d * 4 + case["rope"] * 4),
                    flops=tokens * (case["Hq"] + case["Hkv"]) * d * (7 if case["norm"] else 3))
    own_keys = sum(lens)
    seen = sum(case["P"] + n - m + i + 1 for m, n in zip(new, lens) for i in range(m))
    return dict(bytes=(case["P"] + own_keys) * case["Hkv"] * d * 4
                + tokens * case["Hq"] * (d * 4 + 4), flops=4 * d * case["Hq"] * seen)


def _table(rows, rope, device):
    """(cos, sin) of position * 10000^(-2i / rope), from 64-bit angles."""
    inv = 10000.0 ** (-torch.arange(0, rope, 2, dtype=torch.float64, device=device) / rope)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack((ang.cos(), ang.sin()), -1).float().contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)

    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    heads = Hq + 2 * Hkv
    s = dict(case=case)
    if case["op"] in ("norm_rope", "norm_rope_grad"):
        B, N = case["B"], case["N"]
        kind = torch.float32 if case["w32"] else torch.bfloat16
        s["qkv"] = normal(B, N, heads, d).bfloat16()
        s["wq"] = (1 + 0.1 * normal(d)).to(kind)
        s["wk"] = (1 + 0.1 * normal(d)).to(kind)
        s["rope"] = _table(N, case["rope"], dev)
        s["positions"] = None
        if case["packed"]:  # documents of a few hundred tokens, one behind another
            at = torch.arange(N, device=dev)[None] + 37 * torch.arange(B, device=dev)[:, None]
            s["positions"] = (at % (N // 3 + 1)).int()
        if case["op"] == "norm_rope_grad":
            s["dq"] = normal(B, Hq, N, d).bfloat16()
            s["dk"] = normal(B, Hkv, N, d).bfloat16()
            s["dv"] = normal(B, Hkv, N, d).bfloat16()
        return s

    new, lens = _counts(case)
    page, S, T = case["page"], case["S"], sum(new)
    s["seq_start"] = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32,
                                  device=dev)
    P = case.get("P", 0)
    total = [n + (m if case["op"] == "append" else 0) for m, n in zip(new, lens)]
    need = [-(-n // page) for n in total]
    shared = -(-P // page)
    pages = sum(need) + shared + 8
    order = torch.randperm(pages, generator=gen, device=dev).int()
    s["prefix_pages"] = order[:shared].contiguous()
    table = torch.zeros(S, max(need) + 3, dtype=torch.int32, device=dev)
    rows = torch.repeat_interleave(torch.arange(S), torch.tensor(need)).to(dev)
    cols = torch.cat([torch.arange(n) for n in need]).to(dev)
    table[rows, cols] = order[shared:shared + sum(need)]
    s["table"] = table
    s["k_pages"] = normal(pages, Hkv, page, d).bfloat16()
    s["v_pages"] = normal(pages, Hkv, page, d).bfloat16()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["tokens"], s["most_new"], s["most"] = T, max(new), max(total)
    if case["op"] == "append":
        s["qkv"] = normal(T, heads, d).bfloat16()
        s["wq"] = (1 + 0.1 * normal(d)).bfloat16() if case["norm"] else None
        s["wk"] = (1 + 0.1 * normal(d)).bfloat16() if case["norm"] else None
        s["rope"] = _table(max(total), case["rope"], dev)
    else:
        s["q"] = normal(T, Hq, d).bfloat16()
        s["scale"] = d ** -0.5
    return s


# ------------------------------------------------------------ plain forms


def _turn(x, cs, interleaved, back=False):
    """x [..., heads, d] with its pairs turned by cs [..., rope / 2, 2]."""
    c, sn = cs[..., None, :, 0], cs[..., None, :, 1]
    sn = -sn if back else sn
    r = 2 * c.shape[-1]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((y, x[..., r:]), -1)


def _angles(s):
    case = s["case"]
    if s["positions"] is None:
        return s["rope"][:case["N"]].expand(case["B"], -1, -1, -1)
    return s["rope"][s["positions"].long()]


def _unit(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_norm_rope(s, q, k, v):
    il = s["case"]["interleaved"]
    cs = _angles(s)
    q = _turn(_unit(q.float()) * s["wq"].float(), cs, il)
    k = _turn(_unit(k.float()) * s["wk"].float(), cs, il)
    return [t.bfloat16().transpose(1, 2).contiguous() for t in (q, k, v)]


def _plain_grad_one(x, dy, w, cs, il):
    x, g = x.float(), _turn(dy.transpose(1, 2).float(), cs, il, back=True)
    rstd = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh, gw = x * rstd, g * w.float()
    dx = rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.bfloat16(), (g * xh).sum((0, 1, 2))


def _plain_norm_rope_grad(s, q, k):
    il = s["case"]["interleaved"]
    cs = _angles(s)
    dq, dwq = _plain_grad_one(q, s["dq"], s["wq"], cs, il)
    dk, dwk = _plain_grad_one(k, s["dk"], s["wk"], cs, il)
    return [torch.cat((dq, dk, s["dv"].transpose(1, 2)), 2), dwq, dwk]


def _sequence_of(s):
    """Each token's sequence, and its index among that sequence's tokens."""
    start = s["seq_start"].long()
    seq = torch.repeat_interleave(torch.arange(s["case"]["S"], device=start.device),
                                  start[1:] - start[:-1], output_size=s["tokens"])
    return seq, torch.arange(s["tokens"], device=start.device) - start[seq]


def _plain_append(s, q, k, v):
    case = s["case"]
    seq, i = _sequence_of(s)
    at = s["lens"].long()[seq] + i
    cs = s["rope"][at]
    q, k = q.float(), k.float()
    if case["norm"]:
        q, k = _unit(q) * s["wq"].float(), _unit(k) * s["wk"].float()
    q, k = _turn(q, cs, case["interleaved"]), _turn(k, cs, case["interleaved"])
    page = s["table"].long()[seq, at // case["page"]]
    s["k_pages"][page, :, at % case["page"]] = k.bfloat16()
    s["v_pages"][page, :, at % case["page"]] = v
    return [q.bfloat16(), s["k_pages"], s["v_pages"]]


def _rows(pages, table):
    """The cached rows [..., Hkv, keys, d] of the pages that `table` [..., n] names."""
    t = pages[table.long()].float().transpose(-4, -3)
    return t.flatten(-3, -2)


def _plain_paged(s):
    case = s["case"]
    S, Hkv, d, M = case["S"], case["Hkv"], case["d"], s["most_new"]
    G, T = case["Hq"] // Hkv, s["tokens"]
    seq, i = _sequence_of(s)
    q = s["q"].float().view(T, Hkv, G, d) * s["scale"]
    padded = q.new_zeros(S, M, Hkv, G, d)
    padded[seq, i] = q
    padded = padded.permute(0, 2, 1, 3, 4).reshape(S, Hkv, M * G, d)
    used = s["table"][:, :-(-s["most"] // case["page"])]
    own_s = padded @ _rows(s["k_pages"], used).transpose(-1, -2)
    counts = (s["seq_start"][1:] - s["seq_start"][:-1]).long()
    last = (s["lens"].long() - counts)[:, None] + torch.arange(M, device=q.device)
    hidden = torch.arange(own_s.shape[-1], device=q.device) > last[..., None]
    own_s = own_s.view(S, Hkv, M, G, -1).masked_fill(hidden[:, None, :, None], -math.inf)
    top = own_s.amax(-1)[seq, :, i]  # [T, Hkv, G]
    if case["P"]:
        pre_k = _rows(s["k_pages"], s["prefix_pages"])[:, :case["P"]]
        pre_s = q.permute(1, 0, 2, 3).reshape(Hkv, T * G, d) @ pre_k.transpose(-1, -2)
        top = torch.maximum(top, pre_s.amax(-1).view(Hkv, T, G).transpose(0, 1))
    high = q.new_zeros(S, M, Hkv, G)
    high[seq, i] = top
    own_p = torch.exp(own_s - high.transpose(1, 2)[..., None])
    own_o = own_p.reshape(S, Hkv, M * G, -1) @ _rows(s["v_pages"], used)
    out = own_o.view(S, Hkv, M, G, d)[seq, :, i]
    total = own_p.sum(-1)[seq, :, i]
    if case["P"]:
        pre_p = torch.exp(pre_s - top.transpose(0, 1).reshape(Hkv, T * G, 1))
        pre_o = pre_p @ _rows(s["v_pages"], s["prefix_pages"])[:, :case["P"]]
        out = out + pre_o.view(Hkv, T, G, d).transpose(0, 1)
        total = total + pre_p.sum(-1).view(Hkv, T, G).transpose(0, 1)
    lse = top + torch.log(total)
    return [(out / total[..., None]).bfloat16().view(T, Hkv * G, d), lse.reshape(T, Hkv * G)]


def run(s):
    case = s["case"]
    if case["op"] == "paged":
        if own:
            import exact_attention_109_b200 as fa
            return fa.attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"],
                                      s["seq_start"], s["lens"], s["scale"],
                                      prefix_pages=s["prefix_pages"], prefix_len=case["P"],
                                      max_new=s["most_new"])
        return _plain_paged(s)
    q, k, v = s["qkv"].split([case["Hq"], case["Hkv"], case["Hkv"]], dim=-2)
    if case["op"] == "append":
        if own:
            import exact_attention_109_b200 as fa
            q = fa.paged_append(q, k, v, s["k_pages"], s["v_pages"], s["table"], s["seq_start"],
                                s["lens"], rope=s["rope"], q_weight=s["wq"], k_weight=s["wk"],
                                eps=EPS, interleaved=case["interleaved"])
            return [q, s["k_pages"], s["v_pages"]]
        return _plain_append(s, q, k, v)
    if case["op"] == "norm_rope":
        if own:
            import exact_attention_109_b200 as fa
            return fa.qk_norm_rope(q, k, v, s["wq"], s["wk"], eps=EPS, rope=s["rope"],
                                   positions=s["positions"], interleaved=case["interleaved"])
        return _plain_norm_rope(s, q, k, v)
    if own:
        import exact_attention_109_b200 as fa
        grad = torch.empty_like(s["qkv"])
        dq, dk, dv = grad.split([case["Hq"], case["Hkv"], case["Hkv"]], dim=-2)
        got = fa.qk_norm_rope_backward(s["dq"], s["dk"], s["dv"], q, k, s["wq"], s["wk"], eps=EPS,
                                       rope=s["rope"], positions=s["positions"],
                                       interleaved=case["interleaved"], dq=dq, dk=dk, dv=dv)
        return [grad, got[3], got[4]]
    return _plain_norm_rope_grad(s, q, k)


# ------------------------------------------------------------ 64 bits


def _exact_rotation(x, cos, sin, interleaved):
    """x [tokens, heads, d] in 64 bits; every pair is one complex number times cos + i sin."""
    half = cos.shape[-1]
    if interleaved:
        z = torch.complex(x[..., 0:2 * half:2], x[..., 1:2 * half:2])
    else:
        z = torch.complex(x[..., :half], x[..., half:2 * half])
    z = z * torch.complex(cos, sin)[:, None]
    y = x.clone()
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def _exact_norm(x, w):
    return x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w


def _exact_norm_rope(s, b):
    """q, k, v of batch row b before and after, and its cosines and sines."""
    case = s["case"]
    at = torch.arange(case["N"], device=s["rope"].device) if s["positions"] is None \
        else s["positions"][b].long()
    cs = s["rope"][at].double()
    x = s["qkv"][b].double()
    q, k, v = x[:, :case["Hq"]], x[:, case["Hq"]:case["Hq"] + case["Hkv"]], \
        x[:, case["Hq"] + case["Hkv"]:]
    return q, k, v, cs[..., 0], cs[..., 1]


def _exact_norm_rope_grad(s):
    case, out = s["case"], []
    dws = [0.0, 0.0]
    for b in range(case["B"]):
        q, k, _, c, sn = _exact_norm_rope(s, b)
        parts = []
        for n, (x, dy, w) in enumerate(((q, s["dq"], s["wq"]), (k, s["dk"], s["wk"]))):
            g = _exact_rotation(dy[b].double().transpose(0, 1), c, -sn, case["interleaved"])
            r = 1 / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
            dws[n] = dws[n] + (g * x * r).sum((0, 1))
            along = (g * w.double() * x).sum(-1, keepdim=True) / x.shape[-1]
            parts.append(g * w.double() * r - x * r ** 3 * along)
        parts.append(s["dv"][b].double().transpose(0, 1))
        out.append(torch.cat(parts, 1))
    return [torch.stack(out)] + dws


def _exact_append(s):
    case = s["case"]
    new, lens = _counts(case)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    q_out, t = [], 0
    for i, (m, n) in enumerate(zip(new, lens)):
        at = torch.arange(n, n + m, device=k_pages.device)
        cs = s["rope"][at].double()
        x = s["qkv"][t:t + m].double()
        q, k, v = x[:, :case["Hq"]], x[:, case["Hq"]:case["Hq"] + case["Hkv"]], \
            x[:, case["Hq"] + case["Hkv"]:]
        if case["norm"]:
            q, k = _exact_norm(q, s["wq"].double()), _exact_norm(k, s["wk"].double())
        q_out.append(_exact_rotation(q, cs[..., 0], cs[..., 1], case["interleaved"]))
        k = _exact_rotation(k, cs[..., 0], cs[..., 1], case["interleaved"])
        page = s["table"][i].long()[at // case["page"]]
        k_pages[page, :, at % case["page"]] = k
        v_pages[page, :, at % case["page"]] = v
        t += m
    return [torch.cat(q_out), k_pages, v_pages]


def _exact_paged(s):
    case = s["case"]
    new, lens = _counts(case)
    d, Hkv, page = case["d"], case["Hkv"], case["page"]
    G = case["Hq"] // Hkv

    def keys(pages, ids, count):  # [Hkv, count, d]
        return pages[ids.long()].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :count]

    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    pk, pv = (keys(s[x], s["prefix_pages"], case["P"]) for x in ("k_pages", "v_pages"))
    t = 0
    for i, (m, n) in enumerate(zip(new, lens)):
        ids = s["table"][i, :-(-n // page)]
        k = torch.cat((pk, keys(s["k_pages"], ids, n)), 1)
        v = torch.cat((pv, keys(s["v_pages"], ids, n)), 1)
        for j in range(m):
            seen = case["P"] + n - m + j + 1
            q = s["q"][t].double().view(Hkv, G, d)
            x = s["scale"] * (q @ k[:, :seen].transpose(1, 2))
            lse[t] = torch.logsumexp(x, -1).view(-1)
            out[t] = (torch.softmax(x, -1) @ v[:, :seen]).view(-1, d)
            t += 1
    return [out, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "paged":
        return _exact_paged(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "norm_rope_grad":
        return _exact_norm_rope_grad(s)
    rows = []
    for b in range(case["B"]):
        q, k, v, c, sn = _exact_norm_rope(s, b)
        rows.append([_exact_rotation(_exact_norm(q, s["wq"].double()), c, sn, case["interleaved"]),
                     _exact_rotation(_exact_norm(k, s["wk"].double()), c, sn, case["interleaved"]),
                     v])
    return [torch.stack([r[n].transpose(0, 1) for r in rows]) for n in range(3)]
