"""Attention of packed new tokens over a paged cache behind a shared prefix
(fa_fwd_paged) against the definition in 64 bits; its split plan and refusals
on the CPU; and the whole path of a server's step."""
import pytest
import torch

import exact_attention_109_b200 as fa
import norm_rope_ref
import paged_ref as ref

gpu = pytest.mark.gpu
FAKE = 1 << 20  # aligned, never dereferenced: every case fails validation first
NAN = float("nan")

SIZES = dict(S=2, T=5, Hq=4, Hkv=2, d=128, page_size=16, max_pages=3, prefix_len=40, max_new=3)
ARGS = dict(q=FAKE, k_pages=FAKE, v_pages=FAKE, block_table=FAKE, seq_start=FAKE, kv_len=FAKE,
            prefix_pages=FAKE, o=FAKE, lse=FAKE, num_pages=9, scale=0.1, workspace=FAKE,
            workspace_bytes=1 << 30, **SIZES)


@pytest.mark.parametrize("kwargs,status", [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(lse=0), fa.FA_ERR_INVALID_ARG),
    (dict(kv_len=0), fa.FA_ERR_INVALID_ARG),
    (dict(prefix_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(workspace=0), fa.FA_ERR_INVALID_ARG),
    (dict(workspace_bytes=100), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(scale=3e38), fa.FA_ERR_INVALID_ARG),  # times log2(e): infinite
    (dict(S=0), fa.FA_ERR_INVALID_ARG),
    (dict(T=-1), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=5), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_new=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_new=6), fa.FA_ERR_INVALID_ARG),
    (dict(prefix_len=-1), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=8), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=24), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=512), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=1 << 30), fa.FA_ERR_INVALID_ARG),
    (dict(T=1 << 23), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=1 << 27), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(q=FAKE + 2), fa.FA_ERR_MISALIGNED),
    (dict(v_pages=FAKE + 8), fa.FA_ERR_MISALIGNED),
    (dict(workspace=FAKE + 16), fa.FA_ERR_MISALIGNED),
    (dict(kv_len=FAKE + 1), fa.FA_ERR_MISALIGNED),
])
def test_rejects_bad_arguments(kwargs, status):
    assert fa.fa_fwd_paged(**{**ARGS, **kwargs}) == status


def test_no_new_tokens_is_no_work():
    assert fa.fa_fwd_paged(**{**ARGS, "T": 0}) == fa.FA_OK


@pytest.mark.parametrize("page_size", [16, 64, 256])
@pytest.mark.parametrize("P", [0, 1, 127, 128, 129, 5000, 65536])
@pytest.mark.parametrize("S,max_new,Hq,Hkv", [(1, 1, 1, 1), (1, 1, 16, 16), (3, 1, 8, 2),
                                              (64, 1, 32, 8), (128, 1, 32, 4), (16, 4, 32, 32),
                                              (2, 700, 8, 1), (500, 1, 64, 8)])
def test_split_plan_covers_the_keys_within_the_workspace(S, max_new, Hq, Hkv, P, page_size):
    """Every prefix split has keys, none is left over, and the partial results
    of any plan (whatever the GPU) fit the workspace."""
    T = S * max_new
    for d in (64, 128):
        for max_pages in (1, 7, 600):
            size = (S, T, Hq, Hkv, d, page_size, max_pages, P, max_new)
            have = fa.fa_paged_workspace_size(*size)
            for sms in (1, 80, 148, 1000):
                st, splits, chunk, ctas = fa.fa_paged_split_plan(*size, sms)
                assert st == fa.FA_OK and 1 <= ctas <= 3 * sms
                in_line = T * Hq // Hkv <= 16
                assert (splits == 0) == (P == 0 or in_line)
                if splits:
                    assert chunk % 128 == 0 and (splits - 1) * chunk < P <= splits * chunk
                twice = 2 if d == 64 and T * Hq // Hkv <= 64 else 1
                slots = 0 if P == 0 else 1 + (1 if in_line else twice * splits)
                rows = slots * T * Hq + ctas * 2 * 16
                assert 2 * T * Hq * 8 + rows * (d + 1) * 4 <= have


def test_split_plan_refuses_what_the_call_refuses():
    good = (2, 5, 4, 2, 128, 16, 3, 40, 3)
    assert fa.fa_paged_split_plan(*good, 148)[0] == fa.FA_OK
    assert fa.fa_paged_split_plan(*good, 0)[0] == fa.FA_ERR_INVALID_ARG
    for i, bad in [(0, 0), (2, 3), (5, 20), (6, 0), (7, -1), (8, 0), (8, 6)]:
        size = good[:i] + (bad,) + good[i + 1:]
        assert fa.fa_paged_split_plan(*size, 148)[0] == fa.FA_ERR_INVALID_ARG
        assert fa.fa_paged_workspace_size(*size) == 0
    assert fa.fa_paged_split_plan(*good[:4], 80, *good[5:], 148)[0] == fa.FA_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors():
    c = ref.make([1], [3], 0, 2, 1, 64, 16, seed=0)
    with pytest.raises(ValueError, match="CUDA"):
        fa.attention_paged(c["q"], c["k"], c["v"], c["table"], c["start"], c["len"], 0.1)


# ---------------------------------------------------------------- GPU

def run(c, **kw):
    g = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    Hq, _, d = c["heads"]
    T = c["q"].shape[0]
    out = torch.full((T, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, Hq), 5.0, device="cuda")
    kw.setdefault("max_new", max(1, max(c["new"])))
    fa.attention_paged(g["q"], g["k"], g["v"], g["table"], g["start"], g["len"], c["scale"],
                       prefix_pages=g["prefix"], prefix_len=c["P"], out=out, lse=lse, **kw)
    return out, lse


def untouched(c, out, lse):
    first, last = int(c["start"][0]), int(c["start"][-1])
    for rows in (slice(0, first), slice(last, None)):
        assert (out[rows] == 3).all() and (lse[rows] == 5).all()


def check(c, **kw):
    out, lse = run(c, **kw)
    assert fa.fa_get_device_error() == fa.FA_OK
    ref.check(c, out, lse)
    untouched(c, out, lse)
    return out, lse


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,lens,P,Hq,Hkv,page", [
    ([1], [1], 0, 1, 1, 16),
    ([1], [1], 1, 1, 1, 16),
    ([1], [64], 127, 4, 4, 16),
    ([1], [65], 128, 4, 2, 32),
    ([1], [37], 1024, 16, 16, 16),
    ([1, 1, 1], [1, 300, 17], 129, 8, 2, 64),
    ([1] * 9, [1, 15, 16, 17, 63, 64, 65, 255, 257], 300, 8, 1, 128),
    ([2, 4, 1, 3], [2, 130, 90, 5], 500, 8, 8, 16),
    ([3, 0, 1, 0, 4], [70, 0, 1, 9, 1000], 77, 6, 2, 256),
    ([1] * 20, list(range(1, 400, 20)), 1000, 16, 2, 32),
    ([4] * 40, list(range(4, 44)), 640, 8, 4, 16),
    ([1] * 130, list(range(1, 131)), 260, 6, 3, 16),
    ([1], [5000], 0, 4, 1, 64),
    ([40, 17], [100, 17], 200, 4, 2, 16),
    ([100], [100], 0, 2, 2, 32),
    ([300, 1], [777, 40], 129, 3, 1, 64),
    ([1, 1], [3, 2], 4000, 8, 8, 128),
])
def test_paged(new, lens, P, Hq, Hkv, page, d):
    check(ref.make(new, lens, P, Hq, Hkv, d, page, seed=sum(lens) + P + d, pad=2, lead=1))


@gpu
@pytest.mark.parametrize("P", [0, 64])
def test_rows_that_see_no_key_of_their_own(P):
    """More new tokens than keys: the first ones see the prefix alone, or
    nothing (O = 0, LSE = -inf)."""
    c = ref.make([3, 2, 1], [1, 0, 0], P, 4, 2, 64, 16, seed=1)
    out, lse = check(c)
    if P == 0:
        assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("poison", [NAN, float("inf"), -float("inf")])
def test_unseen_values_reach_nobody(poison, d):
    """Rows behind a sequence's last key, behind the prefix and (for the
    earlier tokens) the later tokens' own rows hold infinities or NaN."""
    c = ref.make([4, 1, 20], [70, 16, 33], 100, 6, 2, d, 16, seed=d, fill=poison)
    good, good_lse = check(c)
    for s in (0, 2):  # the last token's key and value
        j = c["lens"][s] - 1
        page, row = int(c["table"][s, j // 16]), j % 16
        for which in ("k", "v"):
            bad = dict(c, **{which: c[which].clone()})
            bad[which][page, :, row] = poison
            out, lse = run(bad)
            last = int(c["start"][s + 1]) - 1
            rest = [t for t in range(25) if t != last]
            # where the values had to be added row by row the sums' order differs
            ref.check(c, out, lse, rest)
            assert not torch.isfinite(out[last].float()).all()
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
def test_nan_queries_stay_in_their_rows():
    """A NaN query gives NaN (not the zeros of a row that sees nothing), with
    the prefix, without it, over one split and over several."""
    for P, n in ((0, 20), (0, 3000), (200, 20), (2000, 3000)):
        c = ref.make([1, 1], [n, n], P, 4, 2, 128, 16, seed=n)
        c["q"][0, 1, 5] = NAN
        out, lse = run(c)
        assert torch.isnan(out[0, 1].float()).all() and torch.isnan(lse[0, 1])
        c["q"][0, 1, 5] = 0.0
        keep = [h for h in range(4) if h != 1]
        want, want_lse = run(c)
        assert torch.equal(out[0, keep], want[0, keep]) and torch.equal(out[1], want[1])
        assert torch.equal(lse[0, keep], want_lse[0, keep])


@gpu
@pytest.mark.parametrize("P", [0, 300])
def test_large_and_rising_scores(P):
    """Scores of +-100 and more whose maximum keeps moving."""
    c = ref.make([2, 1], [500, 400], P, 4, 2, 128, 16, seed=6)
    c["k"] = c["k"] * torch.linspace(0.1, 30, c["k"].shape[0]).view(-1, 1, 1, 1).bfloat16()
    check(c)


@gpu
def test_loose_bound_and_workspace_reuse():
    """max_new left at its default, and a workspace that was used and holds NaN."""
    c = ref.make([1, 3, 2], [40, 700, 90], 333, 8, 4, 64, 32, seed=7)
    out, lse = check(c)
    loose, loose_lse = check(c, max_new=None)
    assert torch.allclose(out.float(), loose.float(), atol=2 ** -6)
    need = fa.fa_paged_workspace_size(3, 6, 8, 4, 64, 32, c["table"].shape[1], 333, 3)
    ws = torch.full((need // 4,), NAN, device="cuda")
    again, again_lse = check(c, workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    with pytest.raises(Exception, match="fa_fwd_paged"):
        run(c, workspace=ws[:-64])


@gpu
@pytest.mark.parametrize("fault", ["page_high", "page_negative", "length_long", "length_negative",
                                   "prefix_page", "many_new", "start_decreases", "start_late"])
def test_bad_index_is_reported(fault):
    """A page, a length or a count out of range is reported; the other
    sequences' rows come out as before."""
    c = ref.make([2, 2, 2], [20, 30, 40], 50, 4, 2, 64, 16, seed=8, fill=0.0)
    good = run(c)
    bad = dict(c, table=c["table"].clone(), len=c["len"].clone(), prefix=c["prefix"].clone())
    kw = {}
    if fault == "page_high":
        bad["table"][1, 0] = c["k"].shape[0]
    elif fault == "page_negative":
        bad["table"][1, 1] = -1
    elif fault == "length_long":
        bad["len"][1] = 2 ** 31 - 1
        bad["table"][1] = c["table"][1, 0]
    elif fault == "length_negative":
        bad["len"][1] = -5
    elif fault == "prefix_page":
        bad["prefix"][1] = 1 << 20
    elif fault == "many_new":
        kw["max_new"] = 1
    elif fault == "start_decreases":
        bad["start"] = torch.tensor([0, 4, 2, 6], dtype=torch.int32)
        kw["max_new"] = 4
    else:
        bad["start"] = torch.tensor([0, 2, 4, 7], dtype=torch.int32)
    out, lse = run(bad, **kw)
    assert fa.fa_get_device_error() == fa.FA_ERR_INDEX
    assert fa.fa_get_device_error() == fa.FA_OK
    if fault.startswith(("page", "length")):
        for a, b in ((out, good[0]), (lse, good[1])):
            assert torch.equal(a[:2], b[:2]) and torch.equal(a[4:], b[4:])


@gpu
def test_two_sequences_may_share_pages():
    """The same pages under two sequences, and the prefix's pages again as own ones."""
    c = ref.make([1, 1, 1], [50, 50, 64], 64, 4, 2, 128, 16, seed=9)
    c["table"][1] = c["table"][0]
    c["table"][2, :4] = c["prefix"]
    out, _ = check(c)


@gpu
def test_prefix_is_the_same_as_own_keys():
    """Splitting the same keys differently between prefix and own rows."""
    Hq, Hkv, d, page, n = 8, 2, 128, 32, 640
    base = ref.make([1], [n], 0, Hq, Hkv, d, page, seed=10)
    check(base)
    for shared in (1, 7, 19):
        c = dict(base, prefix=base["table"][0, :shared].clone(), P=shared * page,
                 lens=[n - shared * page], len=torch.tensor([n - shared * page], dtype=torch.int32),
                 table=base["table"][:, shared:].contiguous())
        check(c)


@gpu
def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 values, used at both ends."""
    page, d, n = 256, 128, 700
    pages = 2 ** 31 // (page * d) + 5
    kp = torch.empty(pages, 1, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    c = ref.make([2], [n], 300, 4, 1, d, page, seed=11, spare=0)
    use = torch.tensor([pages - 1, 0, pages - 3, 2, pages - 2], dtype=torch.int32)
    assert use.numel() == c["k"].shape[0]
    kp[use.long().cuda()], vp[use.long().cuda()] = c["k"].cuda(), c["v"].cuda()
    table = c["table"].clone()
    table[0, :3] = use[c["table"][0, :3].long()]
    out, lse = fa.attention_paged(c["q"].cuda(), kp, vp, table.cuda(), c["start"].cuda(),
                                  c["len"].cuda(), c["scale"], max_new=2,
                                  prefix_pages=use[c["prefix"].long()].cuda(), prefix_len=300)
    assert fa.fa_get_device_error() == fa.FA_OK
    ref.check(c, out, lse)


@gpu
def test_other_streams_and_two_calls_at_once():
    cs = [ref.make([1] * 6, [100 * i + 50 for i in range(6)], 2000 + i, 8, 2, 128, 16, seed=12 + i)
          for i in range(2)]
    want = [run(c) for c in cs]
    gs = [{n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()} for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(5):
        for i, (g, st) in enumerate(zip(gs, streams)):
            got[i].append(fa.attention_paged(
                g["q"], g["k"], g["v"], g["table"], g["start"], g["len"], g["scale"],
                prefix_pages=g["prefix"], prefix_len=g["P"], max_new=1, stream=st))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for o, l in runs:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])
    assert fa.fa_get_device_error() == fa.FA_OK


def _step(fa, x, kp, vp, table, start, have, rope, weights, prefix, P, heads, scale):
    """One step of a server: the projection's rows in, attention's out."""
    q, k, v = x.split([heads[0], heads[1], heads[1]], dim=1)
    q = fa.paged_append(q, k, v, kp, vp, table, start, have, rope=rope, pos_offset=P,
                        q_weight=weights[0], k_weight=weights[1])
    total = have + (start[1:] - start[:-1])
    return fa.attention_paged(q, kp, vp, table, start, total, scale, prefix_pages=prefix,
                              prefix_len=P)[0], total


@gpu
@pytest.mark.parametrize("Hq,Hkv,d,page,P", [(4, 4, 128, 16, 100), (8, 2, 64, 32, 0)])
def test_a_servers_path_matches_the_forward_pass(Hq, Hkv, d, page, P):
    """Prompt into the prefix, a second prompt chunk and drafted tokens behind
    it, step by step, against one causal forward pass over the whole sequence
    after fa_qk_norm_rope; the step is captured once and replayed."""
    torch.manual_seed(3)
    S, chunks = 2, [70, 1, 1, 3, 1]
    n = P + sum(chunks)
    x = torch.randn(S, n, Hq + 2 * Hkv, d, device="cuda").bfloat16()
    x[:, :P] = x[:1, :P]
    w = [(1 + 0.2 * torch.randn(d, device="cuda")).bfloat16() for _ in range(2)]
    rope = fa.rope_table(n, d)
    q, k, v = x.split([Hq, Hkv, Hkv], dim=2)
    qn, kn, vn = fa.qk_norm_rope(q, k, v, *w, rope=rope)
    G = Hq // Hkv
    want, _ = fa.attention_forward(qn, kn.repeat_interleave(G, 1), vn.repeat_interleave(G, 1),
                                   True, d ** -0.5)
    want = want.transpose(1, 2).float()  # [S, n, Hq, d]
    # Both sides round weights (by h = 2^-8, which moves O by at most
    # sum w |v - O| <= max|v| + |O| times that) and O itself.
    bound = 2.02 * ref.H * (v.abs().max().float() + 2 * want.abs()) + 1e-3

    per, shared = -(-sum(chunks) // page), -(-P // page)
    kp = torch.zeros(S * per + shared, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    order = torch.randperm(S * per + shared, device="cuda").int()
    prefix, table = order[:shared].contiguous(), order[shared:].view(S, per).contiguous()
    if P:  # the prefix comes in as one sequence
        one = torch.tensor([0, P], dtype=torch.int32, device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        got, _ = _step(fa, x[0, :P], kp, vp, prefix[None], one, zero, rope, w, None, 0, (Hq, Hkv),
                       d ** -0.5)
        assert ((got.float() - want[0, :P]).abs() <= bound[0, :P]).all()
    have = torch.zeros(S, dtype=torch.int32, device="cuda")
    at = P
    for m in chunks:
        rows = x[:, at:at + m].reshape(S * m, Hq + 2 * Hkv, d)
        start = torch.arange(S + 1, dtype=torch.int32, device="cuda") * m
        args = (rows, kp, vp, table, start, have, rope, w, prefix, P, (Hq, Hkv), d ** -0.5)
        got, total = _step(fa, *args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            replayed, _ = _step(fa, *args)
        graph.replay()
        assert torch.equal(got, replayed)
        apart = (got.view(S, m, Hq, d).float() - want[:, at:at + m]).abs()
        assert (apart <= bound[:, at:at + m]).all()
        have, at = total, at + m
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
def test_two_graphs_share_a_workspace():
    """Two captured steps with one workspace, replayed in turn on a stream, while
    their lengths move between replays."""
    cs = [ref.make([1, 1], [60, 600], 500, 4, 4, 64, 16, seed=20 + i) for i in range(2)]
    gs = [{n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()} for c in cs]
    need = fa.fa_paged_workspace_size(2, 2, 4, 4, 64, 16, cs[0]["table"].shape[1], 500, 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []

    def call(g, out, lse):
        fa.attention_paged(g["q"], g["k"], g["v"], g["table"], g["start"], g["len"], g["scale"],
                           prefix_pages=g["prefix"], prefix_len=500, max_new=1, out=out, lse=lse,
                           workspace=ws)

    for g in gs:
        out, lse = torch.empty_like(g["q"]), torch.empty(2, 4, device="cuda")
        call(g, out, lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(g, out, lse)
        outs.append((out, lse))
        graphs.append(graph)
    for lens in ([60, 600], [1, 600], [33, 64]):
        for g in gs:
            g["len"].copy_(torch.tensor(lens, dtype=torch.int32))
        for o, l in outs:
            o.zero_(), l.zero_()
        for graph in graphs + graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, (o, l) in zip(cs, outs):
            ref.check(dict(c, lens=lens), o, l)


@gpu
@pytest.mark.parametrize("before", ["memset", "copy", "kernel", "other_stream", "nothing"])
def test_order_behind_other_work(before):
    """The calls start while the stream's previous work ends; what that wrote is
    seen all the same, eagerly and in a captured graph, whatever kind it is."""
    c = ref.make([1, 2], [40, 700], 300, 8, 4, 64, 16, seed=30)
    want = run(c)
    g = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    q, lens = torch.zeros_like(g["q"]), torch.zeros_like(g["len"])
    big = torch.zeros(64 << 20, device="cuda")
    side = torch.cuda.Stream()

    def step():
        if before == "nothing":
            q.copy_(g["q"])
        elif before == "memset":
            big.zero_()
            q.copy_(g["q"])
            lens.zero_()
            lens.add_(g["len"])
            big.zero_()
        elif before == "copy":
            lens.copy_(g["len"])
            big.add_(1)
            q.copy_(g["q"])
        elif before == "kernel":
            big.add_(1)
            torch.add(g["len"], 0, out=lens)
            torch.mul(g["q"], 1, out=q)
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                big.add_(1)
                q.copy_(g["q"])
                lens.copy_(g["len"])
            torch.cuda.current_stream().wait_stream(side)
        n = g["len"] if before == "nothing" else lens
        return fa.attention_paged(q, g["k"], g["v"], g["table"], g["start"], n, c["scale"],
                                  prefix_pages=g["prefix"], prefix_len=c["P"], max_new=2)

    def reset():
        q.fill_(NAN), lens.fill_(1)
        torch.cuda.synchronize()

    for _ in range(3):
        reset()
        got = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_steps_in_a_row_keep_their_order():
    """Twenty decoding steps without a host wait, each reading what the one
    before appended, against the same steps one at a time."""
    torch.manual_seed(5)
    S, Hq, Hkv, d, page = 3, 8, 2, 128, 16
    x = torch.randn(20, S, Hq + 2 * Hkv, d, device="cuda").bfloat16()
    rope = fa.rope_table(64, d)
    w = [torch.ones(d, device="cuda") for _ in range(2)]
    table = torch.randperm(S * 4, device="cuda").int().view(S, 4)
    start = torch.arange(S + 1, dtype=torch.int32, device="cuda")

    def steps(wait):
        kp = torch.zeros(S * 4, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
        vp, have, outs = torch.zeros_like(kp), torch.tensor([0, 5, 17]).int().cuda(), []
        for i in range(20):
            o, have = _step(fa, x[i], kp, vp, table, start, have, rope, w, None, 0, (Hq, Hkv),
                            d ** -0.5)
            outs.append(o)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return torch.stack(outs), kp, vp

    want = steps(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
@pytest.mark.parametrize("P", [0, 70])
def test_many_sequences(P):
    """More sequences than threads, some without tokens, in a table without spare columns."""
    gen = torch.Generator().manual_seed(31)
    new = torch.randint(0, 3, (1300,), generator=gen).tolist()
    lens = [max(n, int(x)) for n, x in zip(new, torch.randint(0, 97, (1300,), generator=gen))]
    c = ref.make(new, lens, P, 2, 1, 64, 32, seed=31)
    c["table"] = c["table"][:, :-2].contiguous()
    check(c)


@gpu
@pytest.mark.parametrize("Hkv,n,d", [(1, 30000, 64), (2, 9000, 128)])
def test_one_sequence_over_the_whole_gpu(Hkv, n, d):
    """A row tile whose keys all CTAs share: hundreds of partial results a row."""
    check(ref.make([2], [n], 0, 4 * Hkv, Hkv, d, 128, seed=32))


@gpu
def test_more_row_tiles_than_splits():
    """A prefix whose query rows alone fill the GPU."""
    check(ref.make([300, 280, 310, 290], [300, 500, 310, 290], 400, 16, 2, 64, 64, seed=33))


@gpu
def test_rows_of_two_row_tiles_see_their_own_keys():
    """Prompt chunks of many rows, whose tiles begin and end inside a token."""
    check(ref.make([33, 7, 50], [200, 7, 129], 0, 10, 2, 128, 16, seed=34))
    check(ref.make([33, 7, 50], [200, 7, 129], 130, 6, 2, 64, 256, seed=35))


@gpu
@pytest.mark.parametrize("rows", [17, 32, 33, 63, 64, 65, 128, 129])
@pytest.mark.parametrize("P", [1, 63, 64, 65, 127, 190, 700])
def test_rows_and_ends_of_the_prefix(rows, P):
    """Row counts around those of the prefix kernel's forms, prefixes that end in
    the first or second half of a block."""
    for d in (64, 128):
        c = ref.make([1] * rows, [1 + 3 * (i % 5) for i in range(rows)], P, 1, 1, d, 16,
                     seed=rows + P)
        check(c)
