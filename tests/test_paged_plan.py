"""How attention over a paged cache divides its work, seen from outside: the
tiles of a short batch's prefix, the CTAs for them, and rows of very many
partial results."""
import pytest
import torch

import exact_attention_109_b200 as fa
import paged_ref as ref
from test_paged import run

gpu = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,n,Hq,Hkv,P", [(2, 8, 1, 1, 4096), (1, 16, 1, 1, 1000), (2, 4, 4, 2, 640),
                                          (9, 1, 2, 2, 2000)])
def test_ctas_for_every_tile_of_a_prefix_in_the_line(S, n, Hq, Hkv, P, d):
    """A CTA for each block of 64 keys, of the prefix's tiles too, as long as the
    GPU has them: two tiles of 8 rows where no sequence has more than 8, one of
    16 otherwise."""
    T, G = S * n, Hq // Hkv
    tile = 8 if n * G <= 8 else 16
    blocks = (S * -(-n * G // tile) + -(-T * G // tile) * -(-P // 64)) * Hkv  # 1 block of own keys
    assert blocks <= 296
    st, splits, _, ctas = fa.fa_paged_split_plan(S, T, Hq, Hkv, d, 16, 4, P, n, 148)
    assert st == fa.FA_OK and splits == 0 and ctas == blocks


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,n,Hq,Hkv", [(8, 1, 2, 2), (9, 1, 1, 1), (16, 1, 2, 2), (4, 1, 6, 2),
                                        (2, 8, 1, 1), (2, 4, 4, 2), (1, 16, 1, 1)])
def test_up_to_sixteen_rows_read_a_long_prefix_once(S, n, Hq, Hkv, d):
    """A long prefix of up to 16 query rows a key head is one tile of the line, so
    that its keys are streamed once.  The workspace begins with the table of
    tiles [own, prefix][Hkv][rows], whose second word ends (mod 16) in the row's
    place in its tile."""
    T, rows, P = S * n, S * n * (Hq // Hkv), 5000
    c = ref.make([n] * S, [n + 5 * i for i in range(S)], P, Hq, Hkv, d, 16, seed=rows)
    need = fa.fa_paged_workspace_size(S, T, Hq, Hkv, d, 16, c["table"].shape[1], P, n)
    ws = torch.zeros(need // 4, dtype=torch.int32, device="cuda")
    out, lse = run(c, workspace=ws)
    assert fa.fa_get_device_error() == fa.FA_OK
    ref.check(c, out, lse)
    prefix = ws[:4 * Hkv * rows].view(2, Hkv, rows, 2)[1].cpu()
    assert (prefix[..., 1] % 16 == torch.arange(rows)).all()


@gpu
@pytest.mark.parametrize("rows,P,n,d", [
    (17, 20000, 40, 64),     # splits of the prefix, two results of each
    (40, 40001, 3, 64),
    (17, 30000, 500, 128),
    (1030, 6000, 2, 64),     # one warp a row joins them
    (3, 20000, 9000, 128),   # pieces of a prefix in the line and of own keys
    (16, 30001, 20, 64),
])
def test_rows_of_many_partial_results(rows, P, n, d):
    """Rows that the merge joins from very many parts; the log-sum-exp's error,
    counted by their number.  In units of u = 2^-24, and with X the row's largest
    sum of |q k| * scale: a score is off by 2 d X, and by 4 X for its scaling and
    the maximum's subtraction; a part's sum over its own keys by 2 a key; its
    log-sum-exp is rounded at its magnitude on the way out and as the row's
    (5 of that with the changes of base); its weight is off by 8; and each part
    adds a product, a sum and at most one scaling to the row's sums (3), before
    the joining of warps (16).

    The bounds of paged_ref hold too, although they count the merge as that of
    16 parts: they allow 2 u for every key in one sum, and R parts, each of a
    key at least, leave 2 (R - 1) of that unused beside the 160 of the merge;
    parts beyond the first three are of 64 keys or more."""
    c = ref.make([1] * rows, [n] * rows, P, 1, 1, d, 64, seed=rows)
    out, lse = run(c)
    assert fa.fa_get_device_error() == fa.FA_OK
    ref.check(c, out, lse)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _, splits, chunk, ctas = fa.fa_paged_split_plan(rows, rows, 1, 1, d, 64, c["table"].shape[1],
                                                    P, 1, sms)
    # The line: every sequence one tile, of two blocks more than its keys.
    own, pre = -(-n // 64), 0 if splits else -(-P // 64)
    quota = max(2, -(-(rows * (own + 2) + (pre + 2 if pre else 0)) // ctas))
    pieces = sum(-(-b // quota) + 1 for b in (own, pre) if b)
    parts = splits * (2 if d == 64 and rows <= 64 else 1) + pieces
    assert parts > 16
    k = ref._keys(c["k"], c["prefix"], P)[0]
    for t in range(0, rows, 7):
        keys = torch.cat((k, ref._keys(c["k"], c["table"][t, :own], n)[0]))
        q = c["q"][t, 0].double()
        top = c["scale"] * (keys.abs() @ q.abs()).max()
        want = torch.logsumexp(c["scale"] * (keys @ q), 0)
        units = (2 * d + 4) * top + 2 * max(chunk, 64 * quota) + 5 * want.abs() + 24 + 3 * parts
        assert abs(lse[t, 0].item() - want.item()) <= ref.U * units.item()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,n,Hq,Hkv", [(9, 1, 1, 1), (16, 1, 2, 2), (2, 8, 1, 1), (4, 1, 6, 2),
                                        (2, 20, 4, 1), (40, 1, 8, 8)])
def test_a_workspace_for_a_longer_prefix_is_enough(S, n, Hq, Hkv, d):
    """A server sizes its workspace for the longest prefix that it holds."""
    for pages in (1, 3):
        size = [fa.fa_paged_workspace_size(S, S * n, Hq, Hkv, d, 16, pages, P, n)
                for P in (0, 1, 64, 700, 2000, 4000, 4096, 4097, 4200, 5000, 8000, 9000, 65536)]
        assert all(a <= b for a, b in zip(size, size[1:]))
