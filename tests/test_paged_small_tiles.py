"""Infinities and NaN among keys that only some rows of a tile see, with so few
new tokens that the tiles of a sequence have 8 rows."""
import pytest
import torch

import exact_attention_109_b200 as fa
import paged_ref as ref
from test_paged import run

gpu = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@gpu
@pytest.mark.parametrize("poison", [NAN, INF, -INF])
@pytest.mark.parametrize("new,Hq,Hkv,P", [
    ([4, 1, 3], 4, 2, 0),              # 8 rows a tile
    ([4, 1, 3], 2, 2, 0),              # 4
    ([8, 2], 1, 1, 0),                 # 8 tokens' limits in one tile
    ([2, 4], 2, 1, 100),               # behind a prefix in the line, of two tiles of 8
    ([4, 1, 3], 2, 2, 100),            # and of one
    ([4, 1, 3, 4, 4, 4], 2, 2, 100),   # behind one whose rows stand twice (heads of 64)
])
@pytest.mark.parametrize("d", [64, 128])
def test_unseen_values_reach_nobody_in_small_tiles(new, Hq, Hkv, P, poison, d):
    """Few rows a sequence: the last token's own key and value, which the earlier
    tokens do not see, in the first and second half of 16 keys."""
    lens = [(70, 62, 16, 33, 48, 9)[i] + 8 for i in range(len(new))]
    c = ref.make(new, lens, P, Hq, Hkv, d, 16, seed=d + len(new), fill=poison)
    out, lse = run(c)
    ref.check(c, out, lse)
    for s, n in enumerate(new):
        if n == 1:
            continue
        for back in (1, 2):  # the last key, and the one before
            j = c["lens"][s] - back
            page, row = int(c["table"][s, j // 16]), j % 16
            end = int(c["start"][s + 1])
            seers = list(range(max(int(c["start"][s]), end - back), end))
            rest = [t for t in range(sum(new)) if t not in seers]
            for which in ("k", "v"):
                bad = dict(c, **{which: c[which].clone()})
                bad[which][page, :, row] = poison
                out, lse = run(bad)
                ref.check(c, out, lse, rest)
                assert not torch.isfinite(out[seers].float()).any(-1).any() or which == "k"
                assert not torch.isfinite(out[seers].float()).all()
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
def test_values_that_few_rows_see_are_added_exactly():
    """Eight tokens in one tile with a NaN value in the last token's row: the
    seven before it add every value row by row, in the first and second half of
    16 keys and in each warp's keys."""
    for d in (64, 128):
        for n in (8, 12, 16, 17, 40, 57, 64, 65, 130):
            c = ref.make([8], [n], 0, 1, 1, d, 16, seed=n + d)
            v = c["v"].clone()
            v[int(c["table"][0, (n - 1) // 16]), :, (n - 1) % 16] = NAN
            out, lse = run(dict(c, v=v))
            ref.check(c, out, lse, list(range(7)))
            assert torch.isnan(out[7].float()).all()
