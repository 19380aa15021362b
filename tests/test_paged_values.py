"""Infinities and NaN among the values of a shared prefix, in every form that
attention over it takes by its number of query rows: they reach the outputs
that the definition sends them to, and no others."""
import pytest
import torch

import exact_attention_109_b200 as fa
import paged_ref as ref
from test_paged import run

gpu = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def put(c, key, head, column, value):
    """A case like c with one value of the prefix's key replaced."""
    v = c["v"].clone()
    v[int(c["prefix"][key // c["page"]]), head, key % c["page"], column] = value
    return dict(c, v=v)


def check_column(c, bad, head, column, value):
    """O of `bad` is `value` where `head` meets `column`, and c's elsewhere."""
    Hq, Hkv, d = c["heads"]
    G = Hq // Hkv
    out, lse = run(bad)
    out = out.cpu().double()
    got = out[:, head * G:(head + 1) * G, column].clone()
    assert torch.isnan(got).all() if value != value else (got == value).all()
    out[:, head * G:(head + 1) * G, column] = ref.exact(c)[0][:, head * G:(head + 1) * G, column]
    ref.check(c, out, lse)


# One row and 16 (the prefix in the line), 17 to 64 (heads of 64: the rows twice
# in the tile), more, and two tiles of them.
@gpu
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 20, 64, 65, 130])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_of_the_prefix(rows, d):
    """A value of +-inf in the prefix, in the first and second half of a block,
    in the last partial one and behind many splits, reaches the rows of its head
    and column alone, as +-inf; both signs, or a NaN, as NaN."""
    for P, keys in ((300, (5, 70, 130, 290)), (1, (0,)), (1500, (1, 1470))):
        c = ref.make([1] * rows, [1 + 3 * (i % 5) for i in range(rows)], P, 2, 2, d, 16,
                     seed=rows + P)
        for i, key in enumerate(keys):
            value = (INF, -INF, NAN)[i % 3]
            head, column = i % 2, (7 * key + i) % d
            bad = put(c, key, head, column, value)
            check_column(c, bad, head, column, value)
            if P == 300:
                other = (key + 64) % 256
                check_column(c, put(bad, other, head, column, value), head, column, value)
                check_column(c, put(bad, other, head, column, -value), head, column, NAN)
    assert fa.fa_get_device_error() == fa.FA_OK
