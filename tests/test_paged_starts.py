"""Sequence starts at the ends of their type: reported, and nothing is read or
written outside the call's buffers."""
import pytest
import torch

import exact_attention_109_b200 as fa
import paged_ref
import test_paged
import test_paged_append as appending

gpu = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1

STARTS = [
    [LOW, 2, 4, 6],
    [LOW + 5, 2, 4, 6],
    [LOW, LOW, LOW, 6],
    [LOW, LOW + 1, LOW + 2, HIGH],
    [-1, 2, 4, 6],
    [0, LOW, 4, 6],
    [0, HIGH, 4, 6],
    [0, 2, 4, HIGH],
]


@gpu
@pytest.mark.parametrize("length", [0, 30, HIGH, LOW])
@pytest.mark.parametrize("start", STARTS)
def test_append(start, length):
    """The last sequence comes out as before where its start is right and the
    search for it meets no larger one; pages of no sequence are left alone."""
    c = appending.make([2, 2, 2], [20, 30, 40], 4, 2, 64, 16, seed=3, rope_dim=64)
    good = appending.run(c)
    bad = dict(c, start=torch.tensor(start, dtype=torch.int32), len=c["len"].clone())
    bad["len"][0] = length
    bad["rope"] = c["rope"].repeat(30, 1, 1)
    out, kp, vp = appending.run(bad)
    assert fa.fa_get_device_error() == fa.FA_ERR_INDEX
    assert fa.fa_get_device_error() == fa.FA_OK
    if start[2:] == [4, 6] and start[1] != HIGH:
        assert torch.equal(out[4:], good[0][4:])
        page = int(c["table"][2, 40 // 16])
        assert torch.equal(kp[page], good[1][page]) and torch.equal(vp[page], good[2][page])
    used = {int(p) for p in c["table"].flatten() if p >= 0}
    rest = [p for p in range(c["k"].shape[0]) if p not in used]
    assert torch.equal(kp[rest].cpu(), c["k"][rest]) and torch.equal(vp[rest].cpu(), c["v"][rest])


@gpu
@pytest.mark.parametrize("P", [0, 50])
@pytest.mark.parametrize("start", STARTS)
def test_attention(start, P):
    c = paged_ref.make([2, 2, 2], [20, 30, 40], P, 4, 2, 64, 16, seed=8, fill=0.0)
    good = test_paged.run(c)
    out, lse = test_paged.run(dict(c, start=torch.tensor(start, dtype=torch.int32)), max_new=6)
    assert fa.fa_get_device_error() == fa.FA_ERR_INDEX
    assert fa.fa_get_device_error() == fa.FA_OK
    if start == [-1, 2, 4, 6]:  # the others' rows, but for the sums' order
        assert torch.allclose(out[2:].float(), good[0][2:].float(), atol=2 ** -6)
        assert torch.allclose(lse[2:], good[1][2:], atol=1e-5)
