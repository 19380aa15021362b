"""Appending packed new tokens to a paged cache (fa_paged_append): the rows
written, against the 64-bit definition, and every other row left as it was;
refusals on the CPU."""
import pytest
import torch

import exact_attention_109_b200 as fa
import norm_rope_ref as ref

gpu = pytest.mark.gpu
EPS = ref.EPS
FAKE = 1 << 20  # aligned, never dereferenced: every case fails validation first

ARGS = dict(q=FAKE, k=FAKE, v=FAKE, strides=[512, 128] * 3, q_weight=FAKE, k_weight=FAKE,
            weight_f32=0, eps=1e-6, rope=FAKE, rope_rows=64, rope_dim=128, interleaved=0,
            pos_offset=0, seq_start=FAKE, cache_len=FAKE, block_table=FAKE, q_out=FAKE,
            k_pages=FAKE, v_pages=FAKE, S=2, T=5, Hq=4, Hkv=2, d=128, page_size=16, num_pages=9,
            max_pages=3)


@pytest.mark.parametrize("kwargs,status", [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(v=0), fa.FA_ERR_INVALID_ARG),
    (dict(seq_start=0), fa.FA_ERR_INVALID_ARG),
    (dict(block_table=0), fa.FA_ERR_INVALID_ARG),
    (dict(k_weight=0), fa.FA_ERR_INVALID_ARG),
    (dict(eps=-1.0), fa.FA_ERR_INVALID_ARG),
    (dict(S=0), fa.FA_ERR_INVALID_ARG),
    (dict(T=-1), fa.FA_ERR_INVALID_ARG),
    (dict(pos_offset=-1), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=8), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=48), fa.FA_ERR_INVALID_ARG),
    (dict(page_size=512), fa.FA_ERR_INVALID_ARG),
    (dict(num_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(max_pages=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=5), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=130), fa.FA_ERR_INVALID_ARG),
    (dict(strides=[512, 100] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(d=80), fa.FA_ERR_UNSUPPORTED),
    (dict(k_pages=FAKE + 8), fa.FA_ERR_MISALIGNED),
    (dict(cache_len=FAKE + 2), fa.FA_ERR_MISALIGNED),
])
def test_rejects_bad_arguments(kwargs, status):
    assert fa.fa_paged_append(**{**ARGS, **kwargs}) == status


def test_no_new_tokens_is_no_work():
    assert fa.fa_paged_append(**{**ARGS, "T": 0}) == fa.FA_OK


# ---------------------------------------------------------------- GPU

def make(new, have, Hq, Hkv, d, page, seed, rope_dim=None, w=None, pad=0, offset=0):
    gen = torch.Generator().manual_seed(seed)
    S, T = len(new), sum(new) + pad
    need = [-(-(a + b) // page) for a, b in zip(new, have)]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((S, max(1, max(need)) + 2), -7, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    c = dict(new=new, have=have, page=page, offset=offset, table=table,
             qkv=torch.randn(T, Hq + 2 * Hkv, d, generator=gen).bfloat16(),
             start=torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32),
             len=torch.tensor(have, dtype=torch.int32), heads=(Hq, Hkv, d),
             k=torch.randn(pages, Hkv, page, d, generator=gen).bfloat16(),
             v=torch.randn(pages, Hkv, page, d, generator=gen).bfloat16(),
             wq=None, wk=None, rope=None)
    if w:
        kind = torch.float32 if w == "f32" else torch.bfloat16
        c["wq"], c["wk"] = (torch.randn(d, generator=gen).to(kind) for _ in range(2))
    if rope_dim:
        c["rope"] = ref.table(max(a + b for a, b in zip(new, have)) + offset, rope_dim)
    return c


def run(c, interleaved=False, **kw):
    g = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    Hq, Hkv, d = c["heads"]
    q, k, v = g["qkv"].split([Hq, Hkv, Hkv], dim=1)
    out = torch.full((q.shape[0], Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    kp, vp = g["k"].clone(), g["v"].clone()
    fa.paged_append(q, k, v, kp, vp, g["table"], g["start"], g["len"], rope=g["rope"],
                    pos_offset=c["offset"], q_weight=g["wq"], k_weight=g["wk"], eps=EPS,
                    interleaved=interleaved, q_out=out, **kw)
    return out, kp, vp


def check(c, interleaved, out, kp, vp):
    Hq, Hkv, d = c["heads"]
    q, k, v = c["qkv"].split([Hq, Hkv, Hkv], dim=1)
    out, kp, vp = out.cpu(), kp.cpu(), vp.cpu()
    want_v, rest_k = c["v"].clone(), c["k"].clone()
    for s, (n, have) in enumerate(zip(c["new"], c["have"])):
        for i in range(n):
            t, j = int(c["start"][s]) + i, have + i
            tab = c["rope"][j + c["offset"]] if c["rope"] is not None else None
            want, bound = ref.forward(q[t], c["wq"], EPS, tab, interleaved)
            ref.check(out[t], want, bound)
            page, row = int(c["table"][s, j // c["page"]]), j % c["page"]
            want, bound = ref.forward(k[t], c["wk"], EPS, tab, interleaved)
            ref.check(kp[page, :, row], want, bound)
            rest_k[page, :, row] = kp[page, :, row]
            want_v[page, :, row] = v[t]
    assert torch.equal(vp, want_v) and torch.equal(kp, rest_k)
    assert (out[sum(c["new"]):] == 3).all()
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("new,have,Hq,Hkv,d,page,rope_dim,w", [
    ([1], [0], 1, 1, 64, 16, 64, None),
    ([1], [1000], 16, 16, 128, 16, 128, None),
    ([1] * 9, [0, 15, 16, 17, 31, 32, 100, 5, 64], 8, 2, 128, 32, 128, "bf16"),
    ([3, 0, 1, 40, 0, 0, 2], [14, 9, 0, 60, 3, 0, 127], 4, 4, 64, 64, 32, "f32"),
    ([0, 0, 5], [7, 7, 7], 6, 2, 128, 16, 48, "bf16"),
    ([200, 130], [0, 33], 8, 1, 64, 256, 64, "bf16"),
    ([5, 6], [1, 2], 2, 2, 128, 128, None, None),
])
def test_append(new, have, Hq, Hkv, d, page, rope_dim, w, interleaved):
    c = make(new, have, Hq, Hkv, d, page, seed=sum(have) + d, rope_dim=rope_dim, w=w, pad=3,
             offset=11)
    check(c, interleaved, *run(c, interleaved))


@gpu
def test_head_major_and_repeated_inputs():
    c = make([2, 3], [4, 30], 4, 2, 128, 16, seed=2, rope_dim=128, w="bf16")
    x = c["qkv"].cuda().transpose(0, 1).contiguous().transpose(0, 1)
    c2 = dict(c, qkv=x)
    check(c, False, *run(c2))
    c["qkv"] = c["qkv"][:1].expand(5, -1, -1)
    check(c, False, *run(c))


@gpu
@pytest.mark.parametrize("fault", ["page_high", "page_negative", "table_short", "length_negative",
                                   "length_huge", "position", "start_decreases", "start_late"])
def test_bad_index_is_reported_and_touches_nothing(fault):
    """A page, a length or a position out of range: the error is reported, the
    sequence's keys are not written, and everybody else's are."""
    c = make([2, 2, 2], [20, 30, 40], 4, 2, 64, 16, seed=3, rope_dim=64)
    good = run(c)
    bad = dict(c, table=c["table"].clone(), len=c["len"].clone())
    if fault == "page_high":
        bad["table"][1, 1] = bad["table"][1, 2] = c["k"].shape[0]
    elif fault == "page_negative":
        bad["table"][1, 1] = bad["table"][1, 2] = -1
    elif fault == "table_short":
        bad["len"][1] = c["table"].shape[1] * 16
        bad["rope"] = ref.table(200, 64)
    elif fault == "length_negative":
        bad["len"][1] = -3
    elif fault == "length_huge":
        bad["len"][1] = 2 ** 31 - 1
    elif fault == "position":
        bad["rope"] = c["rope"][:41]  # the third sequence's last position is 41
    elif fault == "start_decreases":
        bad["start"] = torch.tensor([0, 4, 2, 6], dtype=torch.int32)
    else:
        bad["start"] = torch.tensor([0, 2, 4, 7], dtype=torch.int32)
    out, kp, vp = run(bad)
    assert fa.fa_get_device_error() == fa.FA_ERR_INDEX
    if fault.startswith("start"):
        return
    if fault == "position":
        assert torch.equal(out[:5], good[0][:5]) and torch.equal(vp, good[2])
        return
    assert torch.equal(out[:2], good[0][:2]) and torch.equal(out[4:], good[0][4:])
    want_k, want_v = good[1].clone(), good[2].clone()
    for j in (30, 31):
        page = int(c["table"][1, j // 16])
        want_k[page, :, j % 16] = c["k"][page, :, j % 16].cuda()
        want_v[page, :, j % 16] = c["v"][page, :, j % 16].cuda()
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)


@gpu
def test_captured_graph_follows_lengths():
    """One captured decode step, replayed as the lengths grow."""
    c = make([1, 1, 1], [14, 0, 31], 4, 4, 128, 16, seed=4, rope_dim=128)
    g = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    table = torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3)
    rope = ref.table(48, 128)
    kp = torch.zeros(9, 4, 16, 128, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    q, k, v = g["qkv"].split([4, 4, 4], dim=1)
    rope_c, length = rope.cuda(), g["len"].clone()

    def step():
        fa.paged_append(q, k, v, kp, vp, table, g["start"], length, rope=rope_c)
        length.add_(1)

    step()
    length.copy_(g["len"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kp.zero_(), vp.zero_(), length.copy_(g["len"])
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert length.tolist() == [19, 5, 36]
    _, kc, vc = c["qkv"].split([4, 4, 4], dim=1)
    for s, have in enumerate(c["have"]):
        for j in range(48):
            page, row = 3 * s + j // 16, j % 16
            if have <= j < have + 5:
                want, bound = ref.forward(kc[s], None, EPS, rope[j], False)
                ref.check(kp[page, :, row], want, bound)
                assert torch.equal(vp[page, :, row].cpu(), vc[s])
            else:
                assert (kp[page, :, row] == 0).all() and (vp[page, :, row] == 0).all()
    assert fa.fa_get_device_error() == fa.FA_OK


@gpu
def test_other_stream():
    c = make([2, 1], [3, 4], 4, 2, 64, 16, seed=5, rope_dim=64, w="bf16")
    want = run(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(c, stream=None)
    with torch.cuda.stream(side):
        again = run(c, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, x) for a, b, x in zip(want, got, again))
