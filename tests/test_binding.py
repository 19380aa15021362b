"""The compiled binding of the calls around attention: what it refuses, what it
allocates, and where it runs.  Without a GPU: host tensors and wrong arguments."""
import pytest
import torch

import exact_attention_109_b200 as fa
import paged_ref

gpu = pytest.mark.gpu


def host():
    c = paged_ref.make([1, 2], [3, 20], 30, 4, 2, 64, 16, seed=0, fill=0.0)
    c["x"] = torch.randn(3, 8, 64).bfloat16()
    c["have"] = c["len"] - torch.tensor([1, 2], dtype=torch.int32)
    return c


def test_host_tensors_are_refused():
    c = host()
    q, k, v = c["x"].split([4, 2, 2], 1)
    with pytest.raises(ValueError, match="q: expected a CUDA tensor"):
        fa.paged_append(q, k, v, c["k"], c["v"], c["table"], c["start"], c["have"])
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(q[None], k[None], v[None], torch.ones(64), torch.ones(64))
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope_backward(q[None], k[None], None, None, None, rope=torch.ones(4, 32, 2))


def test_what_is_no_tensor_is_refused():
    c = host()
    with pytest.raises(TypeError, match="q: expected a tensor"):
        fa.attention_paged([1.0], c["k"], c["v"], c["table"], c["start"], c["len"], 0.1)
    with pytest.raises(ValueError, match="T, H, d"):
        fa.paged_append(c["x"][0], c["x"][0], c["x"][0], c["k"], c["v"], c["table"], c["start"],
                        c["have"])


# ---------------------------------------------------------------- GPU

def paged(c, **kw):
    a = dict(q=c["q"], k_pages=c["k"], v_pages=c["v"], block_table=c["table"],
             seq_start=c["start"], kv_len=c["len"], scale=c["scale"], prefix_pages=c["prefix"],
             prefix_len=c["P"], max_new=2)
    return fa.attention_paged(**{**a, **kw})


def append(c, **kw):
    q, k, v = c["x"].split([4, 2, 2], 1)
    a = dict(q=q, k=k, v=v, k_pages=c["k"], v_pages=c["v"], block_table=c["table"],
             seq_start=c["start"], cache_len=c["have"])
    return fa.paged_append(**{**a, **kw})


@gpu
def test_refusals():
    c = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in host().items()}
    before = c["k"].clone()
    ones = torch.ones(64, device="cuda")
    for error, match, call in [
        (TypeError, "q: expected BFloat16", lambda: paged(c, q=c["q"].float())),
        (TypeError, "kv_len: expected Int", lambda: paged(c, kv_len=c["len"].long())),
        (TypeError, "prefix_pages", lambda: paged(c, prefix_pages=c["prefix"].long())),
        (ValueError, "v_pages: expected shape", lambda: paged(c, v_pages=c["v"][:-1])),
        (ValueError, "seq_start: expected shape", lambda: paged(c, seq_start=c["start"][:-1])),
        (ValueError, "table: expected device", lambda: paged(c, block_table=c["table"].cpu())),
        (ValueError, "must be contiguous", lambda: paged(c, k_pages=c["k"].transpose(0, 1)
                                                         .contiguous().transpose(0, 1))),
        (ValueError, "do not hold", lambda: paged(c, prefix_len=33)),
        (ValueError, "without prefix_pages", lambda: paged(c, prefix_pages=None)),
        (ValueError, "out: expected shape", lambda: paged(c, out=torch.empty_like(c["q"][:1]))),
        (ValueError, "out of range", lambda: paged(c, prefix_len=1 << 40)),
        (TypeError, None, lambda: paged(c, scale="1")),
        (TypeError, None, lambda: paged(c, max_new=1.5)),
        (fa.FaError, "fa_fwd_paged", lambda: paged(c, scale=-1.0)),
        (fa.FaError, "fa_fwd_paged", lambda: paged(c, max_new=4)),
        (fa.FaError, "fa_fwd_paged",
         lambda: paged(c, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))),
        (ValueError, "workspace: expected device",
         lambda: paged(c, workspace=torch.empty(1 << 20, dtype=torch.uint8))),
        (ValueError, "last dimension", lambda: append(c, q=c["x"][:, :4].transpose(0, 2)
                                                      .contiguous().transpose(0, 2))),
        (ValueError, "k_pages: expected 4 heads", lambda: append(c, k=c["x"][:, :4],
                                                                v=c["x"][:, :4])),
        (ValueError, "both or neither", lambda: append(c, q_weight=ones)),
        (TypeError, "q_weight: expected BFloat16 or Float",
         lambda: append(c, q_weight=ones.half(), k_weight=ones.half())),
        (ValueError, "rope: expected a", lambda: append(c, rope=torch.ones(9, 64, device="cuda"))),
        (fa.FaError, "fa_paged_append", lambda: append(c, pos_offset=-1)),
        (fa.FaError, "fa_paged_append",
         lambda: append(c, rope=torch.ones(50, 36, 2, device="cuda"))),
    ]:
        with pytest.raises(error, match=match):
            call()
    with pytest.raises(fa.FaError) as e:
        paged(c, scale=float("nan"))
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert torch.equal(c["k"], before) and fa.fa_get_device_error() == fa.FA_OK


@gpu
def test_no_tokens():
    c = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in host().items()}
    c["start"].zero_()
    out, lse = paged(c, q=c["q"][:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    before = c["k"].clone()
    assert append(dict(c, x=c["x"][:0])).shape == (0, 4, 64)
    assert torch.equal(c["k"], before)


@gpu
def test_runs_on_the_current_stream():
    """Work of the call is ordered behind earlier work of the stream that is
    current, and outputs belong to that stream."""
    c = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in host().items()}
    want = paged(c)
    late = torch.zeros_like(c["q"])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
        late.copy_(c["q"])
        got = paged(c, q=late)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
