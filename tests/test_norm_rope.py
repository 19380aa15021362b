"""Norm and rotation in front of attention (fa_qk_norm_rope), and its
gradients, against 64-bit definitions; refusals on the CPU; one run through
attention and back."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import exact_attention_109_b200 as fa
from exact_attention_109_b200.inputs import default_scale, to_f64
import norm_rope_ref as ref

gpu = pytest.mark.gpu
EPS = ref.EPS
FAKE = 1 << 20  # aligned, never dereferenced: every case fails validation first


# ---------------------------------------------------------------- no GPU

def test_gradient_formula_matches_differences():
    """The 64-bit gradients used below against central differences of the
    64-bit forward definition."""
    gen = torch.Generator().manual_seed(1)
    for interleaved, rope_dim in ((False, 16), (True, 16), (False, 0)):
        x = torch.randn(2, 1, 16, generator=gen, dtype=torch.float64)
        w = torch.randn(16, generator=gen, dtype=torch.float64)
        dy = torch.randn(2, 1, 16, generator=gen, dtype=torch.float64)
        tab = ref.table(5, rope_dim)[[3, 4]] if rope_dim else None
        dx, _, dw, _ = ref.backward(dy, x, w, EPS, tab, interleaved)

        def value(x, w):
            return (ref.forward(x, w, EPS, tab, interleaved)[0] * dy).sum().item()

        h = 1e-6
        for grad, arg in ((dx, x), (dw, w)):
            for i in range(arg.numel()):
                up, down = arg.clone(), arg.clone()
                up.view(-1)[i] += h
                down.view(-1)[i] -= h
                a = (value(up, w) - value(down, w) if arg is x else
                     value(x, up) - value(x, down)) / (2 * h)
                assert abs(a - grad.reshape(-1)[i].item()) < 1e-7


FWD = dict(q=FAKE, k=FAKE, v=FAKE, strides=[4096, 512, 128] * 3, q_weight=FAKE, k_weight=FAKE,
           weight_f32=0, eps=1e-6, rope=FAKE, rope_rows=64, rope_dim=128, interleaved=0,
           positions=0, q_out=FAKE, k_out=FAKE, v_out=FAKE, B=2, N=8, Hq=4, Hkv=4, d=128)


@pytest.mark.parametrize("kwargs,status", [
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(k_out=0), fa.FA_ERR_INVALID_ARG),
    (dict(v=0), fa.FA_ERR_INVALID_ARG),
    (dict(q_weight=0), fa.FA_ERR_INVALID_ARG),
    (dict(q_weight=0, k_weight=0, rope=0), fa.FA_ERR_INVALID_ARG),
    (dict(eps=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(weight_f32=2), fa.FA_ERR_INVALID_ARG),
    (dict(interleaved=2), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=24), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=144), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=0), fa.FA_ERR_INVALID_ARG),
    (dict(rope_rows=7), fa.FA_ERR_INVALID_ARG),
    (dict(rope_rows=0), fa.FA_ERR_INVALID_ARG),
    (dict(N=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_ERR_INVALID_ARG),
    (dict(Hq=6), fa.FA_ERR_INVALID_ARG),
    (dict(Hkv=0), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(strides=[4096, 512, 127] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(strides=[4096, -512, 128] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), fa.FA_ERR_MISALIGNED),
    (dict(rope=FAKE + 8), fa.FA_ERR_MISALIGNED),
    (dict(q_weight=FAKE + 1), fa.FA_ERR_MISALIGNED),
    (dict(positions=FAKE + 2), fa.FA_ERR_MISALIGNED),
    (dict(v_out=FAKE + 4), fa.FA_ERR_MISALIGNED),
])
def test_forward_rejects_bad_arguments(kwargs, status):
    assert fa.fa_qk_norm_rope(**{**FWD, **kwargs}) == status


BWD = dict(dq_out=FAKE, dk_out=FAKE, dv_out=FAKE, q=FAKE, k=FAKE, strides=[4096, 512, 128] * 2,
           q_weight=FAKE, k_weight=FAKE, weight_f32=0, eps=1e-6, rope=FAKE, rope_rows=64,
           rope_dim=128, interleaved=0, positions=0, dq=FAKE, dk=FAKE, dv=FAKE,
           grad_strides=[4096, 512, 128] * 3, dq_weight=FAKE, dk_weight=FAKE, B=2, N=8, Hq=4,
           Hkv=4, d=128, workspace=FAKE, workspace_bytes=1 << 24)


@pytest.mark.parametrize("kwargs,status", [
    (dict(dq_out=0), fa.FA_ERR_INVALID_ARG),
    (dict(dv=0), fa.FA_ERR_INVALID_ARG),
    (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(dq_weight=0), fa.FA_ERR_INVALID_ARG),
    (dict(workspace=0), fa.FA_ERR_INVALID_ARG),
    (dict(workspace_bytes=64), fa.FA_ERR_INVALID_ARG),
    (dict(workspace=FAKE + 16), fa.FA_ERR_MISALIGNED),
    # rows of a gradient that overlap: a shared batch, token or head
    (dict(grad_strides=[0, 512, 128] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(grad_strides=[4096, 0, 128] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(grad_strides=[4096, 512, 64] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(grad_strides=[4096, 384, 128] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(grad_strides=[2048, 512, 128] * 3), fa.FA_ERR_INVALID_ARG),
    (dict(d=32), fa.FA_ERR_UNSUPPORTED),
])
def test_backward_rejects_bad_arguments(kwargs, status):
    assert fa.fa_qk_norm_rope_bwd(**{**BWD, **kwargs}) == status


@pytest.mark.parametrize("kwargs,status", [
    (dict(table=0), fa.FA_ERR_INVALID_ARG),
    (dict(rows=0), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=8), fa.FA_ERR_INVALID_ARG),
    (dict(rope_dim=256), fa.FA_ERR_INVALID_ARG),
    (dict(base=0.0), fa.FA_ERR_INVALID_ARG),
    (dict(base=float("inf")), fa.FA_ERR_INVALID_ARG),
    (dict(table=FAKE + 8), fa.FA_ERR_MISALIGNED),
])
def test_table_rejects_bad_arguments(kwargs, status):
    args = dict(table=FAKE, rows=4, rope_dim=64, base=1e4)
    assert fa.fa_rope_table(**{**args, **kwargs}) == status


def test_wrappers_want_cuda_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.qk_norm_rope(x, x, x, torch.ones(64), torch.ones(64))
    with pytest.raises(ValueError):
        fa.rope_table(4, 64, device="cpu")


# ---------------------------------------------------------------- GPU

def make(B, N, Hq, Hkv, d, seed, rope_dim=None, w="bf16", packed=False, rows=None):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, N, Hq + 2 * Hkv, d, generator=gen).bfloat16()
    out = dict(qkv=x, shape=(B, N, Hq, Hkv, d), rope=None, positions=None, wq=None, wk=None)
    if w:
        kind = torch.float32 if w == "f32" else torch.bfloat16
        out["wq"] = torch.randn(d, generator=gen).to(kind)
        out["wk"] = torch.randn(d, generator=gen).to(kind)
    if rope_dim:
        out["rope"] = ref.table(rows or N + 5, rope_dim)
        if packed:
            out["positions"] = torch.randint(0, rows or N, (B, N), generator=gen).int()
    return out


def cuda(t):
    return t.cuda() if t is not None else None


def parts(x, Hq, Hkv):
    return x.split([Hq, Hkv, Hkv], dim=2)


def rows_of_table(c):
    B, N = c["shape"][:2]
    if c["rope"] is None:
        return None
    if c["positions"] is None:
        return c["rope"][:N].expand(B, -1, -1, -1)
    return c["rope"][c["positions"].long()]


def check_forward(c, interleaved, got):
    B, N, Hq, Hkv, d = c["shape"]
    q, k, v = parts(c["qkv"], Hq, Hkv)
    tab = rows_of_table(c)
    for x, w, y in ((q, c["wq"], got[0]), (k, c["wk"], got[1])):
        want, bound = ref.forward(x, w, EPS, tab, interleaved)
        ref.check(y, want.transpose(1, 2), bound.transpose(1, 2))
    if got[2] is not None:
        assert torch.equal(got[2].cpu(), v.transpose(1, 2))
    assert fa.fa_get_device_error() == fa.FA_OK


CASES = [
    # B, N, Hq, Hkv, d, rope_dim, weights, packed positions
    (1, 1, 1, 1, 128, 128, "bf16", False),
    (1, 1, 1, 1, 64, 64, "f32", True),
    (2, 37, 4, 2, 128, 128, "bf16", False),
    (2, 37, 4, 2, 64, 64, "f32", True),
    (3, 50, 8, 1, 64, 16, "bf16", True),
    (3, 50, 8, 1, 128, 48, "f32", False),
    (1, 129, 3, 3, 128, 96, None, True),
    (1, 129, 3, 3, 64, 48, None, False),
    (2, 17, 5, 5, 128, None, "bf16", False),
    (1, 700, 16, 4, 64, 32, "bf16", True),
    (2, 260, 40, 8, 128, 64, "f32", False),
]


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_forward(case, interleaved):
    B, N, Hq, Hkv, d, rope_dim, w, packed = case
    c = make(B, N, Hq, Hkv, d, seed=N + d, rope_dim=rope_dim, w=w, packed=packed)
    q, k, v = parts(c["qkv"].cuda(), Hq, Hkv)
    got = fa.qk_norm_rope(q, k, v, cuda(c["wq"]), cuda(c["wk"]), eps=EPS, rope=cuda(c["rope"]),
                          positions=cuda(c["positions"]), interleaved=interleaved)
    check_forward(c, interleaved, got)


@gpu
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_backward(case, interleaved):
    B, N, Hq, Hkv, d, rope_dim, w, packed = case
    c = make(B, N, Hq, Hkv, d, seed=N + d + 1, rope_dim=rope_dim, w=w, packed=packed)
    gen = torch.Generator().manual_seed(7)
    dy = [torch.randn(B, H, N, d, generator=gen).bfloat16() for H in (Hq, Hkv, Hkv)]
    grad = torch.full((B, N, Hq + 2 * Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k, _ = parts(c["qkv"].cuda(), Hq, Hkv)
    dq, dk, dv = parts(grad, Hq, Hkv)
    need = fa.fa_qk_norm_rope_bwd_workspace_size(d)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    got = fa.qk_norm_rope_backward(
        *[t.cuda() for t in dy], q if w else None, k if w else None, cuda(c["wq"]), cuda(c["wk"]),
        eps=EPS, rope=cuda(c["rope"]), positions=cuda(c["positions"]), interleaved=interleaved,
        dq=dq, dk=dk, dv=dv, workspace=ws)
    assert fa.fa_get_device_error() == fa.FA_OK
    check_backward(c, dy, interleaved, grad, got[3], got[4])


def check_backward(c, dy, interleaved, grad, dwq, dwk):
    B, N, Hq, Hkv, d = c["shape"]
    q, k, _ = parts(c["qkv"], Hq, Hkv)
    dq, dk, dv = parts(grad.cpu(), Hq, Hkv)
    tab = rows_of_table(c)
    for x, g, w, dx, dw in ((q, dy[0], c["wq"], dq, dwq), (k, dy[1], c["wk"], dk, dwk)):
        want, bound, want_w, mag = ref.backward(g.transpose(1, 2), x, w, EPS, tab, interleaved)
        ref.check(dx, want, bound)
        if w is None:
            assert dw is None
            continue
        # A thread adds at most one row of every head of each token block (of
        # 16 or 32) its CTA walks (up to 296 CTAs) and of one more, then 40
        # sums over lanes, warps and CTAs.
        chain = x.shape[2] * (-(-(B * N) // (8 * 592)) + 1) + 40
        ref.check(dw, want_w, (32 + chain) * ref.U * mag)
    assert torch.equal(dv, dy[2].transpose(1, 2))


@gpu
def test_gradient_against_differences():
    """The GPU's gradients against central differences of the 64-bit forward
    definition (not of the formula)."""
    c = make(1, 2, 1, 1, 64, seed=3, rope_dim=64, w="f32")
    gen = torch.Generator().manual_seed(4)
    dy = [torch.randn(1, 1, 2, 64, generator=gen).bfloat16() for _ in range(3)]
    q, k, _ = parts(c["qkv"].cuda(), 1, 1)
    dq, _, _, dwq, _ = fa.qk_norm_rope_backward(*[t.cuda() for t in dy], q, k, cuda(c["wq"]),
                                                cuda(c["wk"]), eps=EPS, rope=cuda(c["rope"]))
    x, w, tab = c["qkv"][:, :, :1].double(), c["wq"].double(), rows_of_table(c)

    def value(x, w):
        return (ref.forward(x, w, EPS, tab, False)[0] * dy[0].double().transpose(1, 2)).sum()

    h = 1e-5
    for got, arg, f in ((dq, x, lambda t: value(t, w)), (dwq, w, lambda t: value(x, t))):
        want = torch.empty(arg.numel(), dtype=torch.float64)
        for i in range(arg.numel()):
            up, down = arg.clone(), arg.clone()
            up.view(-1)[i] += h
            down.view(-1)[i] -= h
            want[i] = (f(up) - f(down)) / (2 * h)
        err = (got.cpu().double().reshape(-1) - want).abs()
        # bf16 rounding of the gradient, and h^2 and 1e-16 / h of the differences
        assert (err <= ref.HALF_BF16 * want.abs() + 1e-5).all()


@gpu
@pytest.mark.parametrize("layout", ["head_major", "broadcast", "padded"])
def test_input_strides(layout):
    B, N, Hq, Hkv, d = 3, 21, 4, 2, 128
    c = make(B, N, Hq, Hkv, d, seed=5, rope_dim=128)
    x = c["qkv"].cuda()
    if layout == "head_major":
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "broadcast":  # one row of the batch for all
        c["qkv"] = c["qkv"][:1].expand(B, -1, -1, -1)
        x = x[:1].expand(B, -1, -1, -1)
    else:
        room = torch.full((B, N + 3, Hq + 2 * Hkv + 1, d + 8), float("nan"),
                          dtype=torch.bfloat16, device="cuda")
        room[:, 1:N + 1, :-1, 8:] = x
        x = room[:, 1:N + 1, :-1, 8:]
    q, k, v = parts(x, Hq, Hkv)
    got = fa.qk_norm_rope(q, k, v, cuda(c["wq"]), cuda(c["wk"]), eps=EPS, rope=cuda(c["rope"]))
    check_forward(c, False, got)
    gen = torch.Generator().manual_seed(8)
    dy = [torch.randn(B, H, N, d, generator=gen).bfloat16() for H in (Hq, Hkv, Hkv)]
    grads = fa.qk_norm_rope_backward(*[t.cuda() for t in dy], q, k, cuda(c["wq"]), cuda(c["wk"]),
                                     eps=EPS, rope=cuda(c["rope"]))
    check_backward(c, dy, False, torch.cat([t.cpu() for t in grads[:3]], 2), *grads[3:])


@gpu
def test_without_values():
    c = make(2, 30, 4, 4, 64, seed=6, rope_dim=64)
    q, k, _ = parts(c["qkv"].cuda(), 4, 4)
    got = fa.qk_norm_rope(q, k, None, cuda(c["wq"]), cuda(c["wk"]), eps=EPS, rope=cuda(c["rope"]))
    assert got[2] is None
    check_forward(c, False, got)


@gpu
def test_rows_do_not_mix():
    """Zero, infinite and NaN rows change no other row; a zero row stays zero."""
    B, N, H, d = 1, 40, 2, 128
    c = make(B, N, H, H, d, seed=9, rope_dim=128)
    clean = c["qkv"].cuda()
    dirty = clean.clone()
    dirty[0, 3, 0] = 0
    dirty[0, 4, 0] = float("inf")
    dirty[0, 5, 1, 7] = float("nan")
    args = dict(eps=EPS, rope=cuda(c["rope"]))
    w = cuda(c["wq"]), cuda(c["wk"])
    a = fa.qk_norm_rope(*parts(clean, H, H), *w, **args)[0]
    b = fa.qk_norm_rope(*parts(dirty, H, H), *w, **args)[0]
    assert (b[0, 0, 3] == 0).all()
    assert b[0, 1, 5].isnan().all()
    same = torch.ones(H, N, dtype=torch.bool)
    same[0, 3] = same[0, 4] = same[1, 5] = False
    assert torch.equal(a[0][same.cuda()], b[0][same.cuda()])


@gpu
def test_unturned_values_keep_infinities():
    """Values beyond rope_dim are moved as they are, infinities included."""
    x = torch.randn(1, 4, 1, 64, device="cuda").bfloat16()
    x[0, 2, 0, 40] = float("inf")
    y, _, _ = fa.qk_norm_rope(x, x, rope=ref.table(4, 32).cuda())
    assert torch.equal(y[0, 0, :, 32:], x[0, :, 0, 32:])


@gpu
def test_table_and_far_positions():
    rows = 1 << 20
    t = fa.rope_table(rows, 64, base=5e5)
    at = torch.tensor([0, 1, 77777, rows - 1])
    inv = 5e5 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = at.double()[:, None] * inv
    want = torch.stack((ang.cos(), ang.sin()), -1)
    # one fp32 rounding, and the 64-bit angle's own 2^-52 * 2^20
    assert (t[at].cpu().double() - want).abs().max() <= 2.0 ** -25 + 1e-9
    x = torch.randn(1, 4, 2, 64, device="cuda").bfloat16()
    y, _, _ = fa.qk_norm_rope(x, x, rope=t, positions=at.int().cuda()[None])
    want, bound = ref.forward(x.cpu(), None, EPS, t[at].cpu()[None], False)
    ref.check(y, want.transpose(1, 2), bound.transpose(1, 2))


@gpu
@pytest.mark.parametrize("bad", [-1, 64, 1 << 30])
def test_position_outside_the_table_is_reported(bad):
    x = torch.randn(1, 8, 2, 64, device="cuda").bfloat16()
    pos = torch.arange(8, device="cuda").int()[None].contiguous()
    table = ref.table(64, 64).cuda()
    good = fa.qk_norm_rope(x, x, rope=table, positions=pos)[0]
    pos[0, 5] = bad
    y = fa.qk_norm_rope(x, x, rope=table, positions=pos)[0]
    assert fa.fa_get_device_error() == fa.FA_ERR_INDEX
    assert fa.fa_get_device_error() == fa.FA_OK
    keep = [0, 1, 2, 3, 4, 6, 7]
    assert torch.equal(good[:, :, keep], y[:, :, keep])


@gpu
def test_runs_are_equal_bit_for_bit():
    c = make(4, 1500, 8, 2, 128, seed=11, rope_dim=128)
    gen = torch.Generator().manual_seed(12)
    dy = [torch.randn(4, H, 1500, 128, generator=gen).bfloat16().cuda() for H in (8, 2, 2)]
    q, k, _ = parts(c["qkv"].cuda(), 8, 2)
    args = (*dy, q, k, cuda(c["wq"]), cuda(c["wk"]))
    a = fa.qk_norm_rope_backward(*args, rope=cuda(c["rope"]))
    for _ in range(3):
        b = fa.qk_norm_rope_backward(*args, rope=cuda(c["rope"]))
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_other_stream_and_graph():
    c = make(2, 300, 4, 2, 128, seed=13, rope_dim=128)
    x = c["qkv"].cuda()
    q, k, v = parts(x, 4, 2)
    w, rope = (cuda(c["wq"]), cuda(c["wk"])), cuda(c["rope"])
    gen = torch.Generator().manual_seed(14)
    dy = [torch.randn(2, H, 300, 128, generator=gen).bfloat16().cuda() for H in (4, 2, 2)]
    want = fa.qk_norm_rope(q, k, v, *w, rope=rope)
    want_g = fa.qk_norm_rope_backward(*dy, q, k, *w, rope=rope)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fa.qk_norm_rope(q, k, v, *w, rope=rope, stream=side)
    got_g = fa.qk_norm_rope_backward(*dy, q, k, *w, rope=rope, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + want_g, got + got_g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.qk_norm_rope(q, k, v, *w, rope=rope)
        got_g = fa.qk_norm_rope_backward(*dy, q, k, *w, rope=rope)
    x.mul_(0.5)
    want = fa.qk_norm_rope(q, k, v, *w, rope=rope)
    want_g = fa.qk_norm_rope_backward(*dy, q, k, *w, rope=rope)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want + want_g, got + got_g))


@gpu
def test_beyond_32_bit_offsets():
    """Rows that lie more than 2^31 elements into a tensor."""
    N, H, d = 70000, 256, 128  # 2.3e9 elements
    x = torch.empty(1, N, H, d, dtype=torch.bfloat16, device="cuda")
    x[:, :8].normal_()
    x[:, -8:] = x[:, :8]
    x[:, 8:-8] = 0
    k = x[:, :, :1]
    y, _, _ = fa.qk_norm_rope(x, k, None, torch.ones(d, device="cuda"),
                              torch.ones(d, device="cuda"), eps=EPS)
    want, bound = ref.forward(x[:, :8].cpu(), torch.ones(d), EPS, None, False)
    ref.check(y[:, :, -8:], want.transpose(1, 2), bound.transpose(1, 2))
    ref.check(y[:, :, :8], want.transpose(1, 2), bound.transpose(1, 2))


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_through_attention_and_back(d):
    """Projection -> norm and rotation -> attention -> gradients, as a training
    step runs them, against the 64-bit chain on the kernels' own bf16 hand-overs."""
    B, N, H = 1, 200, 2
    c = make(B, N, H, H, d, seed=15, rope_dim=d)
    scale = default_scale(d)
    qkv = c["qkv"].cuda()
    qp, kp, vp = parts(qkv, H, H)
    w, rope = (cuda(c["wq"]), cuda(c["wk"])), cuda(c["rope"])
    q, k, v = fa.qk_norm_rope(qp, kp, vp, *w, eps=EPS, rope=rope)
    o, lse = fa.attention_forward(q, k, v, True, scale)
    gen = torch.Generator().manual_seed(16)
    dO = torch.randn(B, H, N, d, generator=gen).bfloat16()
    dqkv = fa.attention_backward(q, k, v, o, lse, dO.cuda(), True, scale)
    grad = torch.empty_like(qkv)
    got = fa.qk_norm_rope_backward(*dqkv, qp, kp, *w, eps=EPS, rope=rope,
                                   **dict(zip(("dq", "dk", "dv"), parts(grad, H, H))))
    assert fa.fa_get_device_error() == fa.FA_OK
    check_forward(c, False, (q, k, v))
    o_ref, _ = oracle.ref_fwd(to_f64(q.cpu()), to_f64(k.cpu()), to_f64(v.cpu()), True, scale)
    assert np.abs(to_f64(o.cpu()) - o_ref).max() <= 1e-2
    check_backward(c, [t.cpu() for t in dqkv], False, grad, got[3], got[4])


@gpu
def test_order_behind_other_work():
    """Forward and backward start while the stream's previous work (copies,
    memsets, kernels) ends and see what it wrote, eagerly and captured."""
    B, N, Hq, Hkv, d = 2, 700, 8, 2, 128
    c = make(B, N, Hq, Hkv, d, seed=21, rope_dim=128, w="f32")
    real, rope = c["qkv"].cuda(), cuda(c["rope"])
    w = cuda(c["wq"]), cuda(c["wk"])
    x = real.clone()
    room = torch.empty(32 << 20, device="cuda")

    def step():
        room.zero_()
        x.copy_(real)
        out = fa.qk_norm_rope(*parts(x, Hq, Hkv), *w, eps=EPS, rope=rope)
        q, k, _ = parts(x, Hq, Hkv)
        grads = fa.qk_norm_rope_backward(*out, q, k, *w, eps=EPS, rope=rope)
        room.add_(1)
        return [t.clone() for t in (*out, *grads)]

    want = step()
    torch.cuda.synchronize()
    for _ in range(5):
        x.fill_(float("nan"))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
