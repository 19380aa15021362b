"""Arguments of the compiled binding's calls whose data pointer is null because
they are empty, which must not be taken for arguments left out."""
import pytest
import torch

import exact_attention_109_b200 as fa
from test_binding import append, host

gpu = pytest.mark.gpu


@gpu
def test_an_empty_table_is_refused():
    """A table of no positions is not a call without rotation."""
    c = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in host().items()}
    q, k, v = (t[None] for t in c["x"].split([4, 2, 2], 1))
    ones = torch.ones(64, device="cuda")
    none = torch.ones(0, 32, 2, device="cuda")
    grads = [torch.ones(1, h, 3, 64, device="cuda").bfloat16() for h in (4, 2, 2)]
    for call in (lambda: fa.qk_norm_rope(q, k, v, ones, ones, rope=none),
                 lambda: fa.qk_norm_rope_backward(*grads, q, k, ones, ones, rope=none),
                 lambda: append(c, rope=none),
                 lambda: append(c, rope=none, q_weight=ones, k_weight=ones)):
        with pytest.raises(ValueError, match="rope: "):
            call()
    with pytest.raises(ValueError, match="rope: "):
        fa.qk_norm_rope(q, k, v, ones, ones, rope=torch.ones(9, 0, 2, device="cuda"))
    assert fa.fa_get_device_error() == fa.FA_OK
