"""What moe_gather_weight_reduce_backward does not read may be left out in the binding as in the C interface."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe


def test_refusals():
    """Without a GPU: refused before any tensor's place is looked at."""
    d, s, w = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    y = torch.zeros(8, 128, dtype=torch.bfloat16)
    g = moe.moe_gather_weight_reduce_backward
    for call in (lambda: g(d, None, s, w), lambda: g(d, None, s, w, want_weights=False), lambda: g(d, None, s, w, d_y=y)):
        with pytest.raises(ValueError, match="y: needed"):
            call()


@pytest.mark.gpu
def test_what_is_not_read_is_not_asked_for():
    gen = torch.Generator(device="cuda").manual_seed(1)
    M, topk, K = 30, 3, 256
    dout = torch.randn(M, K, device="cuda", generator=gen).bfloat16()
    y = torch.randn(M * topk, K, device="cuda", generator=gen).bfloat16()
    s = torch.randperm(M * topk, device="cuda", generator=gen).int().view(M, topk)
    s[::4, 1] = -1
    w = torch.rand(M, topk, device="cuda", generator=gen)
    g = moe.moe_gather_weight_reduce_backward
    want, none = g(dout, y, s, w, d_y=torch.zeros_like(y), want_weights=False)
    got, nothing = g(dout, None, s, w, d_y=torch.zeros_like(y), want_weights=False)
    assert none is None and nothing is None and torch.equal(got, want)
    want, _ = g(dout, y, s, w, True, d_y=torch.zeros_like(y))
    for yy in (y, None):
        got, nothing = g(dout, yy, s, None, True, d_y=torch.zeros_like(y))
        assert nothing is None and torch.equal(got, want)
    with pytest.raises(ValueError, match="topk_weights"):
        g(dout, y, s, None)
