"""The training operators under autograd: what a user of `train` may do with them."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train

pytestmark = pytest.mark.gpu


def test_layer_norm_without_a_bias():
    x = torch.randn(40, 256, device="cuda").requires_grad_()
    w = torch.randn(256, device="cuda").requires_grad_()
    dy = torch.randn(40, 256, device="cuda")
    train.layer_norm(x, w, None).backward(dy)
    _, mean, rstd = moe.moe_layer_norm(x.detach(), w.detach())
    dx, dw, _ = moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    again = moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd, has_bias=False)
    assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[1], dw)
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd, d_bias=torch.empty_like(dw), has_bias=False)
