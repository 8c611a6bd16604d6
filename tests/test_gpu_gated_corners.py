"""The gated experts and the weighted sum without rows, without tokens, in a thread of their own and under recomputation."""
import threading

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train

pytestmark = pytest.mark.gpu
KEEPS = [moe.MOE_KEEP_16BIT, moe.MOE_KEEP_E4M3]


@pytest.mark.parametrize("keep", KEEPS)
@pytest.mark.parametrize("gaps", [False, True])
def test_no_rows(keep, gaps):
    """No row at all: results without rows, weights' gradients of 0."""
    E, N, K = 3, 32, 64
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.zeros(0, K, device="cuda").bfloat16().requires_grad_()
    w13 = torch.randn(E, 2 * N, K, device="cuda", generator=g).bfloat16().requires_grad_()
    w2 = torch.randn(E, K, N, device="cuda", generator=g).bfloat16().requires_grad_()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y = train.gated_experts(x, w13, w2, off, keep=keep, gaps=gaps)
    assert y.shape == (0, K)
    dx, dw13, dw2 = torch.autograd.grad(y, [x, w13, w2], torch.zeros_like(y))
    assert dx.shape == (0, K) and not dw13.any() and not dw2.any() and dw13.shape == w13.shape and dw2.shape == w2.shape


@pytest.mark.parametrize("keep", KEEPS)
@pytest.mark.parametrize("rows", [0, 5])
def test_no_tokens(keep, rows):
    y = torch.ones(rows, 128, device="cuda").bfloat16().requires_grad_()
    w = torch.zeros(0, 2, device="cuda").requires_grad_()
    out = train.weighted_sum(y, torch.zeros(0, 2, dtype=torch.int32, device="cuda"), w, keep=keep)
    assert out.shape == (0, 128)
    dy, dw = torch.autograd.grad(out, [y, w], torch.zeros_like(out))
    assert dy.shape == y.shape and not dy.any() and dw.shape == (0, 2)


@pytest.mark.parametrize("keep", KEEPS)
def test_no_slot_has_a_row(keep):
    y = torch.full((6, 128), float("nan"), device="cuda").bfloat16().requires_grad_()
    w = torch.ones(4, 2, device="cuda").requires_grad_()
    out = train.weighted_sum(y, torch.full((4, 2), -1, dtype=torch.int32, device="cuda"), w, keep=keep)
    dy, dw = torch.autograd.grad(out, [y, w], torch.ones_like(out))
    assert not out.any() and not dy.any() and not dw.any()


def block_step(p, x, dout, keep, wrapped=False):
    def run(x):
        return train.moe_block(p, x, 2, keep=keep)
    out = checkpoint(run, x, use_reentrant=False) if wrapped else run(x)
    return [out.detach(), *torch.autograd.grad(out, [x, *p.values()], dout)]


@pytest.mark.parametrize("keep", KEEPS)
def test_recomputed_and_in_a_thread(keep):
    """The block computed again for its backward pass, and forward and backward in a new thread, give the same bits."""
    p = train.init_block(128, 128, 8, seed=2)
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(75, 128, device="cuda", generator=g).bfloat16().requires_grad_()
    dout = torch.randn(75, 128, device="cuda", generator=g).bfloat16()
    want = block_step(p, x, dout, keep)
    assert all(torch.equal(a, b) for a, b in zip(block_step(p, x, dout, keep, wrapped=True), want))
    got, failed = [], []
    torch.cuda.synchronize()

    def run():
        try:
            got.extend(block_step(p, x, dout, keep))
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)
    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert not failed, failed
    assert all(torch.equal(a, b) for a, b in zip(got, want))
