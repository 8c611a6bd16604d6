"""The training operators together: a pre-norm MoE block against the same block in 64 bits.

The reference is made of plain torch operations under autograd at 64 bits, with the block's
own choice of experts (the choice is discrete and has no gradient). The block rounds to bf16
(2^-9 relative rms per rounding, 2^-8 at most) after the norm, each product, the activation and the
gather: at most eight roundings lie between an input and an output or gradient, and the sums they
enter average them, so that a result's relative 2-norm error stays below 8 * 2^-8 = 2^-5."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train

pytestmark = pytest.mark.gpu


def reference(p, x, ids, topk, renormalize, scoring):
    q = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    x = x.detach().double().requires_grad_()
    mu = x.mean(1, keepdim=True)
    h = (x - mu) / ((x - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * q["norm_weight"] + q["norm_bias"]
    logits = h @ q["gate"][0].T
    s = torch.softmax(logits, 1) if scoring == moe.MOE_SCORE_SOFTMAX else torch.sigmoid(logits)
    w = s.gather(1, ids.long())
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    N = q["w2"].shape[2]
    out = x
    for k in range(topk):
        u = torch.einsum("mk,mnk->mn", h, q["w13"][ids[:, k].long()])
        a = torch.nn.functional.silu(u[:, :N]) * u[:, N:]
        out = out + w[:, k:k + 1] * torch.einsum("mn,mkn->mk", a, q["w2"][ids[:, k].long()])
    return q, x, out


@pytest.mark.parametrize("scoring,renormalize", [(moe.MOE_SCORE_SOFTMAX, True), (moe.MOE_SCORE_SIGMOID, False)])
def test_block_and_its_gradients(scoring, renormalize):
    M, K, N, E, topk = 97, 256, 128, 8, 3
    p = train.init_block(K, N, E, seed=1)
    with torch.no_grad():  # weights large enough that every path contributes
        for name in ("gate", "w13", "w2"):
            p[name].mul_(4)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16().requires_grad_()
    dout = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    out = train.moe_block(p, x, topk, scoring, renormalize)
    out.backward(dout)
    # the block's own choice of experts
    h = train.layer_norm(x.detach(), p["norm_weight"].detach(), p["norm_bias"].detach())
    logits = moe.moe_grouped_matmul(h, p["gate"].detach(), torch.tensor([0, M], dtype=torch.int32, device="cuda"),
                                    out_dtype=torch.float32)
    _, ids = moe.moe_router_topk(logits, topk, scoring, renormalize)
    q, xr, ref = reference(p, x, ids, topk, renormalize, scoring)
    ref.backward(dout.double())

    def near(a, b, what):
        rel = ((a.double() - b).norm() / b.norm()).item()
        assert rel <= 2 ** -5, (what, rel)
    near(out - x, ref - xr, "output")
    near(x.grad - dout, xr.grad - dout.double(), "input gradient")
    for name, v in p.items():
        near(v.grad, q[name].grad, name)
    assert moe.moe_device_error() == 0


def test_training_steps_lower_the_loss_and_clip():
    M, K, N, E, topk = 200, 256, 128, 16, 4
    p = train.init_block(K, N, E, seed=3)
    x = torch.randn(M, K, device="cuda").bfloat16()
    target = x + 0.3 * torch.roll(x, 1, dims=1)
    losses = []
    for _ in range(20):
        loss, norm = train.train_step(p, x, target, topk, lr=5.0, max_norm=0.05)
        losses.append(loss.item())
        total = sum(v.grad.double().square().sum() for v in p.values()).sqrt().item()
        assert total <= 0.05 * (1 + 2 ** -7) or norm.item() <= 0.05
    assert losses[-1] < 0.9 * losses[0], losses


def test_tokens_without_experts_pass_through():
    M, K, N, E = 40, 128, 128, 8
    p = train.init_block(K, N, E, seed=4)
    logits = torch.randn(M, E, device="cuda")
    logits[::3] = -float("inf")
    weights, ids = train.router_topk(logits.requires_grad_(), 2)
    h = torch.randn(M, K, device="cuda").bfloat16().requires_grad_()
    rows, offsets, src2dst, counts = train._Permute.apply(h, ids, weights, E)
    out = train._WeightedGather.apply(train.grouped_matmul(rows, torch.eye(K, device="cuda").bfloat16().repeat(E, 1, 1),
                                                           offsets, counts), src2dst, weights, ids, counts)
    assert not out[::3].any()
    out.sum().backward()
    assert not h.grad[::3].any() and h.grad[1].any() and torch.isfinite(h.grad).all()
    assert not logits.grad[::3].any() and torch.isfinite(logits.grad).all()
