"""One training step of a pre-norm MoE block with 16-bit expert weights.

The library's training operators as autograd functions, and the block they make together:

    h = layer_norm(x);  logits = h gate^T (fp32);  weights, ids = router_topk(logits)
    rows of h, sorted by expert (moe_scatter) -> w13 -> SiLU-and-mul -> w2 (grouped products)
    out = x + the rows' outputs, weighted and summed per token (moe_gather_weight_reduce)

Nothing of it reads the experts' row counts on the host. The permutation's gradients are the
library's own pair again: the gradient of the weighted gather is a scatter of the output's
gradient that applies the weights, the gradient of the scatter a gather with unit weights.
The activation between the products and the dot product that gives the gradient of a routing
weight are plain torch operations. There are no second gradients.

`python -m moe_expert_layer_count_gb300.train` runs a few steps on synthetic data.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

import moe_expert_layer_count_gb300 as moe


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = moe.moe_layer_norm(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = moe.moe_layer_norm_backward(dy.contiguous(), x, weight, mean, rstd, has_bias=ctx.has_bias)
        return dx, dw, db, None


class _RouterTopk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, topk, scoring, renormalize, scale, bias):
        weights, ids = moe.moe_router_topk(logits, topk, scoring, renormalize, scale, bias)
        ctx.save_for_backward(logits, ids)
        ctx.how = (scoring, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dweights, _):
        logits, ids = ctx.saved_tensors
        return moe.moe_router_topk_backward(logits, ids, dweights.contiguous(), *ctx.how), None, None, None, None, None


class _GroupedMatmul(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, counts, out_dtype, gaps):
        ctx.save_for_backward(x, w, offsets, counts)
        ctx.gaps = gaps
        return moe.moe_grouped_matmul(x, w, offsets, counts, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, offsets, counts = ctx.saved_tensors
        dy = dy.to(w.dtype).contiguous()  # the products' operands have one 16-bit type
        dx = None
        if ctx.needs_input_grad[0]:
            # the product does not write the rows of no group
            out = torch.zeros_like(x) if ctx.gaps else None
            dx = moe.moe_grouped_matmul_dgrad(dy, w, offsets, counts, out=out)
        dw = moe.moe_grouped_matmul_wgrad(dy, x, offsets, counts) if ctx.needs_input_grad[1] else None
        return dx, dw, None, None, None, None


class _Permute(torch.autograd.Function):
    """Rows of h sorted by expert in 128-aligned blocks, as moe_scatter lays them out."""

    @staticmethod
    def forward(ctx, h, ids, weights, n_experts):
        counts = torch.empty(n_experts, dtype=torch.int32, device=h.device)
        rows, _, offsets, src2dst = moe.moe_scatter(h, ids, weights, n_experts, n_experts, counts, quant=moe.MOE_QUANT_NONE,
                                                    count_here=True)
        ctx.save_for_backward(src2dst, weights)
        ctx.mark_non_differentiable(offsets, src2dst, counts)
        return rows, offsets, src2dst, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, drows, *_):
        src2dst, weights = ctx.saved_tensors
        # unit weights: every kept slot's row once
        return moe.moe_gather_weight_reduce(drows.contiguous(), src2dst, weights, True), None, None, None


class _WeightedGather(torch.autograd.Function):
    """out[t] = sum over k of weights[t, k] * rows[src2dst[t, k]]."""

    @staticmethod
    def forward(ctx, rows, src2dst, weights, ids, counts):
        ctx.save_for_backward(rows, src2dst, weights, ids, counts)
        return moe.moe_gather_weight_reduce(rows, src2dst, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        rows, src2dst, weights, ids, counts = ctx.saved_tensors
        dout = dout.contiguous()
        n = counts.numel()
        drows, _, _, _ = moe.moe_scatter(dout, ids, weights, n, n, counts, apply_router_weight_on_input=True,
                                         quant=moe.MOE_QUANT_NONE, rp_cap=rows.shape[0])
        # a few tensors of tokens x hidden size at a time, not of every token's chosen rows
        M, topk = src2dst.shape
        dots = torch.empty(M, topk, dtype=torch.float32, device=dout.device)
        step = max(256, -(-2 * M // topk))
        for i in range(0, M, step):
            s = slice(i, i + step)
            dots[s] = (rows[src2dst[s].clamp(min=0).long()] * dout[s].float()[:, None, :]).sum(-1)  # products in fp32
        return drows, None, torch.where(src2dst >= 0, dots, 0.0), None, None


def layer_norm(x, weight, bias=None, eps=1e-5):
    """moe_layer_norm under autograd: y."""
    return _LayerNorm.apply(x, weight, bias, eps)


def router_topk(logits, topk, scoring=moe.MOE_SCORE_SOFTMAX, renormalize=True, scale=1.0, bias=None):
    """moe_router_topk under autograd: (weights, ids)."""
    return _RouterTopk.apply(logits, topk, scoring, renormalize, scale, bias)


def grouped_matmul(x, w, expert_offsets, expert_num_tokens=None, out_dtype=None, gaps=True):
    """moe_grouped_matmul under autograd. Rows of no group have an undefined result and no influence: their
    gradient is 0. gaps=False leaves it undefined too, which saves a pass of writing: for callers whose groups
    hold every row, or who do not use the others'."""
    return _GroupedMatmul.apply(x, w, expert_offsets, expert_num_tokens, out_dtype, gaps)


def init_block(K: int, N: int, E: int, device="cuda", seed: int = 0):
    """Parameters of a block: hidden size K and intermediate size N (multiples of 128), E experts
    (a multiple of 8: the gate is one of the 16-bit products)."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return (0.02 * torch.randn(*shape, device=device, generator=g)).bfloat16().requires_grad_()
    return {"norm_weight": torch.ones(K, device=device).requires_grad_(), "norm_bias": torch.zeros(K, device=device).requires_grad_(),
            "gate": normal(1, E, K), "w13": normal(E, 2 * N, K), "w2": normal(E, K, N)}


def moe_block(p, x, topk: int, scoring=moe.MOE_SCORE_SOFTMAX, renormalize=True, eps=1e-5):
    """x + MoE(layer_norm(x)) for x bf16 [M, K] and the parameters of init_block."""
    E, N2, _ = p["w13"].shape
    h = layer_norm(x, p["norm_weight"], p["norm_bias"], eps)
    # made on the device: the block can be captured in a CUDA graph
    everyone = torch.arange(2, dtype=torch.int32, device=x.device) * x.shape[0]
    logits = grouped_matmul(h, p["gate"], everyone, out_dtype=torch.float32, gaps=False)
    weights, ids = router_topk(logits, topk, scoring, renormalize)
    rows, offsets, src2dst, counts = _Permute.apply(h, ids, weights, E)
    # the permutation's gradient reads no row between the groups, and everything up to it is row by row
    gate, up = grouped_matmul(rows, p["w13"], offsets, counts, gaps=False).split(N2 // 2, dim=1)
    out = grouped_matmul(torch.nn.functional.silu(gate) * up, p["w2"], offsets, counts, gaps=False)
    return x + _WeightedGather.apply(out, src2dst, weights, ids, counts)


def train_step(p, x, target, topk: int, lr: float, max_norm: float):
    """One step of gradient descent on the tokens' mean squared distance to `target`: backward pass, clipping of all gradients by their common norm, update. Returns the loss
    and the norm before clipping, as device tensors."""
    for v in p.values():
        v.grad = None
    loss = (moe_block(p, x, topk).float() - target.float()).square().sum(1).mean()
    loss.backward()
    grads = [v.grad for v in p.values()]
    norm = moe.moe_clip_grad_norm(grads, max_norm)
    with torch.no_grad():
        for v in p.values():
            v.sub_(v.grad.to(v.dtype), alpha=lr)
    return loss.detach(), norm


def main():
    M, K, N, E, topk = 4096, 2048, 768, 128, 8
    p = init_block(K, N, E)
    x = torch.randn(M, K, device="cuda").bfloat16()
    target = x + 0.1 * torch.roll(x, 1, dims=1)
    for i in range(5):
        loss, norm = train_step(p, x, target, topk, lr=2.0, max_norm=1.0)
        print(f"step {i}: loss {loss.item():.6f}, gradient norm {norm.item():.4f}")


if __name__ == "__main__":
    main()
