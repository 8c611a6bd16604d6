"""gated_experts where the down projection's results are of another width than the rows."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train
from test_gpu_gated import U, inside, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out_width", [40, 136])
@pytest.mark.parametrize("gaps", [True, False])
@pytest.mark.parametrize("keep", [moe.MOE_KEEP_16BIT, moe.MOE_KEEP_E4M3])
def test_results_of_another_width(out_width, gaps, keep):
    """The gradients are those of the kernels that the backward pass is made of, bit for bit, and rows of no group have a
    gradient of 0."""
    counts, N, K, gap = [33, 0, 70, 1], 64, 72, 3
    x, _, w13, _, _, off = make(counts, N, K, torch.bfloat16, gap=gap, seed=2)
    R = x.shape[0]
    g = torch.Generator(device="cuda").manual_seed(3)
    w2 = torch.randn(len(counts), out_width, N, device="cuda", generator=g).bfloat16()
    dy = torch.randn(R, out_width, device="cuda", generator=g).bfloat16()
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    t = [v.clone().requires_grad_() for v in (x, w13, w2)]
    y = train.gated_experts(*t, off, cnt, keep=keep, gaps=gaps)
    assert y.shape == (R, out_width)
    dx, dw13, dw2 = torch.autograd.grad(y, t, dy)
    assert dx.shape == x.shape and dw13.shape == w13.shape and dw2.shape == w2.shape
    live = inside(off, counts, R)
    if gaps:
        assert not dx[~live].any()
    h, pre, scale = moe.moe_grouped_gated(x, w13, off, cnt, keep=keep)
    d_pre, again = moe.moe_grouped_gated_backward(dy, w2, pre, off, cnt, pre_scale=scale)
    rows = x if scale is None else moe.moe_checkpoint_unpack(*moe.moe_checkpoint_pack(x), x.dtype)
    assert torch.equal(y[live], moe.moe_grouped_matmul(h, w2, off, cnt)[live])
    assert torch.equal(dx[live], moe.moe_grouped_matmul_dgrad(d_pre, w13, off, cnt)[live])
    assert torch.equal(dw13, moe.moe_grouped_matmul_wgrad(d_pre, rows, off, cnt))
    assert torch.equal(dw2, moe.moe_grouped_matmul_wgrad(dy, again, off, cnt))
    for l, c in enumerate(counts):  # and near the formula: two roundings of factors of at most 2^-8 and one of the result
        s = slice(int(off[l]), int(off[l]) + c)
        want, mag = d_pre[s].double() @ w13[l].double(), d_pre[s].double().abs() @ w13[l].double().abs()
        assert ((dx[s].double() - want).abs() <= U[torch.bfloat16] * want.abs() + 2 * N * 2.0 ** -23 * mag).all()
