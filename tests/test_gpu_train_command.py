"""The training command: what it prints are numbers, and the fused kernels' gradients are those of the torch
activation but for their roundings."""
import re

import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep", ["torch", "16bit", "8bit"])
def test_prints_finite_losses_and_norms(keep, capsys):
    train.main(["--keep", keep])
    found = re.findall(r"^step (\d): loss (\d+\.\d+), gradient norm (\d+\.\d+)$", capsys.readouterr().out, flags=re.M)
    assert [s for s, _, _ in found] == list("01234")
    assert all(float(loss) > 0 and float(norm) > 0 for _, loss, norm in found)


@pytest.mark.parametrize("keep", [moe.MOE_KEEP_16BIT, moe.MOE_KEEP_E4M3])
def test_a_steps_gradients_are_the_torch_activations(keep):
    """One step without clipping, each parameter's gradient. Each way makes at most eight roundings of 2^-8 on the way to
    a gradient, so that two ways are at most 2^-4 apart in the relative 2-norm; 8 bits add 2^-4 for each of three
    factors. A gradient of the wrong sign is 2 away, one without a term about 1."""
    M, K, N, E, topk = 128, 256, 128, 8, 2
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    target = x + 0.3 * torch.roll(x, 1, dims=1)
    grads = []
    for k in (None, keep):
        p = train.init_block(K, N, E, seed=3)
        with torch.no_grad():
            for name in ("gate", "w13", "w2"):
                p[name].mul_(4)
        train.train_step(p, x, target, topk, lr=0.0, max_norm=1e30, keep=k)
        grads.append({n: v.grad.double() for n, v in p.items()})
    bound = 2 ** -4 + (0 if keep == moe.MOE_KEEP_16BIT else 3 * 2 ** -4)
    for n, want in grads[0].items():
        assert (grads[1][n] - want).norm() <= bound * want.norm(), n
