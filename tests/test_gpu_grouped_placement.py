"""The grouped products find every group's rows whatever the groups' number and lengths: one warp's groups or several,
groups of one part, of several, in their own order and by turns, empty ones between. Products of 16-bit values summed in
fp32: off by at most K * 2^-23 * sum |a||b|, and one rounding (2^-8)."""
import random

import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu


def batch(E, kind):
    r = random.Random(E)
    if kind == "short":      # no group of several parts
        return [r.choice([0, 1, 7, 16, 33, 64]) for _ in range(E)]
    if kind == "few long":   # in the groups' own order
        return [r.choice([0, 3, 90, 200]) if l % 37 else 600 for l in range(E)]
    if kind == "long":       # by turns
        return [r.choice([0, 5, 257, 513, 1200]) for l in range(E)]
    return [0] * (E - 1) + [300] if kind == "last" else [300] + [0] * (E - 1)


@pytest.mark.parametrize("E", [1, 31, 32, 33, 64, 192, 193, 200, 577, 1024])
@pytest.mark.parametrize("kind", ["short", "few long", "long", "last", "first"])
def test_every_row_of_every_group(E, kind):
    if kind == "long" and E > 200:
        pytest.skip("covered by 200 groups, and large")
    counts, N, K = batch(E, kind), 72, 40
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    R = off[-1] + 3
    if off[-1] == 0:
        counts[0], off = 2, [0] + [2] * E
        R = 5
    g = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randn(R, K, device="cuda", generator=g).bfloat16()
    dy = torch.randn(R, N, device="cuda", generator=g).bfloat16()
    w = torch.randn(E, N, K, device="cuda", generator=g).bfloat16()
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(counts, device="cuda"))  # each row's group
    n = off[-1]

    def check(got, a, b):
        """got[r] against b[of r] a[r], some thousand rows at a time."""
        for i in range(0, n, 4096):
            s = slice(i, min(i + 4096, n))
            bb = b[of[s]].double()
            ref = torch.einsum("rk,rnk->rn", a[s].double(), bb)
            mag = torch.einsum("rk,rnk->rn", a[s].double().abs(), bb.abs())
            tol = a.shape[1] * 2.0 ** -23 * mag + 2.0 ** -8 * ref.abs() + 2.0 ** -100
            assert ((got[s].double() - ref).abs() <= tol).all()
    out = torch.full((R, N), 7.0, device="cuda").bfloat16()
    check(moe.moe_grouped_matmul(x, w, offsets, out=out), x, w)
    dx = torch.full((R, K), 7.0, device="cuda").bfloat16()
    check(moe.moe_grouped_matmul_dgrad(dy, w, offsets, out=dx), dy, w.transpose(1, 2))
    assert (out[n:] == 7).all() and (dx[n:] == 7).all()
    # the gated forms take the same groups; what is kept is the plain product
    half = w[:, :N - N % 16].contiguous()
    _, pre, _ = moe.moe_grouped_gated(x, half, offsets, keep=moe.MOE_KEEP_16BIT)
    check(pre, x, half)
    assert moe.moe_device_error() == 0
