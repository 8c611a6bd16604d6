"""The router where one value counts as another, and far from the row's maximum."""
import itertools

import numpy as np
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from test_gpu_router import FMAX, SIGM, SOFT, check_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,topk", [(8, 1), (8, 4), (9, 3), (24, 12), (33, 16), (40, 20)])
@pytest.mark.parametrize("scoring,renorm", [(SOFT, True), (SOFT, False), (SIGM, True), (SIGM, False)])
def test_infinity_ties_with_the_largest_finite_value(E, topk, scoring, renorm):
    """+inf counts as the largest finite value: among both, the lowest index comes first."""
    inf = float("inf")
    rows = []
    for a, b, c in itertools.product([FMAX, inf, 1.0], repeat=3):
        row = [0.25 * (i % 5) for i in range(E)]
        row[0], row[E // 2], row[E - 1] = a, b, c
        rows.append(row)
    check_forward(torch.tensor(rows, device="cuda"), topk, scoring, renorm, 1.0)


@pytest.mark.parametrize("E", [128, 100, 1000])
def test_gradient_far_below_the_maximum(E):
    """fp32 logits 0, 0 and negative multiples of 1/4, the first one chosen. Experts that were not chosen get
    rest * exp(l), the second one rest itself: their ratios have the exponential's 2 ulp (4 * 2^-24) and
    the product's rounding, however small they are."""
    rng = np.random.default_rng(E)
    l = -rng.integers(1, 320, (64, E)).astype(np.float32) / 4
    l[:, :2] = 0.0
    ids = torch.zeros(64, 1, dtype=torch.int32, device="cuda")
    g = torch.ones(64, 1, device="cuda")
    d = moe.moe_router_topk_backward(torch.from_numpy(l).cuda(), ids, g, SOFT, False, 1.5).double().cpu().numpy()
    assert (d[:, 1] < 0).all()
    ref = np.exp(l[:, 2:].astype(np.float64))
    rel = np.abs(d[:, 2:] / d[:, 1:2] - ref) / ref
    assert rel.max() <= 5.01 * 2.0 ** -24, rel.max() * 2.0 ** 24
