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
