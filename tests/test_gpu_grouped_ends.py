"""Ragged group ends of the weights' gradient: the values behind an end, which the second CTA of a pair takes
out of its shared memory, never reach the products that the first CTA issues."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from test_gpu_grouped_matmul import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K", [(256, 512), (520, 264)])
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
def test_every_end_in_every_stage(N, K, out_dtype):
    """600 groups of 1 to 200 rows with infinities and NaN between them, so that ends of every length fall
    into every stage of the ring, many times."""
    g = torch.Generator().manual_seed(N)
    counts = torch.randint(1, 201, (600,), generator=g).tolist()
    off, at = [], 0
    for c in counts:
        off.append(at)
        at += c + 16
    x = torch.randn(at, K, device="cuda").bfloat16()
    dy = torch.randn(at, N, device="cuda").bfloat16()
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").bfloat16()
    for o, c in zip(off, counts):
        x[o + c:o + c + 16] = bad[torch.arange(16, device="cuda") % 3][:, None]
        dy[o + c:o + c + 16] = bad[torch.arange(16, device="cuda") % 3][:, None]
    offsets = torch.tensor(off + [at], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    first = moe.moe_grouped_matmul_wgrad(dy, x, offsets, cnt, out_dtype=out_dtype)
    for l in range(0, 600, 7):
        rows = slice(off[l], off[l] + counts[l])
        close(first[l], dy[rows].double().T, x[rows].double(), counts[l])
    assert torch.isfinite(first).all()
    for _ in range(20):
        assert torch.equal(first, moe.moe_grouped_matmul_wgrad(dy, x, offsets, cnt, out_dtype=out_dtype))
    assert moe.moe_device_error() == 0
