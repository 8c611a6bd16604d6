"""Gates and ups that are not finite, through the gated product and its backward pass: the results are finite,
infinite or NaN exactly where the formulas' 64-bit values are, for both activations and both forms of what is kept."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from test_gpu_gated import ACTS, U, parts

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
N = 48  # three groups of the 8-bit form


def kept_values(dtype):
    """g and u [5, 2 N]: a row of each kind of value, and one without any."""
    g = torch.Generator(device="cuda").manual_seed(1)
    pre = (1.0 + torch.rand(5, 2 * N, device="cuda", generator=g)) * torch.where(torch.rand(5, 2 * N, device="cuda", generator=g) < 0.5, -1, 1)
    pre[0, 3], pre[1, 17], pre[2, 40] = NAN, INF, -INF                       # gates
    pre[3, N + 5], pre[3, N + 21], pre[3, N + 47], pre[3, 30] = NAN, INF, -INF, NAN  # ups, and a gate of another group
    return pre.to(dtype)


def same_kind(got, ref, dtype):
    """NaN where the formula's value is, infinities of its sign, and near it elsewhere."""
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.isinf(), ref.isinf())
    assert torch.equal(got[got.isinf()].double(), ref[ref.isinf()])
    fine = ref.isfinite()
    # gates of at most 2 in size: |q| and |t q'| stay below 5, so that the activation and its slope (which crosses 0, so the
    # bound is no relative one) are off by at most (6 + 4 * 5) * 2^-23 * (1 + 5) < 2^-15, times dh * u of at most 4
    assert ((got.double() - ref).abs()[fine] <= U[dtype] * ref.abs()[fine] + 2.0 ** -13).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("eight", [False, True])
def test_backward(dtype, act, eight):
    pre = kept_values(dtype)
    R = pre.shape[0]
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    w2 = torch.eye(N, device="cuda").to(dtype)[None].contiguous()  # dh is dy
    dy = (1.0 + torch.rand(R, N, device="cuda", generator=torch.Generator("cuda").manual_seed(2))).to(dtype)
    if eight:
        codes, scale = moe.moe_checkpoint_pack(pre)
        d, h = moe.moe_grouped_gated_backward(dy, w2, codes, off, activation=ACTS[act], pre_scale=scale)
        pre = moe.moe_checkpoint_unpack(codes, scale, dtype)
        assert pre[0, :16].isnan().all() and pre[1, 16:32].isnan().all() and pre[4].isfinite().all()
    else:
        d, h = moe.moe_grouped_gated_backward(dy, w2, pre, off, activation=ACTS[act])
    g, u, dh = pre[:, :N].double(), pre[:, N:].double(), dy.double()
    a, slope, _, _ = parts(g, act)
    same_kind(d[:, :N], dh * u * slope, dtype)
    same_kind(d[:, N:], dh * a, dtype)
    same_kind(h, a * u, dtype)
    # what the formula makes of a NaN gate: nothing that looks sound
    bad = g.isnan()
    assert d[:, :N][bad].isnan().all() and d[:, N:][bad].isnan().all() and h[bad].isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_forward(dtype, act):
    """Each output's gate and up are one weight times 1."""
    pre = kept_values(dtype)
    for r in range(pre.shape[0]):
        x = torch.ones(1, 8, device="cuda").to(dtype)
        w13 = torch.zeros(1, 2 * N, 8, device="cuda").to(dtype)
        w13[0, :, 0] = pre[r]
        off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        h, kept, _ = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act], keep=moe.MOE_KEEP_16BIT)
        assert torch.equal(kept[0].isnan(), pre[r].isnan()) and torch.equal(kept[0].nan_to_num(9, 8, -8), pre[r].nan_to_num(9, 8, -8))
        g, u = pre[r, :N].double(), pre[r, N:].double()
        same_kind(h[0], parts(g, act)[0] * u, dtype)
        _, codes, scale = moe.moe_grouped_gated(x, w13, off, activation=ACTS[act], keep=moe.MOE_KEEP_E4M3)
        want = moe.moe_checkpoint_pack(pre[r:r + 1].contiguous())
        assert torch.equal(scale, want[1])
        assert torch.equal(moe.moe_checkpoint_unpack(codes, scale, dtype).nan_to_num(99), moe.moe_checkpoint_unpack(*want, dtype).nan_to_num(99))
