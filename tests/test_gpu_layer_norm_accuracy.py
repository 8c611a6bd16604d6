"""The accuracy of layer norm where the mean is large against the spread, and of its statistics.

x - mean is one subtraction: xh = (x - mean) * rstd is good to two roundings relative to itself, however
large the mean. Sums as in test_gpu_layer_norm: c = (K / 256 + 32) * 2^-23 over a row, 512 additions
in a row over the rows. Every product and sum around them adds a rounding: 8 in all."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from test_gpu_layer_norm import inside, make, stored

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


# rows of whole vectors, of several rows a block, of single values, and the looping kernels'
@pytest.mark.parametrize("M,K", [(300, 2048), (700, 96), (64, 8192), (300, 1111), (40, 5001), (5, 16387)])
@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1000.0), (torch.float32, -30.0), (torch.bfloat16, 100.0),
                                         (torch.float16, 1000.0)])
def test_gradients_of_rows_far_from_zero(M, K, dtype, shift):
    x, w, b, dy = make(M, K, dtype, torch.float32, shift=shift, seed=K)
    _, mean, rstd = moe.moe_layer_norm(x, w, b)
    dx, dw, db = moe.moe_layer_norm_backward(dy, x, w, mean, rstd)
    c = (K / 256 + 32) * 2.0 ** -23
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = (x.double() - mu) * rs
    D = dy.double()
    G = D * w.double()
    a, bb = G.mean(1, keepdim=True), (G * xh).mean(1, keepdim=True)
    ref = rs * (G - a - xh * bb)
    tol = rs * (c * G.abs().mean(1, keepdim=True) + xh.abs() * c * (G * xh).abs().mean(1, keepdim=True) +
                8 * E * (G.abs() + a.abs() + (xh * bb).abs()))
    inside(dx, ref, tol + stored(dtype, ref))
    inside(dw, (D * xh).sum(0), (D * xh).abs().sum(0) * 520 * E)
    # the columns' sums over random signs: their errors, too, are far below the worst case
    err = (dw.double() - (D * xh).sum(0)).norm() / (D * xh).sum(0).norm()
    assert err <= 8 * E, err.item()


@pytest.mark.parametrize("K", [96, 1111, 1536, 5000, 9000, 10001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mean_is_the_quotient(K, dtype):
    """Rows of small whole numbers: every sum is exact, so that the mean has one rounding."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randint(-8, 9, (4096, K), device="cuda", generator=g).to(dtype)
    w = torch.ones(K, device="cuda")
    _, mean, _ = moe.moe_layer_norm(x, w, w)
    ref = x.double().sum(1) / K
    assert ((mean.double() - ref).abs() <= E * ref.abs()).all(), ((mean.double() - ref).abs() / ref.abs()).nan_to_num(0).max() / E


@pytest.mark.parametrize("K", [64, 2048, 8192, 32768])
def test_reciprocal_root(K):
    """Rows of +a and -a, a of 8 bits: mean 0 and variance a^2 exactly (no partial sum of the squares has more
    than 23 bits), so that rstd has the root's and the quotient's rounding and no other."""
    a = torch.arange(1, 257, device="cuda", dtype=torch.float32) / 64
    sign = torch.ones(K, device="cuda")
    sign[1::2] = -1
    w = torch.ones(K, device="cuda")
    _, mean, rstd = moe.moe_layer_norm(a[:, None] * sign, w, w, eps=0.0)
    assert not mean.any()
    ref = 1 / a.double()
    assert ((rstd.double() - ref).abs() <= 2 * E * ref).all(), ((rstd.double() - ref).abs() / ref).max().item() / E


@pytest.mark.parametrize("M,K", [(50, 640), (9, 2048), (300, 96), (7, 8192), (33, 1111), (3, 16384), (2, 20000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [1, 3])
def test_results_do_not_depend_on_alignment(M, K, dtype, shift):
    x, w, b, dy = make(M, K, dtype, torch.float32, seed=K)

    def moved(t):
        base = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        base[shift:shift + t.numel()].copy_(t.reshape(-1))
        return base[shift:shift + t.numel()].view(t.shape)
    first = moe.moe_layer_norm(x, w, b)
    second = moe.moe_layer_norm(moved(x), moved(w), moved(b))
    assert all(torch.equal(p, q) for p, q in zip(first, second))
    first = moe.moe_layer_norm_backward(dy, x, w, *first[1:])
    second = moe.moe_layer_norm_backward(moved(dy), moved(x), moved(w), *second[1:])
    assert all(torch.equal(p, q) for p, q in zip(first, second))


@pytest.mark.parametrize("K", [1111, 2048, 20000])
def test_mean_of_rows_that_hold_infinities(K):
    x = torch.randn(4, K, device="cuda")
    x[0, 3], x[1, 5], x[2, 7], x[2, 8] = float("inf"), -float("inf"), float("inf"), -float("inf")
    w = torch.ones(K, device="cuda")
    mean = moe.moe_layer_norm(x, w, w)[1].tolist()
    assert mean[0] == float("inf") and mean[1] == -float("inf") and mean[2] != mean[2] and abs(mean[3]) < 1
