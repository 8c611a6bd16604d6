"""Layer norm and its gradients against their definitions in 64 bits.

Bounds: a sum over K columns is at most K/256 + 32 additions in a row, so with
c = (K/256 + 32) * 2^-23 the mean is off by c * mean|x| and the variance (of the values
minus that mean) by c relative; a sum over rows has at most 512 additions in a row. A stored
value is rounded by u (2^-8 bf16, 2^-11 fp16, 2^-24 fp32), fp16 by 2^-25 at least."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def stored(dtype, ref):
    return U[dtype] * ref.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def inside(got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"worst excess {(err - tol).max().item():.3g} of {tol.max().item():.3g}"


def make(M, K, dtype, pdtype, shift=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(M, K, device="cuda", generator=g) * (0.5 + torch.rand(M, 1, device="cuda", generator=g)) + shift).to(dtype)
    w = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(pdtype)
    b = (0.2 * torch.randn(K, device="cuda", generator=g)).to(pdtype)
    dy = torch.randn(M, K, device="cuda", generator=g).to(dtype)
    return x, w, b, dy


def check(x, w, b, dy, eps=1e-5):
    M, K = x.shape
    c = (K / 256 + 32) * 2.0 ** -23
    y, mean, rstd = moe.moe_layer_norm(x, w, b, eps)
    X, W = x.double(), w.double()
    mu = X.mean(1, keepdim=True)
    var = (X - mu).square().mean(1, keepdim=True)
    rs = 1 / (var + eps).sqrt()
    xh = (X - mu) * rs
    dmu = c * X.abs().mean(1, keepdim=True)
    drs = c * rs + rs * (dmu * rs) ** 2
    inside(mean[:, None], mu, dmu + 1e-40)
    inside(rstd[:, None], rs, drs)
    ref = xh * W + (b.double() if b is not None else 0)
    tol = W.abs() * (rs * dmu + xh.abs() * (c + (dmu * rs) ** 2) + 4 * 2.0 ** -24 * (X.abs() + mu.abs()) * rs)
    inside(y, ref, tol * 1.01 + 2.0 ** -23 * ref.abs() + stored(x.dtype, ref))
    # backward, from the statistics that the forward pass returned
    dx, dw, db = moe.moe_layer_norm_backward(dy, x, w, mean, rstd)
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = (X - mu) * rs
    e = 4 * 2.0 ** -24 * (X.abs() + mu.abs()) * rs          # error of xh itself
    D = dy.double()
    G = D * W
    a, bb = G.mean(1, keepdim=True), (G * xh).mean(1, keepdim=True)
    ref = rs * (G - a - xh * bb)
    da = c * G.abs().mean(1, keepdim=True)
    dbb = c * (G * xh).abs().mean(1, keepdim=True) + (G.abs() * e).mean(1, keepdim=True)
    tol = rs * (da + xh.abs() * dbb + e * bb.abs() + 4 * 2.0 ** -24 * (G.abs() + a.abs() + (xh * bb).abs()))
    inside(dx, ref, tol * 1.01 + stored(x.dtype, ref))
    ref, mag = (D * xh).sum(0), (D * xh).abs().sum(0) * 512 * 2.0 ** -24 + (D.abs() * e).sum(0)
    inside(dw, ref, mag + stored(w.dtype, ref))
    ref, mag = D.sum(0), D.abs().sum(0) * 512 * 2.0 ** -24
    inside(db, ref, mag + stored(w.dtype, ref))
    return dx, dw, db


@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 7), (1, 2048), (64, 2048), (1000, 64), (257, 96), (5, 1111), (300, 1000),
                                 (33, 4096), (7, 8192), (2, 16384), (3, 16385), (2, 40000), (2500, 264), (9, 5000), (4, 12296)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("wide", [False, True])
def test_forward_and_backward(M, K, dtype, wide):
    check(*make(M, K, dtype, torch.float32 if wide else dtype, seed=M + K))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_far_from_zero(dtype):
    check(*make(40, 1024, dtype, torch.float32, shift=50.0))


def test_constant_and_zero_rows():
    x, w, b, dy = make(6, 520, torch.float32, torch.float32)
    x[0], x[1], x[2] = 0.0, 3.0, -1e-20
    check(x, w, b, dy)
    y, _, rstd = moe.moe_layer_norm(x, w, b)
    assert torch.equal(y[0], b) and torch.allclose(rstd[:3], torch.full((3,), 1e-5 ** -0.5, device="cuda"), rtol=1e-6)


def test_a_bad_row_stays_alone():
    x, w, b, dy = make(10, 256, torch.bfloat16, torch.bfloat16)
    good = moe.moe_layer_norm(x, w, b)[0]
    x[4, 7], x[6, 0] = float("nan"), float("inf")
    y, _, _ = moe.moe_layer_norm(x, w, b)
    keep = [i for i in range(10) if i not in (4, 6)]
    assert torch.equal(y[keep], good[keep]) and torch.isnan(y[4]).all() and not torch.isfinite(y[6]).all()


def test_without_bias_in_place_and_views():
    x, w, b, dy = make(50, 640, torch.bfloat16, torch.float32)
    check(x, w, None, dy)
    y, mean, rstd = moe.moe_layer_norm(x, w, b)
    inplace = x.clone()
    moe.moe_layer_norm(inplace, w, b, out=inplace)
    assert torch.equal(inplace, y)
    dx, dw, db = moe.moe_layer_norm_backward(dy, x, w, mean, rstd)
    d2 = dy.clone()
    r = moe.moe_layer_norm_backward(d2, x, w, mean, rstd, dx=d2)
    assert torch.equal(d2, dx) and torch.equal(r[1], dw) and torch.equal(r[2], db)
    # buffers that start between two 16-byte boundaries
    for shift in (1, 3):
        base = torch.empty(50 * 640 + 8, dtype=torch.bfloat16, device="cuda")
        xs = base[shift:shift + 50 * 640].view(50, 640)
        xs.copy_(x)
        assert torch.equal(moe.moe_layer_norm(xs, w, b)[0], y)
        got = moe.moe_layer_norm_backward(dy, xs, w, mean, rstd)
        ref = check(x, w, b, dy)
        assert torch.allclose(got[0].float(), ref[0].float(), rtol=2 ** -7, atol=1e-5)


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert moe.moe_layer_norm(x, w, w)[0].shape == (0, 64)
    e = torch.empty(0, device="cuda")
    dx, dw, db = moe.moe_layer_norm_backward(x, x, w, e, e, d_weight=torch.ones(64, device="cuda"))
    assert not dw.any() and not db.any()


def test_gradients_against_differences():
    x, w, b, dy = make(7, 120, torch.float32, torch.float32, seed=8)
    dx, dw, db = check(x, w, b, dy)

    def loss(x, w, b):
        mu = x.mean(1, keepdim=True)
        return (dy.double() * ((x - mu) / ((x - mu).square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b)).sum()
    at = [t.double() for t in (x, w, b)]
    for k, d in enumerate((dx, dw, db)):
        u = torch.randn_like(at[k])
        h = 1e-5
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + h * u, at[k] - h * u
        num = (loss(*up) - loss(*down)) / (2 * h)
        # differences: h^2 times third derivatives and the loss's rounding over h, below 1e-7
        assert abs(num - (d.double() * u).sum()) <= 1e-5 * (d.double() * u).abs().sum() + 1e-7


def test_same_result_every_call_and_on_another_stream():
    x, w, b, dy = make(3000, 768, torch.bfloat16, torch.float32)
    y, mean, rstd = moe.moe_layer_norm(x, w, b)
    first = moe.moe_layer_norm_backward(dy, x, w, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = moe.moe_layer_norm_backward(dy, x, w, mean, rstd, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_offsets_past_2_31_values():
    M, K = (1 << 31) // 4096 + 5, 4096
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-4:].normal_()
    w, b = torch.ones(K, device="cuda"), torch.zeros(K, device="cuda")
    y, mean, rstd = moe.moe_layer_norm(x, w, b)
    y4, mean4, rstd4 = moe.moe_layer_norm(x[-4:], w, b)
    assert torch.equal(y[-4:], y4) and torch.equal(mean[-4:], mean4)
    dx, dw, db = moe.moe_layer_norm_backward(x, x, w, mean, rstd)
    dx4, dw4, db4 = moe.moe_layer_norm_backward(x[-4:], x[-4:], w, mean4, rstd4)
    assert torch.equal(dx[-4:], dx4) and torch.allclose(dw, dw4, rtol=1e-5, atol=1e-5)
