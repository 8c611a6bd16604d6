"""The norm of a list of tensors and clipping by it, against 64 bits.

Bounds: a thread adds at most 128 squares in fp32 before the sum goes on in fp64: the sum of
squares is good to 128 * 2^-24 relative, the norm to half of that and one rounding. A
clipped value has that error, the quotient's and the product's rounding, and is rounded by
u (2^-8 bf16, 2^-11 fp16)."""
import math

import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
REL = 66 * 2.0 ** -24
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def exact_norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def make(sizes, dtypes, std=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(std * torch.randn(n, device="cuda", generator=g)).to(d) for n, d in zip(sizes, dtypes)]


def check(ts, max_norm, out=None):
    ref = exact_norm(ts)
    norm = moe.moe_grad_norm(ts).item()
    assert abs(norm - ref) <= REL * ref
    before = [t.clone() for t in ts]
    got = moe.moe_clip_grad_norm(ts, max_norm, out=out)
    assert got.item() == norm
    res = ts if out is None else out
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(ts, before))
    c = max_norm / ref if ref > max_norm else 1.0
    for r, b in zip(res, before):
        if norm <= max_norm:
            assert torch.equal(r.view(-1), b.view(-1))
        else:
            want = b.double() * c
            tol = (U[r.dtype] + REL + 2.0 ** -22) * want.abs() + (2.0 ** -25 if r.dtype == HF else 1e-45)
            assert ((r.double().view(-1) - want.view(-1)).abs() <= tol.view(-1)).all()


@pytest.mark.parametrize("sizes", [[1], [7], [16384], [16385, 1], [100001, 3, 0, 65536, 17], [5] * 300, [1 << 22], [8, 0]])
@pytest.mark.parametrize("kind", [[BF], [HF], [FP], [BF, FP, HF]])
@pytest.mark.parametrize("max_norm", [0.05, 1e8])
def test_norm_and_clip(sizes, kind, max_norm):
    ts = make(sizes, [kind[i % len(kind)] for i in range(len(sizes))], 0.5, seed=len(sizes))
    check(ts, max_norm, [torch.full_like(t, 9.0) for t in ts])
    check(ts, max_norm)


def test_views_off_the_16_byte_grid():
    base, other = make([40000, 40000], [BF, BF])
    for a, b in ((1, 1), (3, 0), (0, 5), (2, 6)):
        ts = [base[a:a + 17001], base[18000 + a:18003 + a]]
        check(ts, 0.5, [other[b:b + 17001], other[18000 + b:18003 + b]])
    flat = torch.full((300,), 4.0, device="cuda")
    moe.moe_clip_grad_norm([flat[5:100], flat[101:103]], 1.0)
    assert (flat[:5] == 4).all() and flat[100] == 4 and (flat[103:] == 4).all() and (flat[5:100] < 4).all()


@pytest.mark.parametrize("value", [1e30, 1e-25, 3e-39, 1.2e19, 1e-18])
def test_squares_outside_fp32(value):
    ts = [torch.full((5000,), value, device="cuda"), torch.zeros(100, device="cuda")]
    check(ts, 1.0 if value > 1 else value)
    mixed = [torch.tensor([value, 0.0, 1.0], device="cuda"), torch.tensor([value], device="cuda")]
    check(mixed, 0.25)


def test_zeros_and_max_norm_zero():
    z = [torch.zeros(1000, device="cuda"), torch.zeros(3, device="cuda", dtype=BF)]
    check(z, 0.0)
    ts = make([1000], [FP])
    moe.moe_clip_grad_norm(ts, 0.0)
    assert not ts[0].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_a_norm_that_is_not_finite_leaves_the_values(bad, dtype):
    ts = make([5000, 70], [dtype, FP])
    ts[0][1234] = bad
    before = [t.clone() for t in ts]
    norm = moe.moe_clip_grad_norm(ts, 0.1).item()
    assert not math.isfinite(norm) and math.isnan(norm) == math.isnan(bad)
    out = [torch.zeros_like(t) for t in ts]
    moe.moe_clip_grad_norm(ts, 0.1, out=out)
    for t, b, o in zip(ts, before, out):
        assert torch.equal(t.nan_to_num(3.0), b.nan_to_num(3.0)) and torch.equal(o.nan_to_num(3.0), b.nan_to_num(3.0))


def test_more_values_than_32_bits_count():
    t = torch.zeros((1 << 32) + 5, dtype=BF, device="cuda")
    t[-1], t[0], t[1 << 31] = 3.0, 4.0, 12.0
    assert moe.moe_clip_grad_norm([t], 6.5).item() == 13.0
    assert t[-1] == 1.5 and t[0] == 2.0 and t[1 << 31] == 6.0


def test_same_result_every_call_and_on_another_stream():
    ts = make([300001, 77, 123456], [BF, FP, HF])
    a = moe.moe_grad_norm(ts)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = moe.moe_grad_norm(ts, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
