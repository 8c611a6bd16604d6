"""Gradients of the weighted gather: the rows' gradient is one fp32 product rounded once, so it is exact
bit for bit; a weight's gradient is a sum of K products in fp32, in any order off by at most
K * 2^-24 * sum |y||dout| (products of bf16 values are exact)."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu


def make(M, topk, K, E, dropped=0.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.topk(torch.rand(M, E, device="cuda", generator=g), topk, dim=1).indices.int()
    ids[torch.rand(M, topk, device="cuda", generator=g) < dropped] = -1
    w = torch.rand(M, topk, device="cuda", generator=g)
    h = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    cnt = torch.empty(E, dtype=torch.int32, device="cuda")
    rows, _, _, src2dst = moe.moe_scatter(h, ids.contiguous(), w, E, E, cnt, quant=moe.MOE_QUANT_NONE, count_here=True)
    y = torch.full_like(rows, float("nan"))
    kept = src2dst >= 0
    y[src2dst[kept].long()] = torch.randn(int(kept.sum()), K, device="cuda", generator=g).bfloat16()
    dout = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    return dout, y, src2dst, w


def check(dout, y, src2dst, w, d_y, d_w, unit=False):
    kept = src2dst >= 0
    at = src2dst.clamp(min=0).long()
    want = ((1.0 if unit else w)[..., None] * dout.float()[:, None] if not unit else dout.float()[:, None].expand(*w.shape, -1)).bfloat16()
    assert torch.equal(d_y[at[kept]], want[kept])
    if d_w is not None:
        yy = torch.where(kept[..., None], y[at].double(), 0.0)
        ref, mag = (yy * dout.double()[:, None]).sum(-1), (yy * dout.double()[:, None]).abs().sum(-1)
        assert ((d_w.double() - ref).abs() <= y.shape[1] * 2.0 ** -24 * mag).all()
        assert not d_w[~kept].any()


@pytest.mark.parametrize("M,topk,K,E", [(1, 1, 128, 1), (1, 8, 2048, 16), (17, 2, 256, 8), (100, 8, 640, 32), (333, 3, 1152, 7),
                                        (64, 32, 128, 64), (50, 11, 384, 20), (1000, 1, 4096, 4), (5, 4, 16384, 8)])
@pytest.mark.parametrize("dropped", [0.0, 0.4, 1.0])
def test_gradients(M, topk, K, E, dropped):
    dout, y, src2dst, w = make(M, topk, K, E, dropped, seed=M + K)
    d_y = torch.full_like(y, 7.0)
    got, d_w = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, d_y=d_y)
    assert got is d_y
    check(dout, y, src2dst, w, d_y, d_w)
    free = torch.ones(y.shape[0], dtype=torch.bool, device="cuda")
    free[src2dst[src2dst >= 0].long()] = False
    assert (d_y[free] == 7).all()  # rows of no slot
    alone, none = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, d_y=torch.full_like(y, 7.0), want_weights=False)
    assert none is None and torch.equal(alone, d_y)
    unit, none = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, True, d_y=torch.full_like(y, 7.0))
    assert none is None
    check(dout, y, src2dst, w, unit, None, unit=True)


def test_as_the_scatter_of_the_gradient():
    """The rows' gradient is what moe_scatter makes of dout with the weights applied."""
    M, topk, K, E = 500, 4, 256, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.topk(torch.rand(M, E, device="cuda", generator=g), topk, dim=1).indices.int().contiguous()
    w = torch.rand(M, topk, device="cuda", generator=g)
    dout = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    cnt = torch.empty(E, dtype=torch.int32, device="cuda")
    want, _, _, src2dst = moe.moe_scatter(dout, ids, w, E, E, cnt, apply_router_weight_on_input=True, quant=moe.MOE_QUANT_NONE,
                                          count_here=True)
    got, _ = moe.moe_gather_weight_reduce_backward(dout, want, src2dst, w)
    rows = src2dst.reshape(-1).long()
    assert torch.equal(got[rows], want[rows])


def test_bad_rows_take_no_part():
    """A row outside [0, rows) is an empty slot."""
    dout, y, src2dst, w = make(40, 3, 256, 8, seed=9)
    bad = src2dst.clone()
    bad[::5, 1] = y.shape[0]
    bad[1::5, 0] = 2 ** 31 - 1
    bad[2::5, 2] = -(2 ** 31)
    band = torch.full((y.shape[0] + 32, y.shape[1]), 7.0, device="cuda").bfloat16()
    d_y, d_w = moe.moe_gather_weight_reduce_backward(dout, y, bad, w, d_y=band[:y.shape[0]])
    ok = (bad >= 0) & (bad < y.shape[0])
    check(dout, y, torch.where(ok, bad, -1), w, d_y, d_w)
    assert (band[y.shape[0]:] == 7).all()


def test_no_tokens_and_non_finite_values():
    dout, y, src2dst, w = make(20, 2, 128, 4, seed=2)
    d_y, d_w = moe.moe_gather_weight_reduce_backward(dout[:0], y, src2dst[:0], w[:0])
    assert d_w.shape == (0, 2)
    dout[3, 5] = float("inf")
    y[src2dst[7, 0].long(), 9] = float("nan")
    d_y, d_w = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w)
    bad = torch.zeros(20, 2, dtype=torch.bool, device="cuda")
    bad[3], bad[7, 0] = True, True
    assert torch.equal(~torch.isfinite(d_w), bad) and d_y[src2dst[3].long(), 5].isinf().all()


def test_rows_past_32_bits():
    rows, K = 600_000, 4096
    y = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    y[-2:] = 1.0
    src2dst = torch.tensor([[rows - 1], [rows - 2]], dtype=torch.int32, device="cuda")
    dout = torch.ones(2, K, dtype=torch.bfloat16, device="cuda")
    w = torch.tensor([[0.5], [0.25]], device="cuda")
    d_y = torch.zeros_like(y)
    _, d_w = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, d_y=d_y)
    assert (d_y[-1] == 0.5).all() and (d_y[-2] == 0.25).all() and not d_y[:-2].any() and (d_w == K).all()


def test_captured_and_on_another_stream():
    dout, y, src2dst, w = make(60, 4, 384, 8, seed=5)
    want = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, d_y=torch.zeros_like(y))
    d_y = torch.zeros_like(y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        _, d_w = moe.moe_gather_weight_reduce_backward(dout, y, src2dst, w, d_y=d_y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d_y, want[0]) and torch.equal(d_w, want[1])
