"""The training operators under autograd: what a user of `train` may do with them."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train

pytestmark = pytest.mark.gpu


def test_layer_norm_without_a_bias():
    x = torch.randn(40, 256, device="cuda").requires_grad_()
    w = torch.randn(256, device="cuda").requires_grad_()
    dy = torch.randn(40, 256, device="cuda")
    train.layer_norm(x, w, None).backward(dy)
    _, mean, rstd = moe.moe_layer_norm(x.detach(), w.detach())
    dx, dw, _ = moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    again = moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd, has_bias=False)
    assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[1], dw)
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd, d_bias=torch.empty_like(dw), has_bias=False)


def test_rows_of_no_group_have_no_gradient():
    """Rows between the groups take no part in the product: their gradient is 0, whatever the memory
    that it is written to held before."""
    counts, K, N = [3, 0, 130, 64], 136, 72
    starts = [5, 133, 140, 300]
    R = 400
    off = torch.tensor(starts + [R], dtype=torch.int32, device="cuda")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    inside = torch.zeros(R, dtype=torch.bool, device="cuda")
    for s, c in zip(starts, counts):
        inside[s:s + c] = True
    w = torch.randn(4, N, K, device="cuda").bfloat16().requires_grad_()
    for cnt_or_none, rows in ((cnt, inside), (None, torch.arange(R, device="cuda") >= starts[0])):
        x = torch.randn(R, K, device="cuda").bfloat16().requires_grad_()
        y = train.grouped_matmul(x, w, off, cnt_or_none)
        dy = torch.zeros_like(y)
        dy[rows] = 1.0
        poison = [torch.full((R, K), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        del poison
        dx, = torch.autograd.grad(y, x, dy)
        assert (dx[~rows] == 0).all()
        want = moe.moe_grouped_matmul_dgrad(dy, w.detach(), off, cnt_or_none)
        assert torch.equal(dx[rows], want[rows])


def first_gradient(name):
    """x and a gradient with respect to it that was taken with create_graph."""
    if name == "layer_norm":
        x = torch.randn(8, 64, device="cuda").requires_grad_()
        y = train.layer_norm(x, torch.ones(64, device="cuda"), torch.zeros(64, device="cuda"))
    elif name == "router_topk":
        x = torch.randn(8, 64, device="cuda").requires_grad_()
        y, _ = train.router_topk(x, 4)
    elif name == "grouped_matmul":
        x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_()
        w = torch.randn(2, 64, 64, device="cuda").bfloat16().requires_grad_()
        y = train.grouped_matmul(x, w, torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    else:
        x = torch.randn(40, 128, device="cuda").bfloat16().requires_grad_()
        ids = torch.randint(0, 8, (40, 1), dtype=torch.int32, device="cuda")
        weights = torch.rand(40, 1, device="cuda")
        rows, _, src2dst, counts = train._Permute.apply(x, ids, weights, 8)
        if name == "permute":
            y = rows
        else:
            y = train._WeightedGather.apply(rows, src2dst, weights, ids, counts)
    return x, torch.autograd.grad(y.float().square().sum(), x, create_graph=True)[0]


@pytest.mark.parametrize("name", ["layer_norm", "router_topk", "grouped_matmul", "permute", "weighted_gather"])
def test_second_gradients_are_refused(name):
    """The functions have no second gradients; asking for one is an error and not a missing term."""
    x, g = first_gradient(name)
    with pytest.raises(RuntimeError):
        (g.float().square().sum() + x.float().square().sum()).backward()


def test_block_in_a_graph():
    """The block's forward and backward pass, captured and replayed on other inputs."""
    M, K, N, E, topk = 200, 256, 128, 8, 2
    p = train.init_block(K, N, E, seed=5)
    x = torch.randn(M, K, device="cuda").bfloat16().requires_grad_()
    dout = torch.randn(M, K, device="cuda").bfloat16()

    def step():
        out = train.moe_block(p, x, topk)
        return [out, *torch.autograd.grad(out, [x, *p.values()], dout)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    with torch.no_grad():
        x.copy_(torch.randn(M, K, device="cuda"))
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_memory_of_the_weighted_gathers_backward():
    """Beside its results the backward pass holds a few tensors of tokens x hidden size, not of every
    token's chosen rows."""
    M, K, E, topk = 2048, 2048, 16, 8
    ids = torch.stack([torch.randperm(E)[:topk] for _ in range(M)]).int().cuda()
    weights = torch.rand(M, topk, device="cuda").requires_grad_()
    h = torch.randn(M, K, device="cuda").bfloat16()
    rows, _, src2dst, counts = train._Permute.apply(h, ids, weights, E)
    rows = rows.detach().requires_grad_()
    dout = torch.randn(M, K, device="cuda").bfloat16()
    out = train._WeightedGather.apply(rows, src2dst, weights, ids, counts)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    drows, dweights = torch.autograd.grad(out, [rows, weights], dout)
    torch.cuda.synchronize()
    peak = torch.cuda.max_memory_allocated() - before
    results = drows.numel() * 2 + dweights.numel() * 4
    assert peak <= results + 6 * M * K * 4, (peak, results)
    kept = h.float()[:, None].expand(M, topk, K).double()
    ref = (kept * dout.double()[:, None]).sum(-1)
    # fp32 sums of K products, whatever their order
    assert ((dweights.double() - ref).abs() <= K * 2.0 ** -24 * (kept * dout.double()[:, None]).abs().sum(-1)).all()


def test_an_empty_list_of_gradients():
    """Without tensors the norm is 0; the buffer for it says where."""
    norm = torch.ones(1, device="cuda")
    assert moe.moe_grad_norm([], norm=norm).item() == 0
    norm.fill_(1)
    assert moe.moe_clip_grad_norm([], 1.0, norm=norm).item() == 0
    assert moe.moe_clip_grad_norm([], 1.0, out=[], norm=norm).item() == 0
