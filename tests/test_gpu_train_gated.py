"""The gated feed-forward part and the weighted sum under autograd, and the block they make.

With 16 bits kept the block makes fewer roundings than the one whose activation is made of torch
operations, so the bound of that one's test holds: eight roundings of at most 2^-8, 2^-5 in the relative
2-norm. Kept in 8 bits, the rows, gate, up and results enter the gradients with errors of at most 2^-4
relative each (2^-10 of a group's largest value where that is more); a gradient depends on at most three
of them (gate through the slope, up, and the rows or the results), each at most in proportion."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe
from moe_expert_layer_count_gb300 import train
from test_gpu_gated import U, inside, make, parts
from test_gpu_train import reference

pytestmark = pytest.mark.gpu
KEEPS = [moe.MOE_KEEP_16BIT, moe.MOE_KEEP_E4M3]


@pytest.mark.parametrize("keep", KEEPS)
@pytest.mark.parametrize("scoring,renormalize", [(moe.MOE_SCORE_SOFTMAX, True), (moe.MOE_SCORE_SIGMOID, False)])
def test_block_and_its_gradients(keep, scoring, renormalize):
    M, K, N, E, topk = 97, 256, 128, 8, 3
    p = train.init_block(K, N, E, seed=1)
    with torch.no_grad():  # weights large enough that every path contributes
        for name in ("gate", "w13", "w2"):
            p[name].mul_(4)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16().requires_grad_()
    dout = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    out = train.moe_block(p, x, topk, scoring, renormalize, keep=keep)
    out.backward(dout)
    h = train.layer_norm(x.detach(), p["norm_weight"].detach(), p["norm_bias"].detach())
    logits = moe.moe_grouped_matmul(h, p["gate"].detach(), torch.tensor([0, M], dtype=torch.int32, device="cuda"),
                                    out_dtype=torch.float32)
    _, ids = moe.moe_router_topk(logits, topk, scoring, renormalize)
    q, xr, ref = reference(p, x, ids, topk, renormalize, scoring)
    ref.backward(dout.double())

    def near(a, b, what, bound=2 ** -5 if keep == moe.MOE_KEEP_16BIT else 2 ** -5 + 3 * 2 ** -4):
        rel = ((a.double() - b).norm() / b.norm()).item()
        assert rel <= bound, (what, rel)
    near(out - x, ref - xr, "output", 2 ** -5)
    near(x.grad - dout, xr.grad - dout.double(), "input gradient")
    for name, v in p.items():
        near(v.grad, q[name].grad, name)
    assert moe.moe_device_error() == 0


def test_kept_in_8_bits_changes_the_gradients_only():
    M, K, N, E, topk = 150, 128, 256, 8, 2
    p = train.init_block(K, N, E, seed=7)
    x = torch.randn(M, K, device="cuda").bfloat16()
    a, b = (train.moe_block(p, x, topk, keep=k) for k in KEEPS)
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("keep", KEEPS)
def test_gated_experts_against_the_formula(dtype, act, keep):
    """Gradients in 64 bits from what was kept. Roundings: d_pre and h once each (u relative), the products' results
    once more; the sums' own errors are far below."""
    counts, N, K, gap = [33, 0, 130, 1], 144, 72, 5
    x, dy, w13, w2, _, off = make(counts, N, K, dtype, gap=gap, seed=8)
    R = x.shape[0]
    live = inside(off, counts, R)
    x[~live], dy[~live] = float("nan"), float("inf")
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    x, w13, w2 = x.requires_grad_(), w13.requires_grad_(), w2.requires_grad_()
    code = moe.MOE_ACT_SILU if act == "silu" else moe.MOE_ACT_GELU_TANH
    y = train.gated_experts(x, w13, w2, off, cnt, code, keep)
    dx, dw13, dw2 = torch.autograd.grad(y, [x, w13, w2], dy)
    assert not dx[~live].any()
    h, pre, scale = moe.moe_grouped_gated(x.detach(), w13.detach(), off, cnt, activation=code, keep=keep)
    rows = x.detach()
    if keep == moe.MOE_KEEP_E4M3:
        pre = moe.moe_checkpoint_unpack(pre, scale, dtype)
        rows = moe.moe_checkpoint_unpack(*moe.moe_checkpoint_pack(rows), dtype)
    u = U[dtype]

    def near(got, ref, mag, what):
        # two roundings of the factors and one of the result, and fp32 sums of up to 288 products
        tol = 3 * u * mag + 2.0 ** -14 * mag + 2.0 ** -24
        assert ((got.double() - ref).abs() <= tol).all(), (what, ((got.double() - ref).abs() - tol).max().item())
    for l, c in enumerate(counts):
        s = slice(int(off[l]), int(off[l]) + c)
        near(y[s], h[s].double() @ w2[l].double().T, h[s].double().abs() @ w2[l].double().abs().T, "y")
        dh = dy[s].double() @ w2[l].double()
        dh_mag = dy[s].double().abs() @ w2[l].double().abs()
        g, up = pre[s, :N].double(), pre[s, N:].double()
        a, slope, _, _ = parts(g, act)
        d = torch.cat([dh * up * slope, dh * a], 1)
        d_mag = torch.cat([dh_mag * (up * slope).abs(), dh_mag * a.abs()], 1)
        w = w13[l].double()
        near(dx[s], d @ w, d_mag @ w.abs(), "dx")
        near(dw13[l], d.T @ rows[s].double(), d_mag.T @ rows[s].double().abs(), "dw13")
        near(dw2[l], dy[s].double().T @ (a * up), dy[s].double().abs().T @ (a * up).abs(), "dw2")


def test_only_what_is_asked_for():
    counts, N, K = [40, 24], 64, 128
    x, dy, w13, w2, _, off = make(counts, N, K, torch.bfloat16, seed=12)
    want = None
    for mask in range(1, 8):
        t = [v.detach().clone().requires_grad_(bool(mask >> i & 1)) for i, v in enumerate((x, w13, w2))]
        y = train.gated_experts(*t, off)
        y.backward(dy)
        got = [v.grad for v in t]
        assert [g is not None for g in got] == [bool(mask >> i & 1) for i in range(3)]
        if mask == 7:
            want = got
    for mask in range(1, 7):
        t = [v.detach().clone().requires_grad_(bool(mask >> i & 1)) for i, v in enumerate((x, w13, w2))]
        train.gated_experts(*t, off).backward(dy)
        for v, w in zip(t, want):
            assert v.grad is None or torch.equal(v.grad, w)


@pytest.mark.parametrize("keep", KEEPS)
def test_frozen_weights_keep_no_rows(keep):
    """What only a frozen input's gradient would need is not kept, and the other gradients are the same."""
    M, K, N, E, topk = 512, 256, 128, 8, 4
    p = train.init_block(K, N, E, seed=9)
    x = torch.randn(M, K, device="cuda").bfloat16()
    ids = torch.topk(torch.rand(M, E, device="cuda"), topk, dim=1).indices.int()
    rows, offsets, src2dst, counts = train._Permute.apply(x, ids, torch.rand(M, topk, device="cuda"), E)
    grads, held = {}, {}
    for frozen in (False, True):
        r = rows.detach().clone().requires_grad_()
        w13 = p["w13"].detach().clone().requires_grad_(not frozen)
        weights = torch.full((M, topk), 0.25, device="cuda", requires_grad=not frozen)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = train.weighted_sum(train.gated_experts(r, w13, p["w2"], offsets, counts, keep=keep), src2dst, weights, keep=keep)
        held[frozen] = torch.cuda.memory_allocated() - before
        grads[frozen] = torch.autograd.grad(out, [r, p["w2"]], torch.ones_like(out))
    assert all(torch.equal(a, b) for a, b in zip(grads[False], grads[True]))
    assert held[True] < held[False]


@pytest.mark.parametrize("keep", KEEPS)
def test_weighted_sum(keep):
    """The rows' gradient is that of the scatter; a weight's gradient is made of the rows as they were kept."""
    M, K, E, topk = 90, 256, 8, 3
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.topk(torch.rand(M, E, device="cuda", generator=g), topk, dim=1).indices.int()
    ids[::7, 1] = -1
    weights = torch.rand(M, topk, device="cuda", generator=g).requires_grad_()
    h = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    rows, _, src2dst, counts = train._Permute.apply(h, ids.contiguous(), weights, E)
    rows = rows.detach().requires_grad_()
    dout = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    out = train.weighted_sum(rows, src2dst, weights, keep)
    assert torch.equal(out, train._WeightedGather.apply(rows, src2dst, weights, ids, counts))
    drows, dweights = torch.autograd.grad(out, [rows, weights], dout)
    kept = src2dst >= 0
    at = src2dst[kept].long()
    dead = torch.ones(rows.shape[0], dtype=torch.bool, device="cuda")
    dead[at] = False
    assert not drows[dead].any()
    assert torch.equal(drows[at], (weights[..., None] * dout.float()[:, None]).bfloat16()[kept])
    values = rows.detach()
    if keep == moe.MOE_KEEP_E4M3:
        values = moe.moe_checkpoint_unpack(*moe.moe_checkpoint_pack(values), torch.bfloat16)
    prod = values[src2dst.clamp(min=0).long()].double() * dout.double()[:, None]
    ref, mag = torch.where(kept, prod.sum(-1), 0.0), prod.abs().sum(-1)
    assert ((dweights.double() - ref).abs() <= K * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("name", ["gated_experts", "weighted_sum"])
def test_second_gradients_are_refused(name):
    if name == "gated_experts":
        x = torch.randn(8, 64, device="cuda").bfloat16().requires_grad_()
        w13 = torch.randn(2, 64, 64, device="cuda").bfloat16().requires_grad_()
        w2 = torch.randn(2, 64, 32, device="cuda").bfloat16().requires_grad_()
        y = train.gated_experts(x, w13, w2, torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda"))
    else:
        x = torch.randn(8, 128, device="cuda").bfloat16().requires_grad_()
        y = train.weighted_sum(x, torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2), torch.rand(4, 2, device="cuda"))
    first = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        (first.float().square().sum() + x.float().square().sum()).backward()


@pytest.mark.parametrize("keep", KEEPS)
def test_block_in_a_graph(keep):
    """The block's forward and backward pass, captured and replayed on other inputs."""
    M, K, N, E, topk = 200, 256, 128, 8, 2
    p = train.init_block(K, N, E, seed=5)
    x = torch.randn(M, K, device="cuda").bfloat16().requires_grad_()
    dout = torch.randn(M, K, device="cuda").bfloat16()

    def step():
        out = train.moe_block(p, x, topk, keep=keep)
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


@pytest.mark.parametrize("keep", KEEPS)
def test_twice_through_one_graph(keep):
    """Nothing that is kept is used up: a second backward pass gives the same gradients."""
    p = train.init_block(128, 128, 8, seed=6)
    x = torch.randn(70, 128, device="cuda").bfloat16().requires_grad_()
    out = train.moe_block(p, x, 2, keep=keep)
    dout = torch.randn_like(out)
    a = torch.autograd.grad(out, [x, *p.values()], dout, retain_graph=True)
    b = torch.autograd.grad(out, [x, *p.values()], dout)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_memory_that_is_kept():
    """Bytes held between the passes: rows, gate and up and results in 16 or in 8 bits, beside tensors of
    tokens x hidden size and smaller ones."""
    M, K, N, E, topk = 2048, 1024, 512, 16, 8
    p = train.init_block(K, N, E)
    x = torch.randn(M, K, device="cuda").bfloat16()
    R = moe.moe_rp_cap(M, topk, E)
    big = R * (K + 2 * N + K)
    held = {}
    for keep in KEEPS:
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        out = train.moe_block(p, x, topk, keep=keep)
        held[keep] = torch.cuda.memory_allocated() - before
        del out
    small = 4 * M * K * 2 + 64 * M * topk
    assert held[moe.MOE_KEEP_16BIT] <= 2 * big + small
    assert held[moe.MOE_KEEP_E4M3] <= big * 17 // 16 + small


@pytest.mark.parametrize("keep", ["16bit", "8bit"])
def test_command(keep, capsys):
    train.main(["--keep", keep])
    lines = capsys.readouterr().out.strip().splitlines()
    assert len(lines) == 5 and all("loss" in x for x in lines)


def test_without_gradients_nothing_is_kept():
    counts, N, K = [40, 24], 64, 128
    x, _, w13, w2, _, off = make(counts, N, K, torch.bfloat16, seed=3)
    w13.requires_grad_()
    want = train.gated_experts(x, w13, w2, off)
    with torch.no_grad():
        launches = moe.moe_kernel_launch_count()
        y = train.gated_experts(x, w13, w2, off, keep=moe.MOE_KEEP_E4M3)
        z = train.weighted_sum(y, torch.arange(64, dtype=torch.int32, device="cuda").view(32, 2), torch.ones(32, 2, device="cuda"),
                               keep=moe.MOE_KEEP_E4M3)
        assert moe.moe_kernel_launch_count() - launches == 3  # two products and the sum
    assert torch.equal(y, want) and not z.requires_grad
    for bad in (moe.MOE_KEEP_NONE, 7, None):
        with pytest.raises(ValueError):
            train.gated_experts(x, w13, w2, off, keep=bad)
