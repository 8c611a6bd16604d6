"""The training operators write their outputs and nothing beside them, and can be captured in a
CUDA graph. Outputs lie between guard values in a larger buffer, at sizes that no tile or
vector divides."""
import pytest
import torch

import moe_expert_layer_count_gb300 as moe

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


class Guarded:
    """Buffers with 64 guard elements on both sides."""

    def __init__(self):
        self.all = []

    def empty(self, shape, dtype):
        n = 1
        for d in shape:
            n *= d
        buf = torch.full((n + 128,), 77, dtype=dtype, device="cuda")
        self.all.append((buf, n))
        return buf[64:64 + n].view(shape)

    def check(self):
        torch.cuda.synchronize()
        for buf, n in self.all:
            assert (buf[:64] == 77).all() and (buf[64 + n:] == 77).all()


@pytest.mark.parametrize("M,K", [(1, 1), (5, 1111), (33, 264), (7, 2049), (300, 96), (2, 16384), (3, 20000), (64, 2048)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_layer_norm(M, K, dtype):
    g = Guarded()
    x, dy = torch.randn(M, K, device="cuda").to(dtype), torch.randn(M, K, device="cuda").to(dtype)
    w = torch.ones(K, device="cuda")
    y, mean, rstd = moe.moe_layer_norm(x, w, w, out=g.empty((M, K), dtype), mean=g.empty((M,), FP), rstd=g.empty((M,), FP))
    ws = g.empty((moe.moe_layer_norm_workspace_size(M, K),), torch.uint8)
    moe.moe_layer_norm_backward(dy, x, w, mean, rstd, dx=g.empty((M, K), dtype), d_weight=g.empty((K,), FP),
                                d_bias=g.empty((K,), FP), workspace=ws)
    g.check()


@pytest.mark.parametrize("M,E,topk", [(1, 3, 2), (37, 61, 5), (9, 1000, 13), (5, 64, 20), (16401, 128, 7)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_router(M, E, topk, dtype):
    g = Guarded()
    logits = torch.randn(M, E, device="cuda").to(dtype)
    w, ids = moe.moe_router_topk(logits, topk, topk_weights=g.empty((M, topk), FP), topk_ids=g.empty((M, topk), torch.int32))
    for renorm in (False, True):
        moe.moe_router_topk_backward(logits, ids, torch.ones(M, topk, device="cuda"), renormalize=renorm,
                                     d_logits=g.empty((M, E), dtype))
    g.check()


@pytest.mark.parametrize("counts,N,K", [([1], 8, 8), ([5, 0, 300], 72, 136), ([17] * 30, 264, 200), ([257, 255], 520, 264)])
@pytest.mark.parametrize("out_dtype", [BF, FP])
def test_grouped_products(counts, N, K, out_dtype):
    g = Guarded()
    R, E = sum(counts), len(counts)
    off = torch.tensor([sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    x, dy = torch.randn(R, K, device="cuda").bfloat16(), torch.randn(R, N, device="cuda").bfloat16()
    w = torch.randn(E, N, K, device="cuda").bfloat16()
    moe.moe_grouped_matmul(x, w, off, out=g.empty((R, N), out_dtype))
    moe.moe_grouped_matmul_dgrad(dy, w, off, out=g.empty((R, K), out_dtype))
    moe.moe_grouped_matmul_wgrad(dy, x, off, out=g.empty((E, N, K), out_dtype))
    g.check()


def test_clip():
    g = Guarded()
    sizes = [1, 9, 16385, 70000, 3, 131071]
    types = [BF, FP, HF, BF, FP, FP]
    ts = [torch.randn(n, device="cuda").to(t) for n, t in zip(sizes, types)]
    ws = g.empty((moe.moe_grad_norm_workspace_size(sizes),), torch.uint8)
    moe.moe_clip_grad_norm(ts, 0.5, out=[g.empty((n,), t) for n, t in zip(sizes, types)], norm=g.empty((1,), FP), workspace=ws)
    g.check()


def test_capture_and_replay():
    M, K, N, E, topk = 304, 256, 128, 16, 4  # every row in a group
    x = torch.randn(M, K, device="cuda").bfloat16()
    w = torch.randn(E, N, K, device="cuda").bfloat16()
    wg = torch.randn(1, E, K, device="cuda").bfloat16()
    gamma = torch.ones(K, device="cuda")
    everyone = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    off = torch.arange(E + 1, dtype=torch.int32, device="cuda") * (M // E)
    work = [torch.empty(moe.moe_layer_norm_workspace_size(M, K), dtype=torch.uint8, device="cuda"),
            torch.empty(moe.moe_grad_norm_workspace_size([E * N * K, K]), dtype=torch.uint8, device="cuda")]

    def step():
        h, mean, rstd = moe.moe_layer_norm(x, gamma, gamma)
        logits = moe.moe_grouped_matmul(h, wg, everyone, out_dtype=FP)
        weights, ids = moe.moe_router_topk(logits, topk)
        dlogits = moe.moe_router_topk_backward(logits, ids, weights)
        y = moe.moe_grouped_matmul(h, w, off)
        dh = moe.moe_grouped_matmul_dgrad(y, w, off)
        dw = moe.moe_grouped_matmul_wgrad(y, h, off)
        dx, dgamma, dbeta = moe.moe_layer_norm_backward(dh, x, gamma, mean, rstd, workspace=work[0])
        norm = moe.moe_clip_grad_norm([dw, dgamma], 1.0, workspace=work[1])
        return [weights, ids, dlogits, y, dw, dgamma, dbeta, norm]
    expect = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(graph, stream=s):
            got = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, expect):
        assert torch.equal(a, b)
