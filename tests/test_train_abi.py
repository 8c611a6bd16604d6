"""The training operators' argument checks: each documented error is returned before any
launch, and the binding refuses tensors of the wrong type, shape or place. No GPU needed."""
import ctypes

import pytest
import torch

INVALID, SMALL = 1, 2
BF, HF, FP = 1, 2, 0


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_layer_count_gb300 as moe
    return moe.lib()


def at(mib):
    return ctypes.c_void_p(mib << 20)


def test_layer_norm_refusals(L):
    def fwd(x=at(1), M=4, K=64, dt=BF, w=at(2), b=at(3), pdt=BF, eps=1e-5, y=at(4)):
        return L.moe_layer_norm(x, M, K, dt, w, b, pdt, eps, y, at(5), at(6), None)
    assert fwd(M=0) == 0
    assert fwd(M=-1) == INVALID and fwd(K=0) == INVALID and fwd(dt=5) == INVALID and fwd(K=(1 << 24) + 1) == INVALID
    assert fwd(pdt=HF) == INVALID                                   # neither x's type nor fp32
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID
    assert fwd(x=None) == INVALID and fwd(w=None) == INVALID and fwd(y=None) == INVALID
    assert fwd(x=ctypes.c_void_p((1 << 20) + 1)) == INVALID         # not aligned to its element
    assert fwd(y=ctypes.c_void_p((1 << 20) + 64)) == INVALID        # overlaps x
    assert fwd(y=at(2)) == INVALID                                  # overlaps the weight
    assert L.moe_layer_norm_workspace_size(4, 0) == 0 and L.moe_layer_norm_workspace_size(-1, 8) == 0
    need = L.moe_layer_norm_workspace_size(4, 64)
    assert need > 0

    def bwd(dy=at(1), x=at(2), M=4, K=64, dt=BF, w=at(3), pdt=FP, mean=at(4), dx=at(5), dw=at(6), db=at(7), ws=at(64),
            nb=None):
        return L.moe_layer_norm_backward(dy, x, M, K, dt, w, pdt, mean, at(8), dx, dw, db, ws, need if nb is None else nb,
                                         None)
    assert bwd(nb=need - 1) == SMALL and bwd(ws=None) == INVALID and bwd(dw=None) == INVALID
    assert bwd(ws=ctypes.c_void_p((64 << 20) + 8)) == INVALID
    assert bwd(mean=None) == INVALID and bwd(dy=None) == INVALID and bwd(dx=at(2)) == INVALID
    assert bwd(pdt=HF) == INVALID and bwd(K=-3) == INVALID and bwd(dx=at(64)) == INVALID


def test_router_refusals(L):
    for fn in (L.moe_router_topk, L.moe_router_topk_i64):
        def fwd(x=at(1), M=4, E=64, dt=BF, k=8, sc=0, w=at(2), i=at(3)):
            return fn(x, M, E, dt, k, sc, None, 1, 1.0, w, i, None)
        assert fwd(M=0) == 0
        assert fwd(M=-1) == INVALID and fwd(E=0) == INVALID and fwd(E=1025) == INVALID and fwd(k=0) == INVALID
        assert fwd(k=33) == INVALID and fwd(E=4) == INVALID         # more choices than experts
        assert fwd(dt=3) == INVALID and fwd(sc=2) == INVALID and fwd(M=1 << 29) == INVALID
        assert fwd(x=None) == INVALID and fwd(w=None) == INVALID and fwd(i=None) == INVALID
        assert fwd(w=at(1)) == INVALID and fwd(i=at(1)) == INVALID and fwd(i=at(2)) == INVALID   # overlaps
    for fn in (L.moe_router_topk_backward, L.moe_router_topk_backward_i64):
        def bwd(x=at(1), M=4, E=64, dt=BF, i=at(2), k=8, sc=0, g=at(3), d=at(4)):
            return fn(x, M, E, dt, i, k, sc, 1, 1.0, g, d, None)
        assert bwd(M=0) == 0
        assert bwd(k=0) == INVALID and bwd(E=2000) == INVALID and bwd(dt=-1) == INVALID and bwd(sc=-1) == INVALID
        assert bwd(x=None) == INVALID and bwd(i=None) == INVALID and bwd(g=None) == INVALID and bwd(d=None) == INVALID
        assert bwd(d=at(2)) == INVALID and bwd(d=at(3)) == INVALID
        assert bwd(d=ctypes.c_void_p((1 << 20) + 128)) == INVALID   # overlaps the logits, not exactly


def test_grouped_matmul_refusals(L):
    off = at(100)

    def fwd(a=at(1), R=16, w=at(2), El=4, N=64, K=64, off=off, dt=BF, odt=BF, out=at(3), fn=L.moe_grouped_matmul):
        return fn(a, R, w, El, N, K, off, None, dt, odt, out, None)
    for fn in (L.moe_grouped_matmul, L.moe_grouped_matmul_dgrad):
        assert fwd(R=0, fn=fn) == 0
        for bad in (dict(El=0), dict(El=1025), dict(N=60), dict(K=4), dict(N=0), dict(R=-1), dict(R=1 << 31), dict(dt=FP),
                    dict(dt=7), dict(odt=HF), dict(off=None), dict(a=None), dict(w=None), dict(out=None),
                    dict(a=ctypes.c_void_p((1 << 20) + 8)), dict(out=ctypes.c_void_p((3 << 20) + 8)), dict(out=at(1)),
                    dict(out=at(2))):
            assert fwd(fn=fn, **bad) == INVALID, bad

    def wgrad(dy=at(1), x=at(2), R=16, El=4, N=64, K=64, off=off, dt=BF, odt=FP, out=at(3), ws=None, nb=0):
        return L.moe_grouped_matmul_wgrad(dy, x, R, El, N, K, off, None, dt, odt, out, ws, nb, None)
    for bad in (dict(El=0), dict(N=4), dict(K=12), dict(R=-1), dict(dt=FP), dict(odt=HF), dict(off=None), dict(dy=None),
                dict(x=None), dict(out=None), dict(R=0, out=None), dict(out=at(1)), dict(out=at(2))):
        assert wgrad(**bad) == INVALID, bad
    # few weights, many rows: the sum is split and needs scratch
    size = L.moe_grouped_matmul_wgrad_workspace_size
    assert size(16, 4, 64, 64) == 0 and size(-1, 4, 64, 64) == 0 and size(100, 0, 64, 64) == 0
    assert size(65536, 128, 1536, 2048) == 0
    need = size(8192, 1, 128, 2048)
    assert need >= 2 * 128 * 2048 * 4
    big = dict(R=8192, El=1, N=128, K=2048, dy=at(1 << 10), x=at(1 << 12), out=at(1 << 14))
    assert wgrad(**big) == SMALL and wgrad(**big, ws=at(1 << 16), nb=need - 1) == SMALL
    assert wgrad(**big, ws=at(1 << 12), nb=need) == INVALID and wgrad(**big, ws=ctypes.c_void_p((1 << 36) + 8), nb=need) == INVALID


def test_grad_norm_refusals(L):
    def arrays(ptrs, lens, types):
        n = len(lens)
        return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*lens), (ctypes.c_int32 * n)(*types), n
    good = arrays([1 << 20, 2 << 20], [1000, 0], [BF, FP])
    need = L.moe_grad_norm_workspace_size(good[1], 2)
    assert need > 0 and L.moe_grad_norm_workspace_size(good[1], -1) == 0
    assert L.moe_grad_norm_workspace_size((ctypes.c_int64 * 1)(-5), 1) == 0

    def norm(a=good, out=at(8), ws=at(9), nb=need):
        return L.moe_grad_norm(*a, out, ws, nb, None)
    assert norm(nb=need - 1) == SMALL
    assert norm(out=None) == INVALID and norm(ws=None) == INVALID and norm(ws=ctypes.c_void_p((9 << 20) + 8)) == INVALID
    assert norm(arrays([1 << 20], [-1], [BF])) == INVALID and norm(arrays([1 << 20], [5], [9])) == INVALID
    assert norm(arrays([0], [5], [BF])) == INVALID and norm(arrays([(1 << 20) + 1], [5], [BF])) == INVALID
    assert norm(arrays([9 << 20], [5], [BF])) == INVALID            # overlaps the workspace

    def clip(a=good, m=1.0, outs=None):
        return L.moe_clip_grad_norm(*a, m, outs, at(8), at(9), need, None)
    assert clip(m=-1.0) == INVALID and clip(m=float("nan")) == INVALID
    assert clip(outs=(ctypes.c_void_p * 2)((1 << 20) + 64, 3 << 20)) == INVALID   # overlaps, not exactly
    assert clip(outs=(ctypes.c_void_p * 2)(0, 0)) == INVALID


def test_binding_refusals(L):
    import moe_expert_layer_count_gb300 as moe
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    z = lambda *s, d=bf: torch.zeros(*s, dtype=d)
    with pytest.raises(ValueError):                                 # host tensors
        moe.moe_layer_norm(z(4, 8), z(8), z(8))
    with pytest.raises(TypeError):
        moe.moe_layer_norm(z(4, 8, d=torch.float64), z(8), z(8))
    with pytest.raises(ValueError):
        moe.moe_layer_norm(z(4, 8), z(9), z(9))
    with pytest.raises(ValueError):
        moe.moe_layer_norm_backward(z(4, 8), z(4, 9), z(9), z(4, d=f32), z(4, d=f32))
    with pytest.raises(ValueError):
        moe.moe_router_topk(z(4, 8), 2, bias=z(8))                  # the bias is fp32
    with pytest.raises(TypeError):
        moe.moe_router_topk(z(4, 8), 2, topk_ids=z(4, 2, d=torch.int16))
    with pytest.raises(ValueError):
        moe.moe_router_topk_backward(z(4, 8), z(4, 2, d=i32), z(4, 3, d=f32))
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul(z(4, 8), z(2, 8, 16), z(3, d=i32))   # rows of another width
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul(z(4, 16), z(2, 8, 16), z(2, d=i32))  # one offset too few
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul(z(4, 16), z(2, 8, 16, d=torch.float16), z(3, d=i32))   # two types
    with pytest.raises(ValueError):
        moe.moe_grouped_matmul_wgrad(z(4, 16), z(5, 16), z(3, d=i32))
    with pytest.raises(ValueError):
        moe.moe_clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        moe.moe_clip_grad_norm([z(4)], 1.0)
