"""The training operators' checks of the memory that a call names, and the scratch memory that they ask for.
No GPU needed, and none used: the addresses are made up, so that calls are not tried where a kernel
could be launched on them."""
import ctypes

import pytest
import torch

from test_train_abi import BF, FP, INVALID, L, at  # noqa: F401

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses")
ACCEPTED = (3, 4)  # past the checks: there is no device here


def off(mib, n):
    return ctypes.c_void_p((mib << 20) + n)


def test_layer_norm_workspace_follows_the_rows(L):  # noqa: F811
    """No more partial sums than rows."""
    size = L.moe_layer_norm_workspace_size
    for K in (8, 1000, 1111, 1 << 16, 1 << 20, 1 << 24):
        assert 0 < size(1, K) <= 2 * K * 4
        assert 0 < size(5, K) <= 5 * 2 * K * 4
        assert size(0, K) <= size(1, K) <= size(100, K) <= size(1 << 20, K)
    assert size(1 << 20, 2048) == size(1 << 30, 2048)


# Each call with its pointers, all but the big operands' (their checks are in test_train_abi), and what they
# point to. The other arguments are small and right.
def calls(L):  # noqa: F811
    def layer_norm(mean=at(5), rstd=at(6)):
        return L.moe_layer_norm(at(1), 64, 512, BF, at(2), at(3), FP, 1e-5, at(4), mean, rstd, None)

    def layer_norm_backward(mean=at(4), rstd=at(5)):
        return L.moe_layer_norm_backward(at(1), at(2), 64, 512, BF, at(3), FP, mean, rstd, at(6), at(7), at(8), at(64),
                                         16 << 20, None)

    def router(z):
        fn = L.moe_router_topk if z == 4 else L.moe_router_topk_i64
        return lambda bias=at(2), weights=at(3), ids=at(4): fn(at(1), 64, 128, BF, 8, 0, bias, 1, 1.0, weights, ids, None)

    def router_backward(z):
        fn = L.moe_router_topk_backward if z == 4 else L.moe_router_topk_backward_i64
        return lambda ids=at(2), weights=at(3): fn(at(1), 64, 128, BF, ids, 8, 0, 1, 1.0, weights, at(4), None)

    def grouped(fn):
        return lambda offsets=at(3), counts=at(4): fn(at(1), 256, at(2), 4, 64, 64, offsets, counts, BF, BF, at(5), None)

    def wgrad(offsets=at(3), counts=at(4)):
        return L.moe_grouped_matmul_wgrad(at(1), at(2), 256, 4, 64, 64, offsets, counts, BF, BF, at(5), None, 0, None)
    return [(layer_norm, dict(mean=4, rstd=4)), (layer_norm_backward, dict(mean=4, rstd=4)),
            (router(4), dict(bias=4, weights=4, ids=4)), (router(8), dict(bias=4, weights=4, ids=8)),
            (router_backward(4), dict(ids=4, weights=4)), (router_backward(8), dict(ids=8, weights=4)),
            (grouped(L.moe_grouped_matmul), dict(offsets=4, counts=4)),
            (grouped(L.moe_grouped_matmul_dgrad), dict(offsets=4, counts=4)), (wgrad, dict(offsets=4, counts=4))]


@no_gpu
def test_every_pointer_is_aligned_to_its_elements(L):  # noqa: F811
    for call, sizes in calls(L):
        assert call() in ACCEPTED
        for name, z in sizes.items():
            for shift in (1, z // 2):
                assert call(**{name: off(30, shift)}) == INVALID, (call, name, shift)
            assert call(**{name: off(30, z)}) in ACCEPTED


@no_gpu
def test_layer_norm_overlaps(L):  # noqa: F811
    M, K = 64, 512

    def fwd(x=at(1), w=at(2), b=at(3), y=at(4), mean=at(5), rstd=at(6)):
        return L.moe_layer_norm(x, M, K, BF, w, b, FP, 1e-5, y, mean, rstd, None)
    assert fwd() in ACCEPTED and fwd(y=at(1)) in ACCEPTED and fwd(mean=None, rstd=None) in ACCEPTED
    for bad in (dict(mean=off(1, 64)), dict(rstd=off(1, 64)),                    # rows that other blocks read later
                dict(mean=off(4, 64)), dict(rstd=off(4, 64)), dict(rstd=off(5, 4)),
                dict(mean=at(2)), dict(rstd=at(3))):
        assert fwd(**bad) == INVALID, bad

    def bwd(dy=at(1), x=at(2), w=at(3), mean=at(4), rstd=at(5), dx=at(6), dw=at(7), db=at(8), ws=at(64)):
        return L.moe_layer_norm_backward(dy, x, M, K, BF, w, FP, mean, rstd, dx, dw, db, ws, 16 << 20, None)
    assert bwd() in ACCEPTED and bwd(dx=at(1)) in ACCEPTED and bwd(db=None) in ACCEPTED
    # the column sums are written once everything has been read
    assert bwd(dw=at(3)) in ACCEPTED and bwd(dw=at(4), db=off(2, 64)) in ACCEPTED
    for bad in (dict(dx=at(3)), dict(dx=at(4)), dict(dx=at(5)),
                dict(dw=at(6)), dict(db=off(6, 64)), dict(db=off(7, 64)), dict(dw=off(64, 64)), dict(db=off(64, 64)),
                dict(w=off(64, 64)), dict(mean=off(64, 64)), dict(rstd=off(64, 64))):
        assert bwd(**bad) == INVALID, bad


@no_gpu
def test_router_overlaps(L):  # noqa: F811
    for fn in (L.moe_router_topk, L.moe_router_topk_i64):
        def fwd(x=at(1), bias=at(2), w=at(3), i=at(4)):
            return fn(x, 64, 128, BF, 8, 0, bias, 1, 1.0, w, i, None)
        assert fwd() in ACCEPTED and fwd(bias=None) in ACCEPTED
        for bad in (dict(w=off(2, 64)), dict(i=off(2, 64))):            # the bias that other blocks read later
            assert fwd(**bad) == INVALID, bad


@no_gpu
def test_grouped_overlaps(L):  # noqa: F811
    def fwd(a=at(1), w=at(2), off_=at(3), cnt=at(4), out=at(5), fn=L.moe_grouped_matmul):
        return fn(a, 256, w, 4, 64, 64, off_, cnt, BF, BF, out, None)
    for fn in (L.moe_grouped_matmul, L.moe_grouped_matmul_dgrad):
        assert fwd(fn=fn) in ACCEPTED and fwd(fn=fn, cnt=None) in ACCEPTED
        for bad in (dict(off_=off(5, 64)), dict(cnt=off(5, 64))):
            assert fwd(fn=fn, **bad) == INVALID, bad
    need = L.moe_grouped_matmul_wgrad_workspace_size(8192, 1, 128, 2048)
    assert need > 0

    def wgrad(off_=at(3), cnt=at(4), out=at(1 << 14), ws=at(1 << 16)):
        return L.moe_grouped_matmul_wgrad(at(1 << 10), at(1 << 12), 8192, 1, 128, 2048, off_, cnt, BF, FP, out, ws, need, None)
    assert wgrad() in ACCEPTED and wgrad(cnt=None) in ACCEPTED
    for bad in (dict(off_=off(1 << 14, 64)), dict(cnt=off(1 << 14, 64)), dict(off_=off(1 << 16, 64)),
                dict(cnt=off(1 << 16, 64))):
        assert wgrad(**bad) == INVALID, bad


@no_gpu
def test_clip_overlaps(L):  # noqa: F811
    def call(ptrs, lens, outs=None, clip=True, norm=at(100), ws=at(101)):
        n = len(lens)
        p, c, t = (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*lens), (ctypes.c_int32 * n)(*([FP] * n))
        if not clip:
            return L.moe_grad_norm(p, c, t, n, norm, ws, 1 << 20, None)
        o = None if outs is None else (ctypes.c_void_p * n)(*outs)
        return L.moe_clip_grad_norm(p, c, t, n, 1.0, o, norm, ws, 1 << 20, None)
    a, b, c, d = 1 << 20, 2 << 20, 3 << 20, 4 << 20
    assert call([a, b], [1000, 10]) in ACCEPTED and call([a, b], [1000, 10], [c, d]) in ACCEPTED
    assert call([a, b], [1000, 10], [a, d]) in ACCEPTED and call([a, b], [1000, 10], [c, b]) in ACCEPTED
    # neighbours touch but do not overlap; an empty tensor overlaps nothing
    assert call([a, a + 4000], [1000, 10]) in ACCEPTED and call([a + 4000, a], [10, 1000]) in ACCEPTED
    assert call([a, a + 40, b], [1000, 0, 5]) in ACCEPTED
    # read only: a tensor may be there twice
    assert call([a, a], [1000, 1000], clip=False) in ACCEPTED and call([a, a], [1000, 10], [c, d]) in ACCEPTED
    # scaled twice, or read after another tensor's output has gone over it
    assert call([a, a], [1000, 1000]) == INVALID and call([a, a + 400], [1000, 10]) == INVALID
    assert call([b, a + 400, c, a], [10, 10, 10, 1000]) == INVALID
    assert call([a, b], [1000, 10], [c, c + 400]) == INVALID and call([a, b], [1000, 10], [b, d]) == INVALID
    assert call([a, b], [1000, 10], [c, a + 400]) == INVALID and call([a, a], [1000, 1000], [a, c]) == INVALID
    # the norm is written while tensors and partial sums are still read; moe_grad_norm writes it last
    for norm in (off(1, 400), off(101, 64)):
        assert call([a, b], [1000, 10], norm=norm) == INVALID
        assert call([a, b], [1000, 10], clip=False, norm=norm) in ACCEPTED
    assert call([a, b], [1000, 10], [c, d], norm=off(3, 400)) == INVALID
    # a long list
    many = [a + 64 * i for i in range(1000)]
    assert call(many, [16] * 1000) in ACCEPTED and call(many[::-1], [16] * 1000) in ACCEPTED
    assert call(many, [16] * 700 + [17] + [16] * 299) == INVALID
